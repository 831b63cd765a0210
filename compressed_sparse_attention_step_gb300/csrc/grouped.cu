// Products of the token rows of each expert with its 4-bit weight (E2M1 codes, one E4M3 scale per 16 channels):
// y[r] = act(row_scale[e] * W_e x[src[r]]) for the rows offsets[e] <= r < offsets[e + 1] of expert e.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"

namespace csa2 {
namespace grp {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kRows = 32, kChan = 128;  // of a block of the packed weight (matvec.cu has its layout)
constexpr int kCodeBytes = kRows * kChan / 2;
constexpr int kBlock = kCodeBytes + kRows * kChan / CSA2_GROUP;
constexpr int kTok = 16;

struct Params {
  const uint16_t* x;
  const uint8_t* packed;
  const float* row_scale;
  const int32_t *offsets, *src;
  void* y;
  int64_t n_out, n_in, w_bytes;
  int64_t rows, n_x;
  int E, n_kb, n_rb, y_fp32, act;
  unsigned int* flags;
};

__device__ __forceinline__ int block_place(int r, int j) { return j * 512 + (r ^ (2 * j)) * 16; }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float silu(float v) { return v / (1.f + expf(-v)); }

// A CTA: eight row blocks of an expert, one a warp, and its rows 16 at a time.
__global__ void __launch_bounds__(kThreads) grouped_kernel(const Params p) {
  __shared__ uint4 xs[2][4][32];
  __shared__ float xf[kTok];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3, g = lane >> 2;
  const int e = blockIdx.y;
  const int64_t lo = min(max(int64_t(p.offsets[e]), int64_t(0)), p.rows), hi = min(max(int64_t(p.offsets[e + 1]), lo), p.rows);
  const int rb = int(blockIdx.x) * kWarps + warp;
  const uint8_t* w = p.packed + int64_t(e) * p.w_bytes + int64_t(min(rb, p.n_rb - 1)) * p.n_kb * kBlock;
  for (int64_t r0 = lo; r0 < hi; r0 += kTok) {
    float acc[2][2][4] = {};
    for (int kb = 0; kb < p.n_kb; ++kb) {
      __syncthreads();
      {  // half a warp per token, 8 channels a lane
        const int tok = tid >> 4, j = tid & 15;
        const int64_t ch = int64_t(kb) * kChan + 8 * j;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r0 + tok < hi && ch < p.n_in) {
          const int64_t s = p.src ? p.src[r0 + tok] : r0 + tok;
          if (s >= 0 && s < p.n_x) v = __ldg(reinterpret_cast<const uint4*>(p.x + s * p.n_in + ch));
          else if (s >= p.n_x && kb == 0 && j == 0 && blockIdx.x == 0) atomicOr(p.flags, CSA2_FLAG_INDEX_OOB);
        }
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) am = max(am, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
#pragma unroll
        for (int o = 8; o; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
        const int up = am ? min(max(141 - int(am >> 7), -126), 126) : 0;
        const float f = __uint_as_float(uint32_t(127 + up) << 23);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = attn::h2_bits(__floats2half2_rn(bf16lo(u[i]) * f, bf16hi(u[i]) * f));
        xs[tok >> 3][j & 3][(tok & 7) * 4 + (j >> 2)] = make_uint4(o[0], o[1], o[2], o[3]);
        if (j == 0) xf[tok] = __uint_as_float(uint32_t(127 - up) << 23);
      }
      __syncthreads();
      const uint8_t* blk = w + int64_t(kb) * kBlock;
      float d[2][2][4] = {};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint4 c[2];
        __half2 sc[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 16 * r + 8 * h + g;
          c[h] = __ldg(reinterpret_cast<const uint4*>(blk + block_place(row, t)));
          const __half2 s2 = attn::bits_h2(attn::e4m3x2_to_f16x2(__ldg(reinterpret_cast<const uint16_t*>(blk + kCodeBytes + row * 8 + 2 * t))));
          sc[h][0] = __low2half2(s2), sc[h][1] = __high2half2(s2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            attn::e2m1x8_to_f16x2x4(i == 0 ? c[h].x : i == 1 ? c[h].y : i == 2 ? c[h].z : c[h].w, a[h][0], a[h][1], a[h][2], a[h][3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) a[h][q] = attn::h2_bits(__hmul2(attn::bits_h2(a[h][q]), sc[h][i >> 1]));
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 xb = xs[j][i][lane];
            mma_f16(d[r][j], a[0][0], a[1][0], a[0][1], a[1][1], xb.x, xb.y);
            mma_f16(d[r][j], a[0][2], a[1][2], a[0][3], a[1][3], xb.z, xb.w);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f0 = xf[8 * j + 2 * t], f1 = xf[8 * j + 2 * t + 1];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          acc[r][j][0] = fmaf(d[r][j][0], f0, acc[r][j][0]);
          acc[r][j][1] = fmaf(d[r][j][1], f1, acc[r][j][1]);
          acc[r][j][2] = fmaf(d[r][j][2], f0, acc[r][j][2]);
          acc[r][j][3] = fmaf(d[r][j][3], f1, acc[r][j][3]);
        }
      }
    }
    const int64_t width = p.act ? p.n_out / 2 : p.n_out;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t n = int64_t(rb) * kRows + 16 * r + 8 * h + g;
        const float rs = n < p.n_out && p.row_scale ? p.row_scale[int64_t(e) * p.n_out + n] : 1.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int64_t row = r0 + 8 * j + 2 * t + q;
            float v = acc[r][j][2 * h + q] * rs;
            int64_t at = n;
            bool mine = n < p.n_out && row < hi;
            if (p.act) {
              const float up = __shfl_xor_sync(0xffffffffu, v, 4);  // output n + 1
              v = silu(v) * up;
              mine = mine && !(g & 1);
              at = n / 2;
            }
            if (!mine) continue;
            if (p.y_fp32) static_cast<float*>(p.y)[row * width + at] = v;
            else static_cast<__nv_bfloat16*>(p.y)[row * width + at] = __float2bfloat16_rn(v);
          }
      }
  }
}

}  // namespace grp

size_t fp4_grouped_ws_bytes(int64_t n_x, int64_t n_in) {
  if (n_x <= 0 || n_in <= 0 || n_in % CSA2_GROUP || n_x > (int64_t(1) << 31) || n_in > (1 << 28)) return 0;
  return size_t((n_x * (n_in * 2 + 4) + 255) / 256 * 256 + 1024);
}

}  // namespace csa2

extern "C" csa2_status csa2_fp4_grouped(const uint16_t* x, int64_t n_x, int64_t n_in, const uint8_t* packed, int E,
                                        int64_t n_out, const float* row_scale, const int32_t* offsets, const int32_t* src,
                                        int64_t rows, int act, void* y, int y_fp32, void* ws, size_t ws_bytes,
                                        csa2_stream_t stream) {
  using namespace csa2;
  using namespace csa2::grp;
  if (n_x < 0 || n_x >= (1ll << 31) || rows < 0 || rows >= (1ll << 31) || E < 0 || E > CSA2_MAX_EXPERTS || n_in <= 0 ||
      n_in % CSA2_GROUP || n_in > (1 << 24) || n_out < 0 || n_out > (1 << 24) ||
      (act != CSA2_ACT_NONE && act != CSA2_ACT_SWIGLU) || (act == CSA2_ACT_SWIGLU && n_out % 2))
    return CSA2_ERR_INVALID_ARG;
  if (!src && n_x < rows) return CSA2_ERR_INVALID_ARG;
  if (rows == 0 || n_out == 0 || E == 0) return CSA2_OK;
  if ((!x && n_x > 0) || !packed || !offsets || !y) return CSA2_ERR_INVALID_ARG;
  if (!al(x, 16) || !al(packed, 16) || !al(row_scale, 4) || !al(offsets, 4) || !al(src, 4) || !al(y, 16) || !al(ws, 16))
    return CSA2_ERR_INVALID_ARG;
  const size_t need = fp4_grouped_ws_bytes(n_x, n_in);
  if (need && (!ws || ws_bytes < need)) return CSA2_ERR_WORKSPACE;
  const int64_t width = act ? n_out / 2 : n_out, w_bytes = int64_t(csa2_fp4_packed_bytes(n_out, n_in));
  const Span spans[] = {span(y, rows, width * (y_fp32 ? 4 : 2)), span(need ? ws : nullptr, int64_t(need), 1),
                        span(x, n_x, n_in * 2), span(packed, E, w_bytes), span(row_scale, E, n_out * 4),
                        span(offsets, E + 1, 4), span(src, rows, 4)};
  if (any_overlap(spans, 2, 7)) return CSA2_ERR_INVALID_ARG;
  Params p = {};
  p.x = x, p.packed = packed, p.row_scale = row_scale, p.offsets = offsets, p.src = src, p.y = y;
  p.n_out = n_out, p.n_in = n_in, p.w_bytes = w_bytes, p.rows = rows, p.n_x = n_x, p.E = E, p.y_fp32 = y_fp32, p.act = act;
  p.n_kb = int((n_in + kChan - 1) / kChan), p.n_rb = int((n_out + kRows - 1) / kRows);
  p.flags = device_flags_ptr();
  if (!p.flags) return CSA2_ERR_CUDA;
  const cudaError_t e = launch_pdl(grouped_kernel, dim3(unsigned((p.n_rb + kWarps - 1) / kWarps), unsigned(E)), dim3(kThreads), 0,
                                   reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
