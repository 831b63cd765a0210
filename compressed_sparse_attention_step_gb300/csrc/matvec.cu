// Products of a few token rows with a 4-bit weight: y[m][n] = row_scale[n] sum_k x[m][k] e2m1[n][k] e4m3[n][k/16].
//
// Bound: the weight's 0.5625 bytes per element from HBM (one pass; x and y are small beside it), and for more
// than about 24 token rows the 1024 multiply-adds a cycle and SM of mma.m16n8k16.
//
// Layout.  The weight is packed once into blocks of 16 output rows x 128 input channels, 1152 bytes each,
// in the order in which a warp's lanes use them: lane (g, t) takes rows g and g + 8 and channels
// 32t .. 32t+31 of the block, 16 bytes of codes a row (two coalesced 512-byte loads a warp), and the four
// scale bytes of those (one 128-byte load).  The sum over a block's 128 channels may run in any order, so
// the lane's j-th channel pair stands where the A fragment of m16n8k16 wants the lane's j-th pair, and x is
// staged in the same order.  Rows and channels past the weight are zero codes.
//
// Numbers.  A code times a scale is exact in f16 (6 significant bits, 2^-10 .. 2688).  x is bf16: each
// (token, 128-channel block) is scaled by the power of two that brings its largest magnitude into [2^14, 2^15)
// and is then exact in f16 down to 2^-28 of that magnitude, off by less than 2^-38 of it below; the block's
// sum is scaled back in fp32.  All sums are fp32, in a fixed order.
//
// Work.  A warp owns 32 output rows and every WK-th block of its CTA's share of the channels; a CTA holds
// WR x WK = 8 warps, and a cluster of C CTAs splits the channels further.  Partial sums meet in shared memory
// and over the cluster's distributed shared memory, in a fixed order: no atomics, no workspace.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"

namespace csa2 {
namespace mv {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16, kChan = 128;     // block
constexpr int kBlock = kRows * kChan / 2 + kRows * kChan / CSA2_GROUP;  // 1152 bytes
constexpr int kStage = 64 * 1024;          // bytes of x staged at a time
constexpr int kMaxCluster = 8;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One thread per 16 bytes of packed codes or 4 scale bytes: block (row tile, channel block), lane.
__global__ void __launch_bounds__(256) pack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                   int64_t n_out, int64_t n_in, int64_t n_kb, int64_t n_blocks,
                                                   uint8_t* __restrict__ packed) {
  pdl_wait();
  pdl_trigger();
  const int64_t gid = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t blk = gid >> 5;
  if (blk >= n_blocks) return;
  const int lane = int(gid & 31), g = lane >> 2, t = lane & 3;
  const int64_t tile = blk / n_kb, kb = blk - tile * n_kb;
  const int64_t c0 = kb * kChan + 32 * t;  // this lane's 32 channels: two scale groups
  uint8_t* dst = packed + blk * kBlock;
  uint32_t sb = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = tile * kRows + 8 * h + g;
    uint2 w[2] = {make_uint2(0, 0), make_uint2(0, 0)};
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (row < n_out && c0 + 16 * j < n_in) {  // n_in is a multiple of 16: whole groups
        w[j] = *reinterpret_cast<const uint2*>(codes + row * (n_in / 2) + (c0 + 16 * j) / 2);
        sb |= uint32_t(scales[row * (n_in / CSA2_GROUP) + c0 / CSA2_GROUP + j]) << (16 * h + 8 * j);
      }
    *reinterpret_cast<uint4*>(dst + 512 * h + 16 * lane) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
  }
  *reinterpret_cast<uint32_t*>(dst + 1024 + 4 * lane) = sb;
}

__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t a, uint32_t rank) {
  float v;
  asm volatile("{ .reg .u32 r; mapa.shared::cluster.u32 r, %1, %2; ld.shared::cluster.f32 %0, [r]; }\n"
               : "=f"(v)
               : "r"(a), "r"(rank)
               : "memory");
  return v;
}

struct Unit {  // 32 rows x 128 channels, as loaded
  uint4 c[2][2];
  uint32_t s[2];
};

struct Params {
  const uint16_t* x;
  const uint8_t* packed;
  const float* row_scale;
  void* y;
  int64_t n_out, n_in;
  int m, n_kb, n_tiles;  // token rows, channel blocks, 16-row tiles
  int stage_kb;          // channel blocks staged at a time (a multiple of 8)
  int y_fp32;
};

// TG: groups of 8 token rows; WR: warps along the output rows.
template <int TG, int WR>
__global__ void __launch_bounds__(kThreads, TG <= 2 ? 2 : 1) matvec_kernel(const Params p, int C) {
  constexpr int WK = kWarps / WR;
  constexpr int kTok = TG * 8;
  constexpr int kCtaRows = WR * 32;
  extern __shared__ __align__(16) unsigned char smem[];
  uint4* xs = reinterpret_cast<uint4*>(smem);                                       // [kb][TG][4][32 lanes]
  float* xf = reinterpret_cast<float*>(smem + size_t(p.stage_kb) * kTok * kChan * 2);  // [kb][kTok]
  float* red = reinterpret_cast<float*>(smem);                                      // [WK][kTok][kCtaRows]
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3, g = lane >> 2;
  const int wr = warp / WK, wk = warp % WK;
  const int rank = C > 1 ? int(blockIdx.x % unsigned(C)) : 0;
  const int64_t row0 = int64_t(blockIdx.x / unsigned(C)) * kCtaRows;
  const int kb0 = int(int64_t(p.n_kb) * rank / C), kb1 = int(int64_t(p.n_kb) * (rank + 1) / C);
  const int tile0 = int(row0 / kRows) + wr * 2;
  const bool live0 = tile0 < p.n_tiles, live1 = tile0 + 1 < p.n_tiles;

  auto load = [&](Unit& u, int kb) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool on = (r ? live1 : live0) && kb < kb1;
      const uint8_t* src = p.packed + (int64_t(tile0 + r) * p.n_kb + kb) * kBlock;
      u.c[r][0] = on ? ld_stream16(src + 16 * lane) : make_uint4(0, 0, 0, 0);
      u.c[r][1] = on ? ld_stream16(src + 512 + 16 * lane) : make_uint4(0, 0, 0, 0);
      u.s[r] = on ? __ldcs(reinterpret_cast<const uint32_t*>(src + 1024 + 4 * lane)) : 0u;
    }
  };
  Unit u0, u1;
  load(u0, kb0 + wk);
  load(u1, kb0 + wk + WK);

  float acc[2][TG][4];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int j = 0; j < TG; ++j) acc[r][j][0] = acc[r][j][1] = acc[r][j][2] = acc[r][j][3] = 0.f;

  for (int c0 = kb0; c0 < kb1; c0 += p.stage_kb) {
    const int nk = min(p.stage_kb, kb1 - c0);
    if (c0 != kb0) __syncthreads();
    // stage x: half a warp per (block, token), 8 channels a lane
    for (int it = tid >> 4; it < nk * kTok; it += kThreads / 16) {
      const int kb = it / kTok, tok = it - kb * kTok, j = lane & 15;
      const int64_t ch = int64_t(c0 + kb) * kChan + 8 * j;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (tok < p.m && ch < p.n_in) v = __ldg(reinterpret_cast<const uint4*>(p.x + int64_t(tok) * p.n_in + ch));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) am = max(am, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      const unsigned half = 0xFFFFu << (lane & 16);
#pragma unroll
      for (int o = 8; o; o >>= 1) am = max(am, __shfl_xor_sync(half, am, o));
      const int up = am ? min(max(141 - int(am >> 7), -126), 126) : 0;
      const float f = __uint_as_float(uint32_t(127 + up) << 23);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = attn::h2_bits(__floats2half2_rn(bf16lo(w[i]) * f, bf16hi(w[i]) * f));
      xs[((kb * TG + (tok >> 3)) * 4 + (j & 3)) * 32 + (tok & 7) * 4 + (j >> 2)] = make_uint4(o[0], o[1], o[2], o[3]);
      if (j == 0) xf[kb * kTok + tok] = __uint_as_float(uint32_t(127 - up) << 23);
    }
    __syncthreads();
    for (int kb = wk; kb < nk; kb += WK) {
      float d[2][TG][4];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < TG; ++j) d[r][j][0] = d[r][j][1] = d[r][j][2] = d[r][j][3] = 0.f;
      __half2 sc[2][2][2];  // [tile][row half][16-channel group]
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __half2 s2 = attn::bits_h2(attn::e4m3x2_to_f16x2(uint16_t(u0.s[r] >> (16 * h))));
          sc[r][h][0] = __low2half2(s2), sc[r][h][1] = __high2half2(s2);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 xb[TG];
#pragma unroll
        for (int j = 0; j < TG; ++j) xb[j] = xs[((kb * TG + j) * 4 + i) * 32 + lane];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 cw = u0.c[r][h];
            const uint32_t w = i == 0 ? cw.x : i == 1 ? cw.y : i == 2 ? cw.z : cw.w;
            attn::e2m1x8_to_f16x2x4(w, a[h][0], a[h][1], a[h][2], a[h][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[h][e] = attn::h2_bits(__hmul2(attn::bits_h2(a[h][e]), sc[r][h][i >> 1]));
          }
#pragma unroll
          for (int j = 0; j < TG; ++j) {
            mma_f16(d[r][j], a[0][0], a[1][0], a[0][1], a[1][1], xb[j].x, xb[j].y);
            mma_f16(d[r][j], a[0][2], a[1][2], a[0][3], a[1][3], xb[j].z, xb[j].w);
          }
        }
      }
      u0 = u1;
      load(u1, c0 + kb + 2 * WK);
#pragma unroll
      for (int j = 0; j < TG; ++j) {
        const float2 f = *reinterpret_cast<const float2*>(&xf[kb * kTok + 8 * j + 2 * t]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          acc[r][j][0] = fmaf(d[r][j][0], f.x, acc[r][j][0]);
          acc[r][j][1] = fmaf(d[r][j][1], f.y, acc[r][j][1]);
          acc[r][j][2] = fmaf(d[r][j][2], f.x, acc[r][j][2]);
          acc[r][j][3] = fmaf(d[r][j][3], f.y, acc[r][j][3]);
        }
      }
    }
  }
  __syncthreads();
  // acc[r][j]: rows g (0, 1) and g + 8 (2, 3) of tile r, tokens 8j + 2t and + 1
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int j = 0; j < TG; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[(wk * kTok + 8 * j + 2 * t + (e & 1)) * kCtaRows + wr * 32 + r * 16 + g + 8 * (e >> 1)] = acc[r][j][e];
  if (C > 1) cluster_arrive_wait();
  else __syncthreads();
  const int rows = kCtaRows / C;
  const uint32_t red_a = smem_u32(red);
  for (int e = tid; e < rows * p.m; e += kThreads) {
    const int tok = e / rows, rr = rank * rows + e - tok * rows;
    const int64_t n = row0 + rr;
    if (n >= p.n_out) continue;
    float s = 0.f;
    for (int q = 0; q < C; ++q)
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const int at = (w * kTok + tok) * kCtaRows + rr;
        s += C > 1 ? ld_cluster(red_a + 4u * uint32_t(at), uint32_t(q)) : red[at];
      }
    if (p.row_scale) s *= p.row_scale[n];
    if (p.y_fp32) static_cast<float*>(p.y)[int64_t(tok) * p.n_out + n] = s;
    else static_cast<__nv_bfloat16*>(p.y)[int64_t(tok) * p.n_out + n] = __float2bfloat16_rn(s);
  }
  if (C > 1) cluster_arrive_wait();  // no CTA leaves while its sums are being read
}

template <int TG, int WR>
cudaError_t launch(Params p, int C, cudaStream_t st) {
  constexpr int kTok = TG * 8, WK = kWarps / WR, kCtaRows = WR * 32;
  const int share = (p.n_kb + C - 1) / C;
  p.stage_kb = std::min(kStage / (kTok * kChan * 2), (share + 7) / 8 * 8);
  const size_t smem = std::max(size_t(p.stage_kb) * kTok * (kChan * 2 + 4), size_t(WK) * kTok * kCtaRows * 4);
  auto kern = matvec_kernel<TG, WR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((p.n_tiles + 2 * WR - 1) / (2 * WR) * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, C);
}

template <int TG>
cudaError_t launch_wr(const Params& p, int sms, cudaStream_t st) {
  // the widest CTA and the smallest cluster that still give two CTAs per SM, else the most CTAs there are
  for (int wr = 8; wr >= 1; wr /= 2)
    for (int C = 1; C <= kMaxCluster; C *= 2) {
      const int64_t ctas = int64_t((p.n_tiles + 2 * wr - 1) / (2 * wr)) * C;
      const bool last = wr == 1 && C == kMaxCluster;
      if (ctas < 2 * int64_t(sms) && !last) continue;
      if (wr == 8) return launch<TG, 8>(p, C, st);
      if (wr == 4) return launch<TG, 4>(p, C, st);
      if (wr == 2) return launch<TG, 2>(p, C, st);
      return launch<TG, 1>(p, C, st);
    }
  return cudaErrorInvalidValue;
}

inline bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool sizes_ok(int64_t n_out, int64_t n_in) {
  return n_out >= 0 && n_in >= 0 && n_in % CSA2_GROUP == 0 && n_out <= (int64_t(1) << 30) && n_in <= (int64_t(1) << 30);
}

}  // namespace mv
}  // namespace csa2

extern "C" size_t csa2_fp4_packed_bytes(int64_t n_out, int64_t n_in) {
  using namespace csa2::mv;
  if (!sizes_ok(n_out, n_in)) return 0;
  return size_t((n_out + kRows - 1) / kRows) * size_t((n_in + kChan - 1) / kChan) * kBlock;
}

extern "C" csa2_status csa2_fp4_pack_weight(const uint8_t* codes, const uint8_t* scales, int64_t n_out, int64_t n_in,
                                            uint8_t* packed, csa2_stream_t stream) {
  using namespace csa2;
  using namespace csa2::mv;
  if (!sizes_ok(n_out, n_in)) return CSA2_ERR_INVALID_ARG;
  if (n_out * n_in == 0) return CSA2_OK;
  if (!codes || !scales || !packed || !al(codes, 16) || !al(scales, 16) || !al(packed, 16)) return CSA2_ERR_INVALID_ARG;
  const int64_t n_kb = (n_in + kChan - 1) / kChan, n_blocks = (n_out + kRows - 1) / kRows * n_kb;
  if (n_blocks * 32 / 256 > 0x7FFFFFF0ll) return CSA2_ERR_INVALID_ARG;
  return launch_pdl(pack_kernel, dim3(unsigned((n_blocks * 32 + 255) / 256)), dim3(256), 0,
                    reinterpret_cast<cudaStream_t>(stream), codes, scales, n_out, n_in, n_kb, n_blocks,
                    packed) == cudaSuccess
             ? CSA2_OK
             : CSA2_ERR_CUDA;
}

extern "C" csa2_status csa2_fp4_matvec(const uint16_t* x, int m, const uint8_t* packed, int64_t n_out, int64_t n_in,
                                       const float* row_scale, void* y, int y_fp32, csa2_stream_t stream) {
  using namespace csa2;
  using namespace csa2::mv;
  if (!sizes_ok(n_out, n_in) || m < 0 || m > CSA2_MAX_MV_ROWS || n_in == 0) return CSA2_ERR_INVALID_ARG;
  if (m == 0 || n_out == 0) return CSA2_OK;
  if (!x || !packed || !y || !al(x, 16) || !al(packed, 16) || !al(y, 16) || !al(row_scale, 4))
    return CSA2_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return CSA2_ERR_CUDA;
  Params p = {};
  p.x = x, p.packed = packed, p.row_scale = row_scale, p.y = y;
  p.n_out = n_out, p.n_in = n_in, p.m = m, p.y_fp32 = y_fp32;
  p.n_kb = int((n_in + kChan - 1) / kChan), p.n_tiles = int((n_out + kRows - 1) / kRows);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch ((m + 7) / 8) {
    case 1: e = launch_wr<1>(p, sms, st); break;
    case 2: e = launch_wr<2>(p, sms, st); break;
    case 3: e = launch_wr<3>(p, sms, st); break;
    default: e = launch_wr<4>(p, sms, st); break;
  }
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
