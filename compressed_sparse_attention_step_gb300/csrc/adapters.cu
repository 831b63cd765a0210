// Low-rank adapters of many requests: out[i] = base[i] + scale[l] B_l (A_l x_i), l the adapter of row i.
//
// A cluster of CTAs takes a tile of consecutive rows and one of the adapters that its rows use (a slot; the CTAs of a
// slot without one leave).  Its CTAs share the input channels of A_l x, add their parts up through distributed shared
// memory in order of rank, and share the output channels of B_l t: one launch, no workspace, no atomics.  Rows of other
// adapters are multiplied along in the tile (rows of an MMA do not mix) and not written.  The sums are in one order
// whatever else is in the batch, but not whatever the tile's height: that goes by m.
//
// mma.m16n8k16 on bf16 as it lies in memory.  Channels are handed to the MMA in an order that lets a lane load 16
// neighbouring bytes: the same for both operands, so that the sum over the channels does not change.  t = A x is fp32
// and enters the second product as two bf16 terms (off by 2^-17 of it at most); all sums are fp32, and out is rounded
// once.
//
// Bound: for few rows the adapters' bytes, each once, and the chain load, sum, exchange, load, store; for many rows x
// and base read and out written.
#include <cuda_bf16.h>

#include <algorithm>

#include "cluster.cuh"

namespace csa2 {
namespace lora {

constexpr int kThreads = 256, kWarps = 8, kMaxCluster = 8;

struct Params {
  const uint16_t *x, *a, *b;
  const int32_t *adapter, *ranks;
  const float* scale;
  const void* base;
  void* out;
  int m, n_in, n_out, r, L, slots;
  unsigned int* flags;
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  const uint32_t a[4] = {a0, a1, a2, a3};
  mma_bf16_16816(d, a, b0, b1);
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// NR: groups of eight ranks, an even number; WM: warps along the rows, of MT tiles of 16 each.
// kF32: base and out are fp32; kVec: rows of out are whole 16-byte pieces.
template <int NR, int WM, int MT, bool kF32, bool kVec>
__global__ void __launch_bounds__(kThreads) lora_kernel(const Params p, int C) {
  constexpr int WK = kWarps / WM, TM = 16 * WM * MT, R = 8 * NR, kPitch = R + 8;
  extern __shared__ __align__(16) unsigned char smem[];
  float* part = reinterpret_cast<float*>(smem);                     // [WK][TM][R]; then, from 0, this CTA's sums [TM][R]
  uint16_t* hi = reinterpret_cast<uint16_t*>(part + WK * TM * R);   // [TM][kPitch], channels in the MMA's order
  uint16_t* lo = hi + TM * kPitch;
  __shared__ int which[TM], list[TM];
  __shared__ int n_list;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3, g = lane >> 2;
  const int rank = C > 1 ? int(blockIdx.x % unsigned(C)) : 0;
  const int unit = int(blockIdx.x / unsigned(C)), slot = unit % p.slots, row0 = unit / p.slots * TM;
  const int wm = warp % WM, wk = warp / WM;

  // the adapters of the tile's rows, in the order of their first rows
  if (tid < TM) {
    int l = row0 + tid < p.m ? p.adapter[row0 + tid] : -1;
    if (l >= p.L) {
      l = -1;
      if (rank == 0 && slot == 0) atomicOr(p.flags, CSA2_FLAG_INDEX_OOB);
    }
    which[tid] = l < 0 ? -1 : l;
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int i0 = 0; i0 < TM; i0 += 32) {
      const int i = i0 + lane;
      bool first = i < TM && which[i] >= 0;
      for (int j = 0; first && j < i; ++j) first = which[j] != which[i];
      const unsigned got = __ballot_sync(0xffffffffu, first);
      if (first) list[n + __popc(got & ((1u << lane) - 1u))] = which[i];
      n += __popc(got);
    }
    if (lane == 0) n_list = n;
  }
  __syncthreads();
  const int n_adapters = n_list;

  const int n_blk = (p.n_out + 31) / 32;           // blocks of 32 output channels, taken in turn by the cluster's warps
  const int blk0 = rank * kWarps + warp, blk_step = C * kWarps;

  if (slot == 0 && p.base != p.out) {  // rows without an adapter
    for (int i = 0; i < TM && row0 + i < p.m; ++i) {
      if (which[i] >= 0) continue;
      const int64_t at = int64_t(row0 + i) * p.n_out;
      for (int n = (rank * kThreads + tid); n < p.n_out; n += C * kThreads) {
        if (kF32) static_cast<float*>(p.out)[at + n] = static_cast<const float*>(p.base)[at + n];
        else static_cast<uint16_t*>(p.out)[at + n] = static_cast<const uint16_t*>(p.base)[at + n];
      }
    }
  }

  const int n_chunk = (p.n_in + 31) / 32;
  const int c0 = int(int64_t(n_chunk) * rank / C), c1 = int(int64_t(n_chunk) * (rank + 1) / C);
  for (int s = slot; s < n_adapters; s += p.slots) {
    const int l = list[s];
    const int n_rank = p.ranks ? min(max(p.ranks[l], 0), p.r) : p.r;
    // t = A x over this CTA's channels
    {
      float acc[MT][NR][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;
      const uint16_t* a = p.a + int64_t(l) * p.r * p.n_in;
#pragma unroll 2
      for (int c = c0 + wk; c < c1; c += WK) {
        const int ch = c * 32 + 8 * t;
        uint4 xv[MT][2], av[NR];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = row0 + (wm * MT + i) * 16 + 8 * h + g;
            xv[i][h] = row < p.m && ch < p.n_in ? __ldg(reinterpret_cast<const uint4*>(p.x + int64_t(row) * p.n_in + ch))
                                                : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          const int rr = 8 * j + g;
          av[j] = rr < n_rank && ch < p.n_in ? __ldg(reinterpret_cast<const uint4*>(a + int64_t(rr) * p.n_in + ch))
                                             : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            mma(acc[i][j], xv[i][0].x, xv[i][1].x, xv[i][0].y, xv[i][1].y, av[j].x, av[j].y);
            mma(acc[i][j], xv[i][0].z, xv[i][1].z, xv[i][0].w, xv[i][1].w, av[j].z, av[j].w);
          }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = (wm * MT + i) * 16 + 8 * h + g;
            *reinterpret_cast<float2*>(part + (wk * TM + row) * R + 8 * j + 2 * t) =
                make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
          }
    }
    __syncthreads();
    for (int e = tid; e < TM * R / 4; e += kThreads) {
      float4 v = reinterpret_cast<float4*>(part)[e];
#pragma unroll
      for (int w = 1; w < WK; ++w) {
        const float4 u = reinterpret_cast<float4*>(part)[w * (TM * R / 4) + e];
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      reinterpret_cast<float4*>(part)[e] = v;
    }
    if (C > 1) cluster_arrive(), cluster_wait();
    else __syncthreads();
    // the cluster's sums, scaled, as two bf16 terms
    const float scale = p.scale ? p.scale[l] : 1.f;
    for (int e = tid; e < TM * R / 4; e += kThreads) {
      float4 v;
      if (C > 1) {
        float4 u[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (c < C) u[c] = ld_cluster4(cluster_addr(smem_u32(part + 4 * e), uint32_t(c)));
        v = u[0];
#pragma unroll
        for (int c = 1; c < kMaxCluster; ++c)
          if (c < C) v.x += u[c].x, v.y += u[c].y, v.z += u[c].z, v.w += u[c].w;
      } else {
        v = reinterpret_cast<const float4*>(part)[e];
      }
      v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
      const int row = e / (R / 4), rr = e % (R / 4) * 4;
      if (rr + 4 > n_rank) {  // 0 past the adapter's rank, whatever x holds
        if (rr >= n_rank) v.x = 0.f;
        if (rr + 1 >= n_rank) v.y = 0.f;
        if (rr + 2 >= n_rank) v.z = 0.f;
        v.w = 0.f;
      }
      const uint32_t h0 = bf2(v.x, v.y), h1 = bf2(v.z, v.w);
      const uint32_t l0 = bf2(v.x - bf16lo(h0), v.y - bf16hi(h0)), l1 = bf2(v.z - bf16lo(h1), v.w - bf16hi(h1));
      // four neighbouring ranks are a lane's of one step: places 2q, 2q + 1, 2q + 8, 2q + 9.  With 32 ranks and more a
      // lane has eight neighbouring ones, the first four of one step, the others of the next
      int step, q;
      if (R >= 32) step = rr / 32 * 2 + (rr % 8) / 4, q = rr % 32 / 8;
      else step = 0, q = rr / 4;
      uint16_t* at_h = hi + row * kPitch + step * 16 + 2 * q;
      uint16_t* at_l = lo + row * kPitch + step * 16 + 2 * q;
      *reinterpret_cast<uint32_t*>(at_h) = h0, *reinterpret_cast<uint32_t*>(at_h + 8) = h1;
      *reinterpret_cast<uint32_t*>(at_l) = l0, *reinterpret_cast<uint32_t*>(at_l + 8) = l1;
    }
    __syncthreads();
    if (C > 1) cluster_arrive();
    // out = base + B t over this warp's output channels: a lane gets eight neighbouring ones, 8t .. 8t + 7
    const uint16_t* b = p.b + int64_t(l) * p.n_out * p.r;
    for (int blk = blk0; blk < n_blk; blk += blk_step) {
      uint32_t bv[4][R / 16][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = blk * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
        const uint16_t* row = b + int64_t(n) * p.r;
        if (R >= 32) {
#pragma unroll
          for (int k = 0; k < R / 32; ++k) {
            const int rr = 32 * k + 8 * t;
            const uint4 v = n < p.n_out && rr < n_rank ? __ldg(reinterpret_cast<const uint4*>(row + rr)) : make_uint4(0, 0, 0, 0);
            bv[j][2 * k][0] = v.x, bv[j][2 * k][1] = v.y;
            bv[j][R >= 32 ? 2 * k + 1 : 0][0] = v.z, bv[j][R >= 32 ? 2 * k + 1 : 0][1] = v.w;
          }
        } else {
          const int rr = 4 * t;
          const uint2 v = n < p.n_out && rr < n_rank ? __ldg(reinterpret_cast<const uint2*>(row + rr)) : make_uint2(0, 0);
          bv[j][0][0] = v.x, bv[j][0][1] = v.y;
        }
      }
      if (n_rank < R) {  // what lies past the adapter's rank is not used
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < R / 16; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int rr = R >= 32 ? 32 * (k >> 1) + 8 * t + 4 * (k & 1) + 2 * h : 4 * t + 2 * h;
              if (rr >= n_rank) bv[j][k][h] = 0;
              else if (rr + 1 >= n_rank) bv[j][k][h] &= 0xFFFFu;
            }
      }
      const int n0 = blk * 32 + 8 * t;
#pragma unroll
      for (int i = 0; i < TM / 16; ++i) {
        const bool use0 = which[16 * i + g] == l, use1 = which[16 * i + 8 + g] == l;
        if (!__any_sync(0xffffffffu, use0 || use1)) continue;
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll
        for (int k = 0; k < R / 16; ++k)
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const uint16_t* src = (term ? lo : hi) + (16 * i + (lane & 15)) * kPitch + 16 * k + 8 * (lane >> 4);
            uint32_t f[4];
            ldmatrix_x4(f[0], f[1], f[2], f[3], smem_u32(src));
#pragma unroll
            for (int j = 0; j < 4; ++j) mma(d[j], f[0], f[1], f[2], f[3], bv[j][k][0], bv[j][k][1]);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(h ? use1 : use0)) continue;
          const int64_t at = int64_t(row0 + 16 * i + 8 * h + g) * p.n_out + n0;
          if (kVec) {
            if (n0 >= p.n_out) continue;
            if (kF32) {
              const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.base) + at);
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float4 v = src[q];
                v.x += d[2 * q][2 * h], v.y += d[2 * q][2 * h + 1], v.z += d[2 * q + 1][2 * h], v.w += d[2 * q + 1][2 * h + 1];
                dst[q] = v;
              }
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.base) + at);
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = bf2(bf16lo(w[j]) + d[j][2 * h], bf16hi(w[j]) + d[j][2 * h + 1]);
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (n0 + 2 * j + e >= p.n_out) continue;
                const int64_t o = at + 2 * j + e;
                const float v = d[j][2 * h + e];
                if (kF32) static_cast<float*>(p.out)[o] = static_cast<const float*>(p.base)[o] + v;
                else static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(bf16f(static_cast<const uint16_t*>(p.base)[o]) + v);
              }
          }
        }
      }
    }
    if (C > 1) cluster_wait();  // the others have read this CTA's sums
    __syncthreads();
  }
}

template <int NR, int WM, int MT, bool kF32, bool kVec>
cudaError_t launch(Params p, int C, cudaStream_t st) {
  constexpr int TM = 16 * WM * MT, R = 8 * NR;
  constexpr size_t smem = size_t(kWarps / WM) * TM * R * 4 + size_t(2) * TM * (R + 8) * 2;
  auto kern = lora_kernel<NR, WM, MT, kF32, kVec>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t(p.m) + TM - 1) / TM;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles * p.slots * C));
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

template <int NR, int WM, int MT>
cudaError_t launch_out(const Params& p, int C, bool f32, cudaStream_t st) {
  if (p.n_out % 8 == 0) return f32 ? launch<NR, WM, MT, true, true>(p, C, st) : launch<NR, WM, MT, false, true>(p, C, st);
  return f32 ? launch<NR, WM, MT, true, false>(p, C, st) : launch<NR, WM, MT, false, false>(p, C, st);
}

template <int WM, int MT>
cudaError_t launch_rank(const Params& p, int C, bool f32, cudaStream_t st) {
  if (p.r <= 16) return launch_out<2, WM, MT>(p, C, f32, st);
  if (p.r <= 32) return launch_out<4, WM, MT>(p, C, f32, st);
  if (p.r <= 64) return launch_out<8, WM, MT>(p, C, f32, st);
  return launch_out<16, WM, MT>(p, C, f32, st);
}

}  // namespace lora
}  // namespace csa2

extern "C" csa2_status csa2_lora_add(const uint16_t* x, int m, int n_in, const uint16_t* a, const uint16_t* b, int L, int r,
                                     int n_out, const int32_t* adapter, const int32_t* ranks, const float* scale,
                                     const void* base, void* out, int out_fp32, csa2_stream_t stream) {
  using namespace csa2;
  using namespace csa2::lora;
  if (m < 0 || m > (1 << 24) || n_in < 0 || n_in > (1 << 24) || n_in % 8 || n_out < 0 || n_out > (1 << 24) || L < 0 ||
      r < 8 || r > CSA2_MAX_RANK || r % 8)
    return CSA2_ERR_INVALID_ARG;
  if (m == 0 || n_out == 0) return CSA2_OK;
  if (!adapter || !base || !out || (L > 0 && n_in > 0 && (!x || !a || !b))) return CSA2_ERR_INVALID_ARG;
  if (!al(x, 16) || !al(a, 16) || !al(b, 16) || !al(base, 16) || !al(out, 16) || !al(adapter, 4) || !al(ranks, 4) || !al(scale, 4))
    return CSA2_ERR_INVALID_ARG;
  const int64_t row = int64_t(n_out) * (out_fp32 ? 4 : 2);
  const Span spans[] = {span(out, m, row), span(x, m, 2ll * n_in), span(a, int64_t(L) * r, 2ll * n_in),
                        span(b, int64_t(L) * r, 2ll * n_out), span(adapter, m, 4), span(ranks, L, 4), span(scale, L, 4),
                        span(base == out ? nullptr : base, m, row)};
  if (any_overlap(spans, 1, 8)) return CSA2_ERR_INVALID_ARG;
  const int sms = sm_count();
  Params p = {};
  p.x = x, p.a = a, p.b = b, p.adapter = adapter, p.ranks = ranks, p.scale = scale, p.base = base, p.out = out;
  p.m = m, p.n_in = n_in, p.n_out = n_out, p.r = r, p.L = L;
  p.flags = device_flags_ptr();
  if (!p.flags || sms <= 0) return CSA2_ERR_CUDA;
  const bool tall = m >= 512;
  const int TM = tall ? 64 : 16, C = 8;
  const int64_t tiles = (int64_t(m) + TM - 1) / TM;
  p.slots = int(std::min<int64_t>(std::max<int64_t>(4 * sms / (tiles * C), 1), std::min(TM, std::max(L, 1))));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = tall ? launch_rank<2, 2>(p, C, out_fp32, st) : launch_rank<1, 1>(p, C, out_fp32, st);
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
