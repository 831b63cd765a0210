// Attention of a tree of drafted tokens over the FP4 main-KV cache: every drafted node attends the rows
// its indexer selected, the committed part of its sliding window and its drafted ancestors (itself
// included), o = sum_r softmax_r(q . row_r * scale) row_r with K = V = the (dequantised) row.
//
// A node has 16 heads and its own selected rows, so its two products are [16 x 512] x [512 x rows] and
// [16 x rows] x [rows x 512]: the head count is exactly the M of mma.m16n8k16.  The tcgen05 forms feed
// the gathered rows from shared memory as the M = 128 operand against N = 16 heads and are held to the
// 1024 multiply-adds a cycle at which an SM reads that operand, after the dequantised rows have also been
// written to shared memory once; m16n8k16 reaches the same 1024 (measured: 2.0 cycles an instruction
// and SM) from registers, so here the rows never touch shared memory at all:
//  - four warps split the 512 channels, lane (g, t) of a warp loads 16 bytes of codes of row g: 32
//    consecutive channels of its warp's 128.  Channels may be summed in any order, so the lane's j-th
//    channel pair serves as the j-th pair of the B fragment of S = Q K^T as it is, with Q's fragment
//    loaded in the same order;
//  - the same registers, transposed 8 x 8 by movmatrix, are the B fragments of O = P V, and the
//    accumulator of S has the layout of P's A fragment; a lane's 16 output pairs are again 32
//    consecutive channels, stored as whole 16-byte pieces;
//  - the only traffic through shared memory is the sum of the four warps' partial scores.
// Bound: the tensor pipe (8192 cycles a node with 512 selected rows), then the transposes and the
// conversions.
//
// FP4 rows are multiplied as f16: a code times a scale has at most 6 significant bits and lies between
// 2^-10 and 2688, so the row is exact.  Q is scaled per head by a power of two that puts its largest
// magnitude into [2^14, 2^15), so its bf16 values are exact in f16 down to 2^-28 of that magnitude, and
// below it they are off by less than 2^-38 of it.  P is rounded to f16 (2^-11 relative).  Window rows are
// bf16 and are multiplied as bf16 with P rounded to bf16 (2^-8).  Scores, softmax statistics and outputs
// are accumulated in fp32; the softmax sum takes P before its rounding.
#include <cuda_bf16.h>

#include "attn_common.cuh"

namespace csa2 {
namespace tree {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kTile = 16;                                          // rows per step
constexpr int kMaxSel = CSA2_MAX_ATTN_K;                           // selected rows per node
constexpr int kMaxWin = CSA2_MAX_W - 1 + CSA2_MAX_TREE;            // window rows and ancestors
constexpr int kSelTiles = kMaxSel / kTile;
constexpr int kWinTiles = (kMaxWin + kTile - 1) / kTile;
constexpr int kMaxCluster = 8;
constexpr float kNegInf = -INFINITY;
// The softmax reference m starts kHead below the largest score of a CTA's first step and moves only when a
// score passes it by kHead + 8, so P lies below 2^15 and the largest is at least 2^kHead: in f16's range, whose
// subnormal rounding (2^-25) is then 2^-32 of the largest P.
constexpr float kHead = 7.0f;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool kF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (kF16) mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
  else mma_bf16(d, a0, a1, a2, a3, b0, b1);
}
// 8 x 8 transpose of 16-bit elements held as matrix fragments (row lane / 4, columns 2 (lane % 4), + 1)
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) { return attn::h2_bits(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

struct Params {
  const uint16_t* q;
  const int32_t* parent;
  const int32_t* n_nodes;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t cap, seq_rows;  // rows an index may name; rows from one sequence's cache to the next
  const int32_t* idx;
  const int32_t* n_valid;
  const uint16_t* swa;
  const int32_t* win_len;
  uint16_t* out;
  float* lse;
  float scale_log2;  // softmax scale times log2 e
  int N, k, W;
  unsigned int* flags;
};

struct Shared {
  float4 part[2][kWarps][2][32];     // partial scores of a step: [buffer][warp][half][lane]
  int32_t sel[kMaxSel];              // selected rows (-1: empty)
  int32_t win[kWinTiles * kTile];    // window buffer rows (-1: empty)
  uint32_t sel_mask[kSelTiles];      // valid rows of a step
  int32_t parent[CSA2_MAX_TREE];
  float qmax[kWarps][16];
  float2 ml[16];                     // (reference maximum, sum) of this CTA's part, for the merge
};
struct SharedMerge : Shared {
  float o[16][CSA2_D];
};

// State of a lane: O of heads g and g + 8 over its 32 channels, and the softmax statistics of both.
struct State {
  float o[16][4];
  float m0, m1, l0, l1;
};

// One step of 16 rows held as fragments kf (rows g and g + 8; 16 channel pairs each).
template <bool kF16>
__device__ __forceinline__ void step(State& s, const uint32_t (&qf)[2][16], const uint32_t (&kf)[2][16], uint32_t vmask,
                                     float sc0, float sc1, float4 (*part)[2][32], int warp, int lane) {
  const int t = lane & 3;
  float S0[4] = {0.f, 0.f, 0.f, 0.f}, S1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mma<kF16>(S0, qf[0][2 * i], qf[1][2 * i], qf[0][2 * i + 1], qf[1][2 * i + 1], kf[0][2 * i], kf[0][2 * i + 1]);
    mma<kF16>(S1, qf[0][2 * i], qf[1][2 * i], qf[0][2 * i + 1], qf[1][2 * i + 1], kf[1][2 * i], kf[1][2 * i + 1]);
  }
  part[warp][0][lane] = make_float4(S0[0], S0[1], S0[2], S0[3]);
  part[warp][1][lane] = make_float4(S1[0], S1[1], S1[2], S1[3]);
  __syncthreads();
  // every warp sums the four parts in the same order, so all of them take the same decisions below
  float x[8];
  {
    float4 a = part[0][0][lane], b = part[1][0][lane], c = part[2][0][lane], d = part[3][0][lane];
    x[0] = (a.x + b.x) + (c.x + d.x), x[1] = (a.y + b.y) + (c.y + d.y);
    x[2] = (a.z + b.z) + (c.z + d.z), x[3] = (a.w + b.w) + (c.w + d.w);
    a = part[0][1][lane], b = part[1][1][lane], c = part[2][1][lane], d = part[3][1][lane];
    x[4] = (a.x + b.x) + (c.x + d.x), x[5] = (a.y + b.y) + (c.y + d.y);
    x[6] = (a.z + b.z) + (c.z + d.z), x[7] = (a.w + b.w) + (c.w + d.w);
  }
  // x[0..1]: head g, rows 2t, 2t+1; x[2..3]: head g+8; x[4..7]: the same of rows 8+2t, 9+2t
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= (i & 2) ? sc1 : sc0;
  if (vmask != 0xFFFFu) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!((vmask >> (8 * (i >> 2) + 2 * t + (i & 1))) & 1u)) x[i] = kNegInf;
  }
  const float t0 = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[4], x[5]));
  const float t1 = fmaxf(fmaxf(x[2], x[3]), fmaxf(x[6], x[7]));
  if (__any_sync(0xffffffffu, t0 > s.m0 + (kHead + 8.f) || t1 > s.m1 + (kHead + 8.f))) {
    const float n0 = fmaxf(s.m0, quad_max(t0) - kHead), n1 = fmaxf(s.m1, quad_max(t1) - kHead);
    const float c0 = s.m0 == kNegInf ? 0.f : attn::ex2(s.m0 - n0), c1 = s.m1 == kNegInf ? 0.f : attn::ex2(s.m1 - n1);
    s.m0 = n0, s.m1 = n1;
    s.l0 *= c0, s.l1 *= c1;
#pragma unroll
    for (int i = 0; i < 16; ++i) s.o[i][0] *= c0, s.o[i][1] *= c0, s.o[i][2] *= c1, s.o[i][3] *= c1;
  }
  const float r0 = s.m0 == kNegInf ? 0.f : s.m0, r1 = s.m1 == kNegInf ? 0.f : s.m1;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = attn::ex2(x[i] - ((i & 2) ? r1 : r0));
  s.l0 += (x[0] + x[1]) + (x[4] + x[5]);
  s.l1 += (x[2] + x[3]) + (x[6] + x[7]);
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = kF16 ? pack_f16(x[2 * i], x[2 * i + 1]) : pack_bf16(x[2 * i], x[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    mma<kF16>(s.o[i], p[0], p[1], p[2], p[3], transpose8(kf[0][i]), transpose8(kf[1][i]));
}

// The raw bytes of rows g and g + 8 of a step, as a lane loads them ahead.
struct Raw {
  uint4 c[2];
  uint32_t s[2];
};
__device__ __forceinline__ void load_raw(Raw& r, const Params& p, const int32_t* sel, int64_t seq, int tile, int g,
                                         int part) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int32_t row = sel[tile * kTile + 8 * h + g];
    r.c[h] = make_uint4(0, 0, 0, 0);
    r.s[h] = 0;
    if (row >= 0) {
      const int64_t at = seq + row;
      r.c[h] = __ldg(reinterpret_cast<const uint4*>(p.codes + at * CSA2_CODE_BYTES) + part);
      r.s[h] = __ldg(reinterpret_cast<const uint16_t*>(p.scales + at * CSA2_SCALE_BYTES) + part);
    }
  }
}
__device__ __forceinline__ void dequant(const Raw& r, uint32_t (&kf)[2][16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t s2 = attn::e4m3x2_to_f16x2(uint16_t(r.s[h]));
    const __half2 lo = __low2half2(attn::bits_h2(s2)), hi = __high2half2(attn::bits_h2(s2));
    const uint32_t w[4] = {r.c[h].x, r.c[h].y, r.c[h].z, r.c[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t f[4];
      attn::e2m1x8_to_f16x2x4(w[i], f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) kf[h][4 * i + j] = attn::h2_bits(__hmul2(attn::bits_h2(f[j]), i < 2 ? lo : hi));
    }
  }
}

__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// One node per cluster of C CTAs (C = 1: per CTA), which share its steps of 16 rows and merge their
// parts through distributed shared memory, in rank order.
template <bool kMerge>
__global__ void __launch_bounds__(kThreads, 3) tree_attn_kernel(const Params p, int C) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  pdl_wait();
  pdl_trigger();
  const int rank = kMerge ? int(blockIdx.x % unsigned(C)) : 0;
  const int64_t row = kMerge ? int64_t(blockIdx.x / unsigned(C)) : int64_t(blockIdx.x);
  const int b = int(row / p.N), node = int(row - int64_t(b) * p.N);
  if (p.n_nodes && node >= p.n_nodes[b]) return;  // the whole cluster: its outputs stay as they were
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int chan = warp * 128 + t * 32;  // this lane's 32 channels

  // Q of heads g and g + 8, as bf16 pairs
  const uint16_t* qrow = p.q + row * (CSA2_H * CSA2_D) + chan;
  uint32_t qf[2][16];
  auto load_q = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(qrow + (g + 8 * h) * CSA2_D) + i);
        qf[h][4 * i] = v.x, qf[h][4 * i + 1] = v.y, qf[h][4 * i + 2] = v.z, qf[h][4 * i + 3] = v.w;
      }
  };
  load_q();

  // the row lists
  const int nv = p.n_valid ? min(max(p.n_valid[row], 0), p.k) : p.k;
  const int nsel = (nv + kTile - 1) / kTile;
  for (int i = tid; i < (nsel + 1) / 2 * 32; i += kThreads) {  // whole warps: two steps each
    const int32_t r = i < nv ? p.idx[row * p.k + i] : -1;
    const bool ok = r >= 0 && int64_t(r) < p.cap;
    if (r >= 0 && !ok) atomicOr(p.flags, CSA2_FLAG_INDEX_OOB);
    sm.sel[i] = ok ? r : -1;
    const uint32_t bal = __ballot_sync(0xffffffffu, ok);
    if ((i & 15) == 0) sm.sel_mask[i >> 4] = (bal >> (lane & 16)) & 0xFFFFu;
  }
  if (tid < p.N) sm.parent[tid] = p.parent[int64_t(b) * p.N + tid];
  // per head: the largest magnitude of Q (as bf16 bits)
  uint32_t am[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 16; ++i) am[h] = max(am[h], max(qf[h][i] & 0x7FFFu, (qf[h][i] >> 16) & 0x7FFFu));
    am[h] = max(am[h], __shfl_xor_sync(0xffffffffu, am[h], 1));
    am[h] = max(am[h], __shfl_xor_sync(0xffffffffu, am[h], 2));
    if (t == 0) sm.qmax[warp][g + 8 * h] = __uint_as_float(am[h] << 16);
  }
  __syncthreads();

  // ancestors of the node, itself included
  uint64_t anc = 0;
  int depth = -1;
  for (int cur = node; cur >= 0;) {
    anc |= 1ull << cur;
    ++depth;
    const int up = sm.parent[cur];
    if (up < -1 || up >= cur) {  // not a tree in node order: taken as a root
      if (tid == 0 && rank == 0) atomicOr(p.flags, CSA2_FLAG_INDEX_OOB);
      break;
    }
    cur = up;
  }
  // window rows: the committed rows [first, W - 1), then the ancestors less than W tokens away
  int n_com = 0, nw = 0, first = 0;
  if (p.W > 0) {
    const int wl = min(max(p.win_len ? p.win_len[b] : p.W - 1, 0), p.W - 1);
    first = max(depth, p.W - 1 - wl);
    n_com = max(p.W - 1 - first, 0);
    // the node's ancestors in order of depth: the bits of anc ascend with it
    const int drop = max(depth + 1 - p.W, 0);
    for (int i = 0; i < drop; ++i) anc &= anc - 1;
    nw = n_com + __popcll(anc);
    const int nwt = (nw + kTile - 1) / kTile * kTile;
    for (int i = tid; i < nwt; i += kThreads) {
      int32_t r = -1;
      if (i < n_com) r = first + i;
      else if (i < nw) {
        uint64_t m = anc;
        for (int j = n_com; j < i; ++j) m &= m - 1;
        r = p.W - 1 + (__ffsll(static_cast<long long>(m)) - 1);
      }
      sm.win[i] = r;
    }
  }
  const int nwin = (nw + kTile - 1) / kTile;
  const int steps = nsel + nwin;
  const int i0 = kMerge ? steps * rank / C : 0, i1 = kMerge ? steps * (rank + 1) / C : steps;
  const int s0 = i0, s1 = min(i1, nsel);                      // selected steps of this CTA
  const int w0 = max(i0 - nsel, 0), w1 = max(i1 - nsel, 0);   // window steps

  State st;
  st.m0 = st.m1 = kNegInf;
  st.l0 = st.l1 = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
  int buf = 0;

  if (s0 < s1) {
    const int64_t seq = int64_t(b) * p.seq_rows;
    const int part = warp * 4 + t;
    Raw ra, rb;
    load_raw(ra, p, sm.sel, seq, s0, g, part);
    if (s0 + 1 < s1) load_raw(rb, p, sm.sel, seq, s0 + 1, g, part);
    float sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int hd = g + 8 * h;
      const float mx = fmaxf(fmaxf(sm.qmax[0][hd], sm.qmax[1][hd]), fmaxf(sm.qmax[2][hd], sm.qmax[3][hd]));
      const int e = int(__float_as_uint(mx) >> 23);                    // biased exponent of the largest magnitude
      const int up = mx > 0.f ? min(max(141 - e, -126), 126) : 0;      // 2^up puts it into [2^14, 2^15)
      const float f = __uint_as_float(uint32_t(127 + up) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i) qf[h][i] = pack_f16(bf16lo(qf[h][i]) * f, bf16hi(qf[h][i]) * f);
      sc[h] = p.scale_log2 * __uint_as_float(uint32_t(127 - up) << 23);
    }
    for (int i = s0; i < s1; ++i) {
      uint32_t kf[2][16];
      dequant(ra, kf);
      ra = rb;
      if (i + 2 < s1) load_raw(rb, p, sm.sel, seq, i + 2, g, part);
      step<true>(st, qf, kf, sm.sel_mask[i], sc[0], sc[1], sm.part[buf], warp, lane);
      buf ^= 1;
    }
  }
  if (w0 < w1) {
    if (s0 < s1) load_q();
    else __syncthreads();  // the window list
    const uint16_t* wrow = p.swa + int64_t(b) * (p.W - 1 + p.N) * CSA2_D + chan;
    for (int i = w0; i < w1; ++i) {
      uint32_t kf[2][16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t r = sm.win[i * kTile + 8 * h + g];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r >= 0) v = __ldg(reinterpret_cast<const uint4*>(wrow + int64_t(r) * CSA2_D) + j);
          kf[h][4 * j] = v.x, kf[h][4 * j + 1] = v.y, kf[h][4 * j + 2] = v.z, kf[h][4 * j + 3] = v.w;
        }
      }
      const int left = nw - i * kTile;
      step<false>(st, qf, kf, left >= kTile ? 0xFFFFu : (1u << left) - 1u, p.scale_log2, p.scale_log2, sm.part[buf], warp,
                  lane);
      buf ^= 1;
    }
  }

  float l[2] = {quad_sum(st.l0), quad_sum(st.l1)};
  float m[2] = {st.m0, st.m1};
  uint16_t* orow = p.out + row * (CSA2_H * CSA2_D);
  if (!kMerge) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float inv = l[h] > 0.f ? __fdividef(1.0f, l[h]) : 0.f;
      const float keep = inv;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = pack_bf16(st.o[4 * i + j][2 * h] * keep, st.o[4 * i + j][2 * h + 1] * keep);
        *(reinterpret_cast<uint4*>(orow + (g + 8 * h) * CSA2_D + chan) + i) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      if (p.lse && warp == 0 && t == 0)
        p.lse[row * CSA2_H + g + 8 * h] = l[h] > 0.f ? (m[h] + log2f(l[h])) * attn::kLn2 : kNegInf;
    }
    return;
  }
  SharedMerge& mg = *reinterpret_cast<SharedMerge*>(smem_raw);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (warp == 0 && t == 0) mg.ml[g + 8 * h] = make_float2(m[h], l[h]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(&mg.o[g + 8 * h][chan + 4 * i]) =
          make_float4(st.o[2 * i][2 * h], st.o[2 * i][2 * h + 1], st.o[2 * i + 1][2 * h], st.o[2 * i + 1][2 * h + 1]);
  }
  cluster_arrive_wait();
  // rank r finishes heads r * 16 / C ..
  const int heads = 16 / C;
  const uint32_t ml_a = smem_u32(mg.ml), o_a = smem_u32(mg.o);
  for (int e = tid; e < heads * (CSA2_D / 4); e += kThreads) {
    const int hd = rank * heads + e / (CSA2_D / 4), c4 = e % (CSA2_D / 4);
    float mm = kNegInf;
    for (int r = 0; r < C; ++r) mm = fmaxf(mm, ld_cluster(cluster_addr(ml_a + uint32_t(hd) * 8u, r)));
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < C; ++r) {
      const float mr = ld_cluster(cluster_addr(ml_a + uint32_t(hd) * 8u, r));
      const float w = mr == kNegInf ? 0.f : attn::ex2(mr - mm);
      sum += w * ld_cluster(cluster_addr(ml_a + uint32_t(hd) * 8u + 4u, r));
      const float4 v = ld_cluster4(cluster_addr(o_a + uint32_t(hd) * (CSA2_D * 4u) + uint32_t(c4) * 16u, r));
      acc.x += w * v.x, acc.y += w * v.y, acc.z += w * v.z, acc.w += w * v.w;
    }
    const float inv = sum > 0.f ? __fdividef(1.0f, sum) : 0.f;
    *reinterpret_cast<uint2*>(orow + hd * CSA2_D + 4 * c4) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (p.lse && c4 == 0) p.lse[row * CSA2_H + hd] = sum > 0.f ? (mm + log2f(sum)) * attn::kLn2 : kNegInf;
  }
  cluster_arrive_wait();  // no CTA leaves while its part is being read
}

cudaError_t launch(const Params& p, int64_t rows, int C, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  if (C == 1) {
    cfg.dynamicSmemBytes = sizeof(Shared);
    return cudaLaunchKernelEx(&cfg, tree_attn_kernel<false>, p, C);
  }
  cfg.dynamicSmemBytes = sizeof(SharedMerge);
  const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(sizeof(SharedMerge)));
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, tree_attn_kernel<true>, p, C);
}

}  // namespace tree
}  // namespace csa2

extern "C" csa2_status csa2_tree_attn(const uint16_t* q, int B, int N, const int32_t* parent, const int32_t* n_nodes,
                                      const uint8_t* codes, const uint8_t* scales, int64_t cap, int shared_pool,
                                      const int32_t* idx, const int32_t* n_valid, int k, const uint16_t* swa,
                                      const int32_t* win_len, int W, float softmax_scale, uint16_t* out, float* lse,
                                      csa2_stream_t stream) {
  using namespace csa2;
  if (B < 0 || N < 0 || N > CSA2_MAX_TREE || k < 0 || k > CSA2_MAX_ATTN_K || W < 0 || W > CSA2_MAX_W || cap < 0)
    return CSA2_ERR_INVALID_ARG;
  const int64_t rows = int64_t(B) * N;
  if (rows == 0) return CSA2_OK;
  auto al = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
  if (!q || !parent || !out || !al(q, 16) || !al(out, 16) || !al(parent, 4) || !al(n_nodes, 4) || !al(lse, 4))
    return CSA2_ERR_INVALID_ARG;
  if (k > 0 && (!idx || !codes || !scales || !al(codes, 16) || !al(scales, 16) || !al(idx, 4) || !al(n_valid, 4)))
    return CSA2_ERR_INVALID_ARG;
  if (W > 0 && (!swa || !al(swa, 16) || !al(win_len, 4))) return CSA2_ERR_INVALID_ARG;
  if (rows * tree::kMaxCluster > 0x7FFFFFFFll) return CSA2_ERR_INVALID_ARG;
  unsigned int* flags = device_flags_ptr();
  const int sms = sm_count();
  if (!flags || sms <= 0) return CSA2_ERR_CUDA;
  tree::Params p;
  p.q = q, p.parent = parent, p.n_nodes = n_nodes, p.codes = codes, p.scales = scales;
  p.cap = cap, p.seq_rows = shared_pool ? 0 : cap;
  p.idx = idx, p.n_valid = n_valid, p.swa = swa, p.win_len = win_len, p.out = out, p.lse = lse;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.N = N, p.k = k, p.W = W, p.flags = flags;
  int C = 1;
  while (C < tree::kMaxCluster && rows * C * 2 <= int64_t(sms) * 2) C *= 2;
  return tree::launch(p, rows, C, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
