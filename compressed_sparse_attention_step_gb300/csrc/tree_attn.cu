// Attention of a tree of drafted tokens over the FP4 main-KV cache: every drafted node attends the rows
// its indexer selected, the committed part of its sliding window and its drafted ancestors (itself
// included), o = sum_r softmax_r(q . row_r * scale) row_r with K = V = the (dequantised) row.
//
// A node has 16 heads and its own selected rows, so its two products are [16 x 512] x [512 x rows] and
// [16 x rows] x [rows x 512]: the head count is exactly the M of mma.m16n8k16, which multiplies from registers, so
// that the dequantised rows never touch shared memory (the tcgen05 kernels of the chain's attention write them
// there once and have them read twice; a chain of the same rows takes them 1.5 to 1.8 times as long):
//  - four warps split the 512 channels, lane (g, t) of a warp reads 16 bytes of codes of row g: 32
//    consecutive channels of its warp's 128.  Channels may be summed in any order, so the lane's j-th
//    channel pair serves as the j-th pair of the B fragment of S = Q K^T as it is, with Q's fragment
//    loaded in the same order;
//  - the same registers, transposed 8 x 8 by movmatrix, are the B fragments of O = P V, and the
//    accumulator of S has the layout of P's A fragment; a lane's 16 output pairs are again 32
//    consecutive channels, stored as whole 16-byte pieces;
//  - rows arrive by cp.async a few steps ahead; between the warps only partial scores and P pass.
//
// What bounds it.  A step of 16 selected rows needs 256 cycles of an SM's tensor pipe (2.0 an instruction; a step of
// window rows 384, for P's second term), about 290 issue slots of each scheduler and as many cycles of the
// shared-memory pipe (128 of them transposes), and takes a CTA 960 cycles from end to end alone (1180).  Three CTAs an
// SM (their registers) give 560 cycles a step (725): no pipe is full, the chain of a step is.  64 sequences x 32 nodes,
// all real, 512 selected and 128 window rows: 185 us on the device (4.5 waves of 456 nodes), 0.12 of the bf16 peak over
// the plain count of operations; 64 x 8 nodes 56 us.  Measured and not kept, for a ragged 64 x 32 batch that took 162
// to 169 us in this form: rows dequantised a second time for P V instead of transposed (181 us), Q in shared memory
// (205), steps of 32 rows (179), a pipeline of three steps with two CTAs an SM (190), plain loads one step ahead (223),
// bulk copies per row (307).  One sequence of five nodes, eight CTAs a node, 9.1 us: 4100 cycles until the lists stand,
// 1400 until the first rows do, 5000 for five or six steps, 5800 for the merge and its two barriers (parts pushed to the
// CTA that finishes a head 10.2 us, 16 CTAs a node 8.9 and with nine nodes 10.5 instead of 9.3).
//
// FP4 rows are multiplied as f16: a code times a scale has at most 6 significant bits and lies between
// 2^-10 and 2688, so the row is exact.  Q is scaled per head by a power of two that puts its largest
// magnitude into [2^14, 2^15), so its bf16 values are exact in f16 down to 2^-28 of that magnitude, and
// below it they are off by less than 2^-38 of it.  P is rounded to f16 (2^-11 relative; held in two terms it
// would cost 16%, 64 x 32 nodes 215 instead of 185 us, beside an output that is rounded to 2^-8).  Window rows are
// bf16 and are multiplied as bf16, with P in two bf16 terms, the second for what the first left (2^-16): one term,
// 2^-8, is as coarse as the output itself (of nodes with window rows alone a quarter of the outputs were not the
// nearest bf16), and the second costs 2% (64 x 32 nodes 185 instead of 181 us).  Scores, softmax statistics and
// outputs are accumulated in fp32; the softmax sum takes P before its rounding.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"

namespace csa2 {
namespace tree {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kMaxSel = CSA2_MAX_ATTN_K;                  // selected rows per node
constexpr int kMaxWin = CSA2_MAX_W - 1 + CSA2_MAX_TREE;   // window rows and ancestors
constexpr int kStep = 16, kSelRows = 32;                  // rows per step, selected rows per slot
constexpr int kWinList = (kMaxWin + kStep - 1) / kStep * kStep;
constexpr int kMaxCluster = 8;
constexpr float kNegInf = -INFINITY;
// The softmax reference m starts kHead below the largest score of a CTA's first step and moves only when a
// score passes it by kHead + 8, so P lies below 2^15 and the largest is at least 2^kHead: in f16's range, whose
// subnormal rounding (2^-25) is then 2^-32 of the largest P.
constexpr float kHead = 7.0f;
constexpr float kFloor = -3.402823466e38f;  // the reference before any score

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit elements held as matrix fragments (row lane / 4, columns 2 (lane % 4), + 1)
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
template <bool kF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (kF16) mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
  else mma_bf16(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) { return attn::h2_bits(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// What rounding to a pair of bf16 leaves, rounded to bf16 itself.
__device__ __forceinline__ uint32_t rest_bf16(float lo, float hi, uint32_t pair) {
  return pack_bf16(lo - bf16lo(pair), hi - bf16hi(pair));
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
  int64_t row0;  // the launch's first node
  unsigned int* flags;
};

// Staged rows.  The 16-byte pieces of a row are stored at their index XOR a function of the row, so that the
// eight lanes of a 16-byte access phase (rows g and g + 1, four t) fall into different banks.
constexpr int kSelSlots = 3, kWinSlots = 2;
__device__ __forceinline__ int sel_swz(int r) { return (r & 1) << 2; }
__device__ __forceinline__ int win_swz(int r) { return (r & 1) << 1; }

struct alignas(128) SelSlot {
  unsigned char codes[kSelRows][CSA2_CODE_BYTES];
  unsigned char scales[kSelRows][CSA2_SCALE_BYTES];
};
struct alignas(128) WinSlot {
  unsigned char rows[kStep][CSA2_D * 2];
};
struct Shared {
  WinSlot win_slot[kWinSlots];    // at the end: O of this CTA's part, for the merge
  SelSlot sel_slot[kSelSlots];
  float2 part[4][kWarps][32];     // partial scores of a step: [fragment register][warp][lane]
  uint4 prob[32];                 // P fragment of a step, one register from each warp
  uint4 rest[32];                 // what P's rounding to bf16 left, likewise (window rows)
  uint64_t sel_full[kSelSlots], win_full[kWinSlots];  // mbarriers: a slot's copies have landed
  int32_t sel[kMaxSel];           // this node's selected rows, without gaps; the last slot filled up
  int32_t win[kWinList];          // its window buffer rows, likewise
  int32_t n_sel, n_win;
  int32_t parent[CSA2_MAX_TREE];
  float qmax[kWarps][16];
  float tops[kWarps][8];          // a step's largest scores per head, where the reference moves
  float sums[kWarps][8];
  float2 ml[16];                  // (reference, sum) of this CTA's part, for the merge
};
static_assert(CSA2_H * CSA2_D * 4 <= sizeof(WinSlot) * kWinSlots, "a part's O fits the window slots");
static_assert(3 * (sizeof(Shared) + 1024) <= 228 * 1024, "three CTAs per SM");

// State of a lane: O of heads g and g + 8 over its 32 channels, the references of both, and the sum of
// the P values that this lane computes (warps 0 and 2: head g, warps 1 and 3: head g + 8).
struct State {
  float o[16][4];
  float m0, m1, l;
};

// One step of 16 rows held as fragments kf (rows g and g + 8; 16 channel pairs each), the first `left`
// of them real.  Warp w sums the four warps' partial scores for register w of P's fragment, takes their
// exponentials and hands the register to the others.  `loaded` runs once every warp holds its fragments, behind
// the second barrier, where its instructions pass beside the products (between the barriers they cost 2%).
template <bool kF16, typename F>
__device__ __forceinline__ void step(State& s, const uint32_t (&qf)[2][16], uint32_t (&kf)[2][16], int left, float scale,
                                     Shared& sm, int warp, int lane, F loaded) {
  const int t = lane & 3, g = lane >> 2;
  {
    // two chains per accumulator: a dependent MMA waits 20 cycles
    float S0[4] = {0.f, 0.f, 0.f, 0.f}, S1[4] = {0.f, 0.f, 0.f, 0.f}, T0[4] = {0.f, 0.f, 0.f, 0.f},
          T1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      mma<kF16>(S0, qf[0][2 * i], qf[1][2 * i], qf[0][2 * i + 1], qf[1][2 * i + 1], kf[0][2 * i], kf[0][2 * i + 1]);
      mma<kF16>(S1, qf[0][2 * i], qf[1][2 * i], qf[0][2 * i + 1], qf[1][2 * i + 1], kf[1][2 * i], kf[1][2 * i + 1]);
      mma<kF16>(T0, qf[0][2 * i + 2], qf[1][2 * i + 2], qf[0][2 * i + 3], qf[1][2 * i + 3], kf[0][2 * i + 2],
                kf[0][2 * i + 3]);
      mma<kF16>(T1, qf[0][2 * i + 2], qf[1][2 * i + 2], qf[0][2 * i + 3], qf[1][2 * i + 3], kf[1][2 * i + 2],
                kf[1][2 * i + 3]);
    }
    sm.part[0][warp][lane] = make_float2(S0[0] + T0[0], S0[1] + T0[1]);  // head g, rows 2t, 2t + 1
    sm.part[1][warp][lane] = make_float2(S0[2] + T0[2], S0[3] + T0[3]);  // head g + 8
    sm.part[2][warp][lane] = make_float2(S1[0] + T1[0], S1[1] + T1[1]);  // rows 8 + 2t, 9 + 2t
    sm.part[3][warp][lane] = make_float2(S1[2] + T1[2], S1[3] + T1[3]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) kf[0][i] = transpose8(kf[0][i]), kf[1][i] = transpose8(kf[1][i]);
  __syncthreads();
  const float2 a = sm.part[warp][0][lane], b = sm.part[warp][1][lane], c = sm.part[warp][2][lane],
               d = sm.part[warp][3][lane];
  float x0 = ((a.x + b.x) + (c.x + d.x)) * scale, x1 = ((a.y + b.y) + (c.y + d.y)) * scale;
  if (left < kStep) {
    const int r = 8 * (warp >> 1) + 2 * t;
    if (r >= left) x0 = kNegInf;
    if (r + 1 >= left) x1 = kNegInf;
  }
  const float m = (warp & 1) ? s.m1 : s.m0;
  float p0 = attn::ex2(x0 - m), p1 = attn::ex2(x1 - m);
  auto put = [&]() {
    const uint32_t pair = kF16 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
    reinterpret_cast<uint32_t*>(&sm.prob[lane])[warp] = pair;
    if (!kF16) reinterpret_cast<uint32_t*>(&sm.rest[lane])[warp] = rest_bf16(p0, p1, pair);
  };
  put();
  if (__syncthreads_or(fmaxf(x0, x1) > m + (kHead + 8.f))) {
    // the references move: to the largest scores of this step less kHead, where that is more
    const float top = quad_max(fmaxf(x0, x1));
    if (t == 0) sm.tops[warp][g] = top;
    __syncthreads();
    const float n0 = fmaxf(s.m0, fmaxf(sm.tops[0][g], sm.tops[2][g]) - kHead);
    const float n1 = fmaxf(s.m1, fmaxf(sm.tops[1][g], sm.tops[3][g]) - kHead);
    const float c0 = s.m0 == n0 ? 1.f : attn::ex2(s.m0 - n0), c1 = s.m1 == n1 ? 1.f : attn::ex2(s.m1 - n1);
    s.m0 = n0, s.m1 = n1;
    const float n = (warp & 1) ? n1 : n0;
    s.l *= (warp & 1) ? c1 : c0;
#pragma unroll
    for (int i = 0; i < 16; ++i) s.o[i][0] *= c0, s.o[i][1] *= c0, s.o[i][2] *= c1, s.o[i][3] *= c1;
    p0 = attn::ex2(x0 - n), p1 = attn::ex2(x1 - n);
    put();
    __syncthreads();
  }
  const uint4 p = sm.prob[lane];
  s.l += p0 + p1;
  loaded();
#pragma unroll
  for (int i = 0; i < 16; ++i) mma<kF16>(s.o[i], p.x, p.y, p.z, p.w, kf[0][i], kf[1][i]);
  if (!kF16) {
    const uint4 r = sm.rest[lane];
#pragma unroll
    for (int i = 0; i < 16; ++i) mma<kF16>(s.o[i], r.x, r.y, r.z, r.w, kf[0][i], kf[1][i]);
  }
}

// Rows g and g + 8 of a step of selected rows: f16 pairs of this lane's 32 channels.
__device__ __forceinline__ void dequant(const unsigned char* codes, const unsigned char* scales, uint32_t (&kf)[2][16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 c = *reinterpret_cast<const uint4*>(codes + 8 * h * CSA2_CODE_BYTES);
    const __half2 s2 =
        attn::bits_h2(attn::e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(scales + 8 * h * CSA2_SCALE_BYTES)));
    const __half2 lo = __low2half2(s2), hi = __high2half2(s2);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      attn::e2m1x8_to_f16x2x4(w[i], kf[h][4 * i], kf[h][4 * i + 1], kf[h][4 * i + 2], kf[h][4 * i + 3]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        kf[h][4 * i + j] = attn::h2_bits(__hmul2(attn::bits_h2(kf[h][4 * i + j]), i < 2 ? lo : hi));
    }
  }
}

// The calling thread's cp.async copies so far arrive at the mbarrier when they have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cluster_arrive_wait() {
  __syncwarp();  // an aligned barrier counts a warp that comes in two parts twice
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// (not volatile: several may be under way; the cluster barriers around them order them)
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm("ld.shared::cluster.v2.f32 {%0,%1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// One node per cluster of C CTAs (C = 1: per CTA), which share its steps of 16 rows and merge their
// parts through distributed shared memory, in rank order.
template <int C>
__global__ void __launch_bounds__(kThreads, 3) tree_attn_kernel(const Params p) {
  constexpr bool kMerge = C > 1;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  pdl_wait();
  pdl_trigger();
  const int rank = kMerge ? int(blockIdx.x % C) : 0;
  const int64_t row = p.row0 + (kMerge ? int64_t(blockIdx.x / C) : int64_t(blockIdx.x));
  const int b = int(row / p.N), node = int(row - int64_t(b) * p.N);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // everything that the row lists need is asked for at once
  const int nodes = p.n_nodes ? __ldg(p.n_nodes + b) : p.N;
  int nv = p.k;
  int32_t ids[kMaxSel / 32];
  if (warp == 0) {
    if (p.n_valid) nv = min(max(__ldg(p.n_valid + row), 0), p.k);
#pragma unroll
    for (int j = 0; j < kMaxSel / 32; ++j) ids[j] = 32 * j + lane < p.k ? __ldg(p.idx + row * p.k + 32 * j + lane) : -1;
  }
  int up0 = -1, up1 = -1, wl = p.W - 1;
  if (warp == 1) {
    if (lane < p.N) up0 = __ldg(p.parent + int64_t(b) * p.N + lane);
    if (lane + 32 < p.N) up1 = __ldg(p.parent + int64_t(b) * p.N + lane + 32);
    if (p.win_len) wl = __ldg(p.win_len + b);
  }
  const int chan = warp * 128 + t * 32;  // this lane's 32 channels

  // Q of heads g and g + 8, as bf16 pairs
  const uint16_t* qrow = p.q + row * (CSA2_H * CSA2_D) + chan;
  uint32_t qf[2][16];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // in the order of the window's pieces
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(qrow + (g + 8 * h) * CSA2_D) + (i ^ (t >> 1)));
      qf[h][4 * i] = v.x, qf[h][4 * i + 1] = v.y, qf[h][4 * i + 2] = v.z, qf[h][4 * i + 3] = v.w;
    }
  if (node >= nodes) return;  // the whole cluster: its outputs stay as they were
  if (tid == 0) {
    for (int j = 0; j < kSelSlots; ++j)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(&sm.sel_full[j])), "n"(kThreads) : "memory");
    for (int j = 0; j < kWinSlots; ++j)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(&sm.win_full[j])), "n"(kThreads) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }

  // The row lists, without gaps: warp 0 the selected rows, warp 1 the window rows.  The entries that fill a
  // list's last step repeat a row of the node's own; their P is zero.
  if (warp == 0) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < kMaxSel / 32; ++j) {
      const bool ok = 32 * j + lane < nv && ids[j] >= 0 && int64_t(ids[j]) < p.cap;
      if (32 * j + lane < nv && int64_t(ids[j]) >= p.cap) atomicOr(p.flags, CSA2_FLAG_INDEX_OOB);
      const uint32_t bal = __ballot_sync(0xffffffffu, ok);
      if (ok) sm.sel[n + __popc(bal & ((1u << lane) - 1u))] = ids[j];
      n += __popc(bal);
    }
    __syncwarp();
    if (n & (kSelRows - 1)) {
      const int i = n + lane;
      if (i < (n + kSelRows - 1) / kSelRows * kSelRows) sm.sel[i] = sm.sel[0];
    }
    if (lane == 0) sm.n_sel = n;
  } else if (warp == 1) {
    sm.parent[lane] = up0, sm.parent[lane + 32] = up1;
    __syncwarp();
    // ancestors of the node, itself included
    uint64_t anc = 0;
    int depth = -1;
    for (int cur = node; cur >= 0;) {
      anc |= 1ull << cur;
      ++depth;
      const int up = sm.parent[cur];
      if (up < -1 || up >= cur) {  // not a tree in node order: taken as a root
        if (lane == 0 && rank == 0) atomicOr(p.flags, CSA2_FLAG_INDEX_OOB);
        break;
      }
      cur = up;
    }
    // the committed rows [first, W - 1), then the ancestors less than W tokens away
    int nw = 0;
    if (p.W > 0) {
      wl = min(max(wl, 0), p.W - 1);
      const int first = max(depth, p.W - 1 - wl), n_com = max(p.W - 1 - first, 0);
      const int drop = max(depth + 1 - p.W, 0);  // the bits of anc ascend with the depth
      for (int i = 0; i < drop; ++i) anc &= anc - 1;
      nw = n_com + __popcll(anc);
      for (int i = lane; i < (nw + kStep - 1) / kStep * kStep; i += 32) {
        int32_t r = p.W - 1 + node;
        if (i < n_com) r = first + i;
        else if (i < nw) {
          uint64_t m = anc;
          for (int j = n_com; j < i; ++j) m &= m - 1;
          r = p.W - 1 + (__ffsll(static_cast<long long>(m)) - 1);
        }
        sm.win[i] = r;
      }
    }
    if (lane == 0) sm.n_win = nw;
  }
  // per head: the largest magnitude of Q
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) am = max(am, max(qf[h][i] & 0x7FFFu, (qf[h][i] >> 16) & 0x7FFFu));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    if (t == 0) sm.qmax[warp][g + 8 * h] = __uint_as_float(am << 16);
  }
  __syncthreads();

  const int n_sel = sm.n_sel, n_win = sm.n_win;
  const int win_steps = (n_win + kStep - 1) / kStep, sel_steps = (n_sel + kSelRows - 1) / kSelRows;
  const bool any = win_steps + sel_steps > 0;
  // this CTA's steps: of the list of window steps (weight 1) and selected steps (weight 2)
  int w0 = 0, w1 = win_steps, s0 = 0, s1 = sel_steps;
  if (kMerge) {
    const int total = win_steps + 2 * sel_steps;
    const int i0 = total * rank / C, i1 = total * (rank + 1) / C;
    w0 = min(i0, win_steps), w1 = min(i1, win_steps);
    s0 = (max(i0 - win_steps, 0) + 1) / 2, s1 = (max(i1 - win_steps, 0) + 1) / 2;
  }

  // Copies of a step's rows, by all threads; every row of the lists is valid.
  const int64_t win_base = int64_t(b) * (p.W - 1 + p.N), sel_base = int64_t(b) * p.seq_rows;
  auto fill_win = [&](int i) {
    if (i >= w1) return;
    const int sl = (i - w0) % kWinSlots, r = tid >> 3, c = tid & 7;
    const unsigned char* src = reinterpret_cast<const unsigned char*>(p.swa + (win_base + sm.win[i * kStep + r]) * CSA2_D);
    const uint32_t dst = smem_u32(&sm.win_slot[sl].rows[r][(c ^ win_swz(r)) * 16]);
#pragma unroll
    for (int j = 0; j < 8; ++j) cp_async16(dst + 128 * j, src + 16 * c + 128 * j, 16);
    cp_async_arrive(smem_u32(&sm.win_full[sl]));
  };
  auto fill_sel = [&](int i) {
    if (i >= s1) return;
    const int sl = (i - s0) % kSelSlots, r = tid >> 2, c = tid & 3;
    const int64_t row = sel_base + sm.sel[i * kSelRows + r];
    const uint8_t* src = p.codes + row * CSA2_CODE_BYTES + 16 * c;
    const uint32_t dst = smem_u32(&sm.sel_slot[sl].codes[r][(c ^ sel_swz(r)) * 16]);  // piece c + 4j: XOR 4j
#pragma unroll
    for (int j = 0; j < 4; ++j) cp_async16((dst ^ (64 * (j & 1))) + 128 * (j >> 1), src + 64 * j, 16);
    if (c < 2) cp_async16(smem_u32(&sm.sel_slot[sl].scales[r][16 * c]), p.scales + row * CSA2_SCALE_BYTES + 16 * c, 16);
    cp_async_arrive(smem_u32(&sm.sel_full[sl]));
  };
  for (int j = 0; j < kWinSlots; ++j) fill_win(w0 + j);
  for (int j = 0; j < kSelSlots; ++j) fill_sel(s0 + j);
  bool late = false;  // copies did not land within a second: flagged, and no more waiting
  auto wait_full = [&](uint64_t* bar, int use) {
    if (!late && !bar_wait(smem_u32(bar), uint32_t(use) & 1u)) {
      late = true;
      atomicOr(p.flags, CSA2_FLAG_TIMEOUT);
    }
    __syncwarp();  // (the lanes' waits end one by one)
  };

  State st;
  st.m0 = st.m1 = kFloor;
  st.l = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;

  for (int i = w0; i < w1; ++i) {
    wait_full(&sm.win_full[(i - w0) % kWinSlots], (i - w0) / kWinSlots);
    const unsigned char* src = &sm.win_slot[(i - w0) % kWinSlots].rows[g][0];
    uint32_t kf[2][16];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // lanes t >= 2 take their pieces in the order 1, 0, 3, 2 (as qf then holds Q's)
        const int piece = (warp * 16 + t * 4 + (j ^ (t >> 1))) ^ win_swz(g);
        const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * h * CSA2_D * 2 + piece * 16);
        kf[h][4 * j] = v.x, kf[h][4 * j + 1] = v.y, kf[h][4 * j + 2] = v.z, kf[h][4 * j + 3] = v.w;
      }
    step<false>(st, qf, kf, n_win - i * kStep, p.scale_log2, sm, warp, lane, [&]() { fill_win(i + kWinSlots); });
  }
  if (w0 < w1) {  // O in the order of the channels
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & 4)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = st.o[i][e], c = st.o[i + 4][e];
          st.o[i][e] = t < 2 ? a : c, st.o[i + 4][e] = t < 2 ? c : a;
        }
      }
  }
  if (s0 < s1) {
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
#pragma unroll
      for (int i = 0; i < 16; ++i)  // back to the order of the channels
        if (!(i & 4)) {
          const uint32_t a = qf[h][i], c = qf[h][i + 4];
          qf[h][i] = t < 2 ? a : c, qf[h][i + 4] = t < 2 ? c : a;
        }
      sc[h] = p.scale_log2 * __uint_as_float(uint32_t(127 - up) << 23);
    }
    const float scale = (warp & 1) ? sc[1] : sc[0];
    const int code_off = g * CSA2_CODE_BYTES + ((warp * 4 + t) ^ sel_swz(g)) * 16;
    const int scale_off = g * CSA2_SCALE_BYTES + warp * 8 + t * 2;
    for (int i = s0; i < s1; ++i) {
      const int k = i - s0;
      wait_full(&sm.sel_full[k % kSelSlots], k / kSelSlots);
      const unsigned char* codes = &sm.sel_slot[k % kSelSlots].codes[0][0] + code_off;
      const unsigned char* scales = &sm.sel_slot[k % kSelSlots].scales[0][0] + scale_off;
      int left = n_sel - i * kSelRows;
      if (left > kStep) {
        uint32_t kf[2][16];
        dequant(codes, scales, kf);
        step<true>(st, qf, kf, left, scale, sm, warp, lane, []() {});
        codes += kStep * CSA2_CODE_BYTES, scales += kStep * CSA2_SCALE_BYTES, left -= kStep;
      }
      uint32_t kf[2][16];
      dequant(codes, scales, kf);
      step<true>(st, qf, kf, left, scale, sm, warp, lane, [&]() { fill_sel(i + kSelSlots); });
    }
  }

  if (late) bar_drain<kWinSlots>(sm.win_full, w1 - w0), bar_drain<kSelSlots>(sm.sel_full, s1 - s0);
  {
    const float l = quad_sum(st.l);
    if (t == 0) sm.sums[warp][g] = l;
  }
  __syncthreads();
  const float l[2] = {sm.sums[0][g] + sm.sums[2][g], sm.sums[1][g] + sm.sums[3][g]};
  const float m[2] = {st.m0, st.m1};
  uint16_t* orow = p.out + row * (CSA2_H * CSA2_D);
  if (!kMerge) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float inv = any ? __fdividef(1.0f, l[h]) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pack_bf16(st.o[4 * i + j][2 * h] * inv, st.o[4 * i + j][2 * h + 1] * inv);
        *(reinterpret_cast<uint4*>(orow + (g + 8 * h) * CSA2_D + chan) + i) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      if (p.lse && warp == 0 && t == 0)
        p.lse[row * CSA2_H + g + 8 * h] = any ? (m[h] + log2f(l[h])) * attn::kLn2 : kNegInf;
    }
    return;
  }
  if constexpr (kMerge) {
    // O of this CTA's part into the window slots (every copy into them has landed), as 16-byte pieces placed at
    // their index XOR a function of head and lane, so that eight lanes fall into different banks
    float4(*mo)[CSA2_D / 4] = reinterpret_cast<float4(*)[CSA2_D / 4]>(sm.win_slot);
    auto place = [](int head, int c4) { return c4 ^ (((c4 >> 3) & 3) | ((head & 1) << 2)); };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (warp == 0 && t == 0) sm.ml[g + 8 * h] = make_float2(m[h], l[h]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        mo[g + 8 * h][place(g + 8 * h, chan / 4 + i)] = make_float4(st.o[2 * i][2 * h], st.o[2 * i][2 * h + 1],
                                                                    st.o[2 * i + 1][2 * h], st.o[2 * i + 1][2 * h + 1]);
    }
    cluster_arrive_wait();
    // rank r finishes heads r * 16 / C ..: the parts' weights first, then their sums, all loads of a thread at once
    constexpr int kHeads = 16 / C;
    float* weight = sm.qmax[0];  // [kHeads][C]
    if (tid < kHeads) {
      const int hd = rank * kHeads + tid;
      float2 part[C];
      float mm = kFloor, sum = 0.f;
#pragma unroll
      for (int r = 0; r < C; ++r) part[r] = ld_cluster2(cluster_addr(smem_u32(&sm.ml[hd]), r));
#pragma unroll
      for (int r = 0; r < C; ++r) mm = fmaxf(mm, part[r].x);
#pragma unroll
      for (int r = 0; r < C; ++r) {
        part[r].x = part[r].x == mm ? 1.f : attn::ex2(part[r].x - mm);
        sum += part[r].x * part[r].y;
      }
      const float inv = any ? __fdividef(1.0f, sum) : 0.f;
#pragma unroll
      for (int r = 0; r < C; ++r) weight[tid * C + r] = part[r].x * inv;
      if (p.lse) p.lse[row * CSA2_H + hd] = any ? (mm + log2f(sum)) * attn::kLn2 : kNegInf;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int hd = rank * kHeads + i;
      const uint32_t at = smem_u32(&mo[hd][place(hd, tid)]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const float4 v = ld_cluster4(cluster_addr(at, r));
        const float w = weight[i * C + r];
        acc.x += w * v.x, acc.y += w * v.y, acc.z += w * v.z, acc.w += w * v.w;
      }
      *reinterpret_cast<uint2*>(orow + hd * CSA2_D + 4 * tid) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
    cluster_arrive_wait();  // no CTA leaves while its part is being read
  }
}

template <int C>
cudaError_t launch(const Params& p, int64_t rows, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(tree_attn_kernel<C>), sizeof(Shared), done);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, tree_attn_kernel<C>, p);
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
  if (!q || !parent || !out || !al(q, 16) || !al(out, 16) || !al(parent, 4) || !al(n_nodes, 4) ||
      !al(n_valid, 4) || !al(win_len, 4) || !al(lse, 4))
    return CSA2_ERR_INVALID_ARG;
  if (k > 0 && (!idx || (cap > 0 && (!codes || !scales)) || !al(codes, 16) || !al(scales, 16) || !al(idx, 4)))
    return CSA2_ERR_INVALID_ARG;
  if (W > 0 && (!swa || !al(swa, 16))) return CSA2_ERR_INVALID_ARG;
  if (rows * tree::kMaxCluster > 0x7FFFFFFFll) return CSA2_ERR_INVALID_ARG;
  const int64_t row_bytes = CSA2_H * CSA2_D * 2, pool = k == 0 ? 0 : shared_pool ? 1 : B;
  const Span spans[] = {span(out, rows, row_bytes),
                        span(lse, rows, CSA2_H * 4),
                        span(parent, rows, 4),
                        span(n_nodes, B, 4),
                        span(codes, pool, std::min(cap, int64_t(1) << 48) * CSA2_CODE_BYTES),
                        span(scales, pool, std::min(cap, int64_t(1) << 48) * CSA2_SCALE_BYTES),
                        span(idx, rows, int64_t(k) * 4),
                        span(n_valid, rows, 4),
                        span(W > 0 ? swa : nullptr, B, (int64_t(W) - 1 + N) * CSA2_D * 2),
                        span(win_len, B, 4),
                        span(out == q ? nullptr : q, rows, row_bytes)};  // in place, but not moved by some rows
  if (any_overlap(spans, 2, 11) || overlap(spans[1], span(q, rows, row_bytes))) return CSA2_ERR_INVALID_ARG;
  unsigned int* flags = device_flags_ptr();
  const int sms = sm_count();
  if (!flags || sms <= 0) return CSA2_ERR_CUDA;
  tree::Params p;
  p.q = q, p.parent = parent, p.n_nodes = n_nodes, p.codes = codes, p.scales = scales;
  p.cap = cap, p.seq_rows = shared_pool ? 0 : cap;
  p.idx = idx, p.n_valid = n_valid, p.swa = swa, p.win_len = win_len, p.out = out, p.lse = lse;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.N = N, p.k = k, p.W = W, p.row0 = 0, p.flags = flags;
  // Few nodes are shared by several CTAs each, which costs a merge.  Measured, us for 1 / 2 / 4 / 8 CTAs a node, 512
  // selected and 128 window rows: 5 nodes 24.0 / 16.6 / 11.6 / 9.3, 20 nodes 24.2 / 16.9 / 11.9 / 11.2, 38 nodes 24.4 /
  // 17.1 / 14.0 / 14.7, 80 nodes 24.7 / 21.2 / 18.1 / 26.8, 95 nodes 24.6 / 21.8 / 18.2 / 27.9, 104 nodes 24.6 / 21.9 /
  // 18.3 / 32.4, 112 nodes (whose clusters of four no longer run at once) 24.6 / 21.8 / 26.8 / 35.6.  Fewer rows, for
  // 1 / 4: 95 nodes 256 rows 12.2 / 11.8, 192 of them 11.5 / 12.3, 128 of them 8.3 / 10.0; 38 nodes 128 rows 8.2 / 7.9,
  // 64 of them 6.2 / 7.9; for 1 / 8: 5 nodes 128 rows 7.8 / 7.1, 64 of them 5.9 / 6.9.
  auto ctas = [&](int64_t r) {
    if (k + W < 128 || r * 8 > 5 * int64_t(sms) || (r * 4 > sms && k + W < 256)) return 1;
    return r * 8 <= sms ? 8 : 4;
  };
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto launch = [&](int64_t row0, int64_t r) {
    p.row0 = row0;
    switch (ctas(r)) {
      case 1: return tree::launch<1>(p, r, st);
      case 4: return tree::launch<4>(p, r, st);
      default: return tree::launch<8>(p, r, st);
    }
  };
  // Three nodes an SM run at once.  A few nodes behind the last full wave would take as long as a whole one: they are
  // shared by several CTAs each, in a second launch, where there are rows to pay for it.  Measured, us for two launches /
  // one, selected + window rows: behind one wave, 58 x 8 nodes 512 + 128 50.8 / 60.6, 192 + 128 33.3 / 36.0, 256 + 0 27.0 /
  // 28.2, 64 + 0 16.8 / 13.6; 64 x 8 nodes 56.2 / 61.3, 36.3 / 36.9, 29.5 / 28.9, 18.4 / 14.1; behind two, 120 x 8 nodes
  // 512 + 128 98.1 / 99.9, 384 + 128 83.6 / 84.1, 256 + 128 68.4 / 67.8, 256 + 0 47.9 / 45.7; more nodes than half the SMs
  // gain little or nothing (546 x 1, 90 behind the wave: 512 + 128 66.1 / 66.4, 512 + 0 50.9 / 50.0).  Not with n_nodes:
  // nodes that are not real leave room in the last wave (of 64 x 8 nodes, 437 to 496 real ones took 46.3 us in one).
  const int64_t wave = 3 * int64_t(sms), rest = rows % wave;
  cudaError_t e;
  if (!n_nodes && rows > wave && rest > 0 && 2 * rest <= sms && k + W >= (rows < 2 * wave ? 320 : 512) &&
      ctas(rest) > 1) {
    e = launch(0, rows - rest);
    if (e == cudaSuccess) e = launch(rows - rest, rest);
  } else {
    e = launch(0, rows);
  }
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
