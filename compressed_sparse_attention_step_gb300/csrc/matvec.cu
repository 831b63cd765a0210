// Products of a few token rows with a 4-bit weight: y[m][n] = row_scale[n] sum_k x[m][k] e2m1[n][k] e4m3[n][k/16].
//
// Bound: the weight's 0.5625 bytes per element from HBM, in one pass; x and y are small beside it.
//
// Layout.  The weight is packed once into blocks of 32 output rows x 128 input channels, 2304 bytes each: four
// pieces of 32 channels, 16 bytes of codes per row and piece, then eight scale bytes per row; row r of piece j lies
// at place r ^ 2j, so that a warp's 16-byte reads fall into different banks of shared memory whether its lanes own a
// row each or, as fragments of m16n8k16, eight rows and four pieces.  Blocks of the same rows follow each other
// along the channels.  Rows and channels past the weight are zero codes.  A warp brings its blocks into shared
// memory itself, by one bulk copy each, a few blocks ahead (plain loads into registers reached less than half of
// the bandwidth, however many were in flight).
//
// Numbers.  A code times a scale is exact in f16 (6 significant bits, 2^-10 .. 2688).  x is bf16: it is scaled by
// the power of two that brings the largest magnitude of a token's share of channels (a block's 128, or a CTA's)
// into [2^14, 2^15), and is then exact in f16 down to 2^-28 of that magnitude, off by less than 2^-38 of it below;
// the sums are scaled back in fp32.  All sums are fp32, in a fixed order, and are rounded once.
//
// Two kernels.  matvec_tc_kernel: the weight is the M = 128 operand of tcgen05.mma, dequantised into tensor
// memory, so that a weight element costs one conversion and one multiplication and no pass through shared memory,
// and the token rows (N = 16 or 32) cost the warps nothing.  matvec_kernel: mma.m16n8k16 from registers, with
// less to set up.
//
// Measured (us, weights from HBM; in brackets at the copy bandwidth): one row x 512 x 4096 3.8 (0.17), 4096 x 4096
// 6.2 (1.4), 16384 x 8192 17.0 (11.1), 32768 x 16384 55 (44.4); eight rows 4.3, 6.8, 19.6, 65; five rows x 8200 x 4112
// 9.4 (2.8; 8.2 with the weight in L2); 32 rows x 16384 x 8192 28.7 (26.9 with the weight partly in L2), 32768 x 16384
// 92.  Packing 16384 x 8192: 65 us (22 at the copy bandwidth), once per weight: a lane reads eight bytes of its own row.
// What bounds matvec_kernel: 4 us of launch, staging and exchange, behind which the copies alone take as long as the
// products alone (16384 x 8192, eight rows: 17.8 and 17.7 with those 4; more blocks under way, more CTAs or even shares
// of the rows gain nothing).  matvec_tc_kernel: 6 us before the first product (x, 128 KB a CTA), then about 560 cycles
// per 128 x 128 block, of which the copies need 390, a dequantising group 380 and the issuing threads 380, coupled by
// the six tensor-memory buffers between them.  Copies of four blocks by warps of their own gained nothing (24.6 for 16
// rows, 29.6 for 32, whose staging then spills).
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "matvec_plan.h"

namespace csa2 {
namespace mv {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 32, kChan = 128;     // block
constexpr int kCodeBytes = kRows * kChan / 2;
constexpr int kBlock = kCodeBytes + kRows * kChan / CSA2_GROUP;  // 2304 bytes
constexpr int kStage = 36 * 1024;          // bytes of x staged at a time (two CTAs per SM with up to 16 tokens)
constexpr int kSlots = 3;                  // blocks a warp of matvec_kernel has under way
constexpr int kMaxCluster = 8;
// of matvec_kernel: the rings, x of 8 blocks x 32 tokens (or kStage), the partial sums
constexpr size_t kMaxSmem = size_t(kWarps) * kSlots * kBlock + 8 * 32 * (kChan * 2 + 4) + 8 * 32 * 32 * 4;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// where piece j (32 channels) of row r lies in a block
__device__ __forceinline__ int block_place(int r, int j) { return j * 512 + (r ^ (2 * j)) * 16; }

// A block into shared memory; one thread.
__device__ __forceinline__ void block_copy(void* dst, const uint8_t* src, uint64_t* bar) {
  const uint32_t b = smem_u32(bar);
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(b), "r"(kBlock) : "memory");
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(kBlock), "r"(b)
               : "memory");
}

// A warp per block, a lane per row.
__global__ void __launch_bounds__(256) pack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                   int64_t n_out, int64_t n_in, int64_t n_kb, int64_t n_blocks,
                                                   uint8_t* __restrict__ packed) {
  pdl_wait();
  pdl_trigger();
  const int64_t blk = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (blk >= n_blocks) return;
  const int lane = int(threadIdx.x & 31);
  const int64_t rb = blk / n_kb, kb = blk - rb * n_kb, row = rb * kRows + lane;
  uint8_t* dst = packed + blk * kBlock;
  uint32_t sb[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // groups of 16 channels; n_in is a multiple of 16
    const int64_t c0 = kb * kChan + 16 * j;
    uint2 w = make_uint2(0, 0);
    if (row < n_out && c0 < n_in) {
      w = *reinterpret_cast<const uint2*>(codes + row * (n_in / 2) + c0 / 2);
      sb[j >> 2] |= uint32_t(scales[row * (n_in / CSA2_GROUP) + c0 / CSA2_GROUP]) << (8 * (j & 3));
    }
    *reinterpret_cast<uint2*>(dst + block_place(lane, j >> 1) + (j & 1) * 8) = w;
  }
  *reinterpret_cast<uint2*>(dst + kCodeBytes + lane * 8) = make_uint2(sb[0], sb[1]);
}

// (A warp that comes to an aligned barrier in two parts is counted twice, and others pass before it has arrived: the
// lanes are brought together first.)
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_wait() { cluster_arrive(), cluster_wait(); }
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
// a shared-memory address of this CTA is one of the cluster's as well
__device__ __forceinline__ void st_cluster(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(a), "f"(v) : "memory");
}
struct Unit {  // a block as fragments: rows 16 r + 8 h + g, channels 32t .. 32t+31
  uint4 c[2][2];
  uint32_t s[2][2];
};

struct Params {
  const uint16_t* x;
  const uint8_t* packed;
  const float* row_scale;
  void* y;
  int64_t n_out, n_in;
  int m, n_kb, n_rb;     // token rows, channel blocks, row blocks
  int stage_kb;          // channel blocks staged at a time (a multiple of 8)
  int y_fp32;
  unsigned int* flags;
};

// TG: groups of 8 token rows; WR: warps along the output rows.
template <int TG, int WR>
__global__ void __launch_bounds__(kThreads, TG <= 2 ? 2 : 1) matvec_kernel(const Params p, int C) {
  constexpr int WK = kWarps / WR;
  constexpr int kTok = TG * 8;
  constexpr int kCtaRows = WR * 32;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kWarps][kSlots];
  unsigned char* ring = smem + (threadIdx.x >> 5) * (kSlots * kBlock);                 // of this warp
  unsigned char* stage = smem + kWarps * kSlots * kBlock;
  uint4* xs = reinterpret_cast<uint4*>(stage);                                         // [kb][TG][4][32 lanes]
  float* xf = reinterpret_cast<float*>(stage + size_t(p.stage_kb) * kTok * kChan * 2);  // [kb][kTok]
  // partial sums of the rows that this CTA finishes: [rank][WK][kTok][kCtaRows / C]
  float* red = reinterpret_cast<float*>(stage + size_t(p.stage_kb) * kTok * (kChan * 2 + 4));
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3, g = lane >> 2;
  const int wr = warp / WK, wk = warp % WK;
  if (C > 1) cluster_arrive();
  const int rank = C > 1 ? int(blockIdx.x % unsigned(C)) : 0;
  const int64_t row0 = int64_t(blockIdx.x / unsigned(C)) * kCtaRows;
  const int kb0 = int(uint32_t(p.n_kb) * uint32_t(rank) / uint32_t(C)),
            kb1 = int(uint32_t(p.n_kb) * uint32_t(rank + 1) / uint32_t(C));
  const int rb = int(row0 / kRows) + wr;

  // this warp's blocks: channel blocks kb0 + wk, + WK, ... of row block rb; none past the weight's rows
  const int n_blk = rb < p.n_rb && kb1 - kb0 > wk ? (kb1 - kb0 - wk + WK - 1) / WK : 0;
  const uint8_t* src = p.packed + (int64_t(rb) * p.n_kb + kb0 + wk) * kBlock;
  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&full[warp][i])) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    for (int i = 0; i < min(n_blk, kSlots); ++i)
      block_copy(ring + i * kBlock, src + int64_t(i) * WK * kBlock, &full[warp][i]);
  }
  __syncwarp();
  int slot = 0, use = 0, done = 0;
  int late = 0;  // a copy did not land within a second: flagged, no more waiting or copying; the copies begun

  float acc[2][TG][4];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int j = 0; j < TG; ++j) acc[r][j][0] = acc[r][j][1] = acc[r][j][2] = acc[r][j][3] = 0.f;

  for (int c0 = kb0; c0 < kb1; c0 += p.stage_kb) {
    const int nk = min(p.stage_kb, kb1 - c0);
    if (c0 != kb0) __syncthreads();
    // stage x: half a warp per (block, token), 8 channels a lane, four of them loaded together.  Rows past the last
    // token are left as they are: they reach their own columns of the sums alone.
    for (int it0 = tid >> 4; it0 < nk * p.m; it0 += 4 * (kThreads / 16)) {
      const int j = tid & 15;
      int kb[4], tok[4];
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int it = it0 + e * (kThreads / 16);
        kb[e] = it / p.m, tok[e] = it - kb[e] * p.m;
        const int64_t ch = int64_t(c0 + kb[e]) * kChan + 8 * j;
        v[e] = make_uint4(0, 0, 0, 0);
        if (kb[e] < nk && ch < p.n_in) v[e] = __ldg(reinterpret_cast<const uint4*>(p.x + int64_t(tok[e]) * p.n_in + ch));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (kb[e] >= nk) break;
        const uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
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
        xs[((kb[e] * TG + (tok[e] >> 3)) * 4 + (j & 3)) * 32 + (tok[e] & 7) * 4 + (j >> 2)] = make_uint4(o[0], o[1], o[2], o[3]);
        if (j == 0) xf[kb[e] * kTok + tok[e]] = __uint_as_float(uint32_t(127 - up) << 23);
      }
    }
    // Every CTA of the cluster has started.  All warps are past this wait before one comes to the next arrival: a warp
    // that was still to wait would count as arrived there.
    if (C > 1 && c0 == kb0) cluster_wait();
    __syncthreads();
    for (int kb = wk; kb < nk && done < n_blk; kb += WK, ++done) {
      if (!late && !bar_wait(smem_u32(&full[warp][slot]), uint32_t(use) & 1u)) {
        late = min(n_blk, done + kSlots);
        atomicOr(p.flags, CSA2_FLAG_TIMEOUT);
      }
      Unit u0;
      {
        const unsigned char* blk = ring + slot * kBlock;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = 16 * r + 8 * h + g;
            u0.c[r][h] = *reinterpret_cast<const uint4*>(blk + block_place(row, t));
            u0.s[r][h] = *reinterpret_cast<const uint16_t*>(blk + kCodeBytes + row * 8 + 2 * t);
          }
      }
      attn::fence_async_smem();  // what the lanes have read comes before what the copy writes
      __syncwarp();
      if (lane == 0 && !late && done + kSlots < n_blk)
        block_copy(ring + slot * kBlock, src + int64_t(done + kSlots) * WK * kBlock, &full[warp][slot]);
      if (++slot == kSlots) slot = 0, ++use;
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
          const __half2 s2 = attn::bits_h2(attn::e4m3x2_to_f16x2(uint16_t(u0.s[r][h])));
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
  if (lane == 0 && late) bar_drain<kSlots>(full[warp], late);
  // Each partial sum goes to the CTA of the cluster that finishes its row, rank row / (kCtaRows / C), which adds them
  // up in order of rank and warp.  acc[r][j]: rows g (0, 1) and g + 8 (2, 3) of half r, tokens 8j + 2t and + 1.
  const int rows = kCtaRows / C;
  const uint32_t red_a = smem_u32(red) + 4u * uint32_t((rank * WK + wk) * kTok * rows);
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = wr * 32 + r * 16 + 8 * h + g, owner = row / rows;
      const uint32_t at = C > 1 ? cluster_addr(red_a, uint32_t(owner)) : red_a;
#pragma unroll
      for (int j = 0; j < TG; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          st_cluster(at + 4u * uint32_t((8 * j + 2 * t + e) * rows + row - owner * rows), acc[r][j][2 * h + e]);
    }
  if (C > 1) cluster_arrive(), cluster_wait();
  else __syncthreads();
  for (int e = tid; e < rows * p.m; e += kThreads) {
    const int tok = e / rows;
    const int64_t n = row0 + rank * rows + e - tok * rows;
    if (n >= p.n_out) continue;
    float s = 0.f;
    for (int w = 0; w < C * WK; ++w) s += red[w * kTok * rows + e];
    if (p.row_scale) s *= p.row_scale[n];
    if (p.y_fp32) static_cast<float*>(p.y)[int64_t(tok) * p.n_out + n] = s;
    else static_cast<__nv_bfloat16*>(p.y)[int64_t(tok) * p.n_out + n] = __float2bfloat16_rn(s);
  }
}

template <int TG, int WR>
cudaError_t launch(Params p, int C, cudaStream_t st) {
  constexpr int kTok = TG * 8, WK = kWarps / WR, kCtaRows = WR * 32;
  const int share = (p.n_kb + C - 1) / C;
  p.stage_kb = std::min(std::max(kStage / (kTok * kChan * 2) / kWarps, 1) * kWarps, (share + kWarps - 1) / kWarps * kWarps);
  const size_t smem = size_t(kWarps) * kSlots * kBlock + size_t(p.stage_kb) * kTok * (kChan * 2 + 4) +
                      size_t(WK) * kTok * kCtaRows * 4;
  auto kern = matvec_kernel<TG, WR>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kMaxSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((p.n_rb + WR - 1) / WR * C));
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


// ---- the tensor-memory form ----------------------------------------------------------------------------------
// A cluster of C CTAs (one per SM) shares the channels of a contiguous range of row blocks, which it takes in
// steps of four (128 rows).  Warps 4 .. 15, as three groups of four, take every third channel block: a lane reads its
// row's 128 channels from its warp's ring of copied blocks, and dequantises them into 64 tensor-memory columns; warps 0 .. 3 issue
// the eight MMAs of each channel block against the CTA's share of x, which was staged once in the
// 128-byte-swizzled K-major layout; warps 16 .. 19 read the accumulators of a step and exchange the C partial sums
// through distributed shared memory, while the next step is under way.
namespace tc {

constexpr int kGroups = 3;                        // dequantising groups of four warps
constexpr int kSlots = 3;                         // blocks under way per dequantising warp
constexpr int kIssuers = 4;                       // warps that issue MMAs: [half of a block][block parity]
constexpr int kThreads = (4 + 4 * kGroups + 4) * 32;
constexpr int kStep = 4;                          // row blocks per step: M = 128
// Dequantised blocks in tensor memory, columns each.  A multiple of the groups and of 2: a buffer is filled by one
// group and each of its halves used by one issuer only, so none waits for a phase of a barrier that lies two ahead.
constexpr uint32_t kABufs = 6, kACols = kChan / 2;
static_assert(kABufs % kGroups == 0 && kABufs % 2 == 0, "one filler and one user of each half per buffer");
constexpr uint32_t kDCol = kABufs * kACols;       // accumulators of N columns, one per issuer
static_assert(kChan == kPlanChan, "the plan counts the blocks of this layout");
static_assert(kDCol + kIssuers * 32 <= 512, "tensor memory");

struct Tail {
  alignas(16) unsigned char ring[4 * kGroups][kSlots][kBlock];  // per dequantising warp
  alignas(16) float red[32][128];                 // partial sums of a step: [token][row]
  uint64_t full[4 * kGroups][kSlots];
  float inv[32];                                  // per token: scale of its sums
  uint64_t a_full[kABufs], a_empty[kABufs], d_full, d_empty, red_full, red_empty;
  uint32_t tmem;
};

struct Params {
  const uint16_t* x;
  const uint8_t* packed;
  const float* row_scale;
  void* y;
  int64_t n_out, n_in;
  int m, n_kb, n_rb, y_fp32, x_bytes;
  unsigned int* flags;
};

__device__ __forceinline__ void mbar_init(uint64_t* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(b)) : "memory");
}
// the barrier at the same place of CTA `rank` of the cluster; what this CTA wrote before is visible to its waiters
__device__ __forceinline__ void mbar_arrive_cluster(uint64_t* b, uint32_t rank) {
  asm volatile("{ .reg .u32 r; mapa.shared::cluster.u32 r, %0, %1;\n\t"
               "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r]; }\n" ::"r"(smem_u32(b)),
               "r"(rank)
               : "memory");
}
// D (+)= A B with A in tensor memory
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {  // valid after tcgen05.wait::ld
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a)
      : "memory");
}
// A loaded register used behind the wait (which the compiler does not tie to the load).
__device__ __forceinline__ float tmem_value(uint32_t& r) {
  asm volatile("" : "+r"(r));
  return __uint_as_float(r);
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a, uint32_t rank) {
  float4 v;
  asm volatile("{ .reg .u32 r; mapa.shared::cluster.u32 r, %4, %5; ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r]; }\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a), "r"(rank)
               : "memory");
  return v;
}

struct Row {  // a row's share of a block, as loaded
  uint4 c[4];
  uint2 s;
};

// kTok: token rows of the MMA (N), 16 or 32.  C: CTAs of a cluster.
template <int kTok, int C>
__global__ void __launch_bounds__(kThreads, 1) matvec_tc_kernel(const Params p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  Tail& sm = *reinterpret_cast<Tail*>(smem + p.x_bytes);
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(blockIdx.x % unsigned(C));
  const int n_clusters = int(gridDim.x / unsigned(C)), cluster = int(blockIdx.x / unsigned(C));
  // even shares (the products stay below 2^32: sizes_ok)
  const int kb0 = int(uint32_t(p.n_kb) * uint32_t(rank) / uint32_t(C)),
            nk = int(uint32_t(p.n_kb) * uint32_t(rank + 1) / uint32_t(C)) - kb0;
  const int rb0 = int(uint32_t(p.n_rb) * uint32_t(cluster) / uint32_t(n_clusters)),
            rb1 = int(uint32_t(p.n_rb) * uint32_t(cluster + 1) / uint32_t(n_clusters));
  const int n_steps = (rb1 - rb0 + kStep - 1) / kStep;

  bool late = false;  // a wait ran out: flagged, and no more waiting
  auto wait = [&](uint64_t* b, uint32_t use) {  // the use-th completion of a barrier
    if (!late && !bar_wait(smem_u32(b), use & 1u)) {
      late = true;
      atomicOr(p.flags, CSA2_FLAG_TIMEOUT);
    }
  };

  if (tid == 0) {
    for (uint32_t i = 0; i < kABufs; ++i) mbar_init(&sm.a_full[i], 4), mbar_init(&sm.a_empty[i], 2);
    mbar_init(&sm.d_full, kIssuers), mbar_init(&sm.d_empty, 4);
    mbar_init(&sm.red_full, C), mbar_init(&sm.red_empty, C);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  // A dequantising warp takes row block q of each step, of the channel blocks grp, grp + kGroups, ... of the steps
  // one after the other; its first blocks are on their way while x is staged.
  const int grp = (warp - 4) >> 2, q = warp & 3;
  const int me = warp - 4;  // its ring
  int l_k = grp, l_rb = rb0 + q;  // the next block to copy: of the share's channel blocks, and its row block
  const uint8_t* l_src = p.packed + (int64_t(l_rb) * p.n_kb + kb0 + l_k) * kBlock;
  int copied = 0;
  auto copy = [&](int slot) {  // one thread; nothing where the step has no such row block
    while (l_k >= nk && l_rb < rb1) l_k -= nk, l_rb += kStep, l_src += (int64_t(kStep) * p.n_kb - nk) * kBlock;
    if (l_rb < rb1 && !late) block_copy(sm.ring[me][slot], l_src, &sm.full[me][slot]), ++copied;
    l_k += kGroups, l_src += kGroups * kBlock;
  };
  if (warp >= 4 && grp < kGroups) {
    if (lane == 0) {
      for (int i = 0; i < kSlots; ++i) mbar_init(&sm.full[me][i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
      for (int i = 0; i < kSlots; ++i) copy(i);
    }
    __syncwarp();
  }
  // x: a warp per token; groups of 64 channels, each [kTok rows][128 bytes], 16-byte pieces swizzled by the row.
  // A lane keeps the first 2048 channels of the share between the two passes, and reads what lies behind again.
  // Rows past the last token are left as they are: they reach their own columns of the sums alone.
  {
    constexpr int W = kThreads / 32, U = (kTok + W - 1) / W;  // tokens of a warp, loaded together
    const int tok0 = (warp + W - 4) % W;                      // warp 3 comes last
    const uint16_t* src = p.x + int64_t(tok0) * p.n_in;
    auto at = [&](int u, int c) -> uint4 {  // channels c .. c+7 of the share
      const int64_t ch = int64_t(kb0) * kChan + c;
      return tok0 + u * W < p.m && c < nk * kChan && ch < p.n_in
                 ? __ldg(reinterpret_cast<const uint4*>(src + u * W * p.n_in + ch))
                 : make_uint4(0, 0, 0, 0);
    };
    auto mag = [](uint32_t am, const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) am = max(am, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      return am;
    };
    uint4 keep[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) keep[u][i] = at(u, lane * 8 + 256 * i);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tok = tok0 + u * W;
      if (tok >= p.m) break;
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) am = mag(am, keep[u][i]);
      for (int c0 = 2048; c0 < nk * kChan; c0 += 1024) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = at(u, c0 + lane * 8 + 256 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) am = mag(am, v[i]);
      }
      am = __reduce_max_sync(0xffffffffu, am);
      const int up = am ? min(max(141 - int(am >> 7), -126), 126) : 0;
      const float f = __uint_as_float(uint32_t(127 + up) << 23);
      auto put = [&](int c, const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = attn::h2_bits(__floats2half2_rn(bf16lo(w[i]) * f, bf16hi(w[i]) * f));
        if (c < nk * kChan)
          *reinterpret_cast<uint4*>(smem + (c >> 6) * (kTok * 128) + tok * 128 + ((((c >> 3) & 7) ^ (tok & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) put(lane * 8 + 256 * i, keep[u][i]);
      for (int c0 = 2048; c0 < nk * kChan; c0 += 1024) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = at(u, c0 + lane * 8 + 256 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) put(c0 + lane * 8 + 256 * i, v[i]);
      }
      if (lane == 0) sm.inv[tok] = __uint_as_float(uint32_t(127 - up) << 23);
    }
  }
  attn::fence_async_smem();
  attn::tc_fence_before();
  cluster_arrive_wait();
  __syncthreads();  // all warps are past this wait before one comes to the last arrival (as in matvec_kernel)
  attn::tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < kIssuers) {
    // An issuer takes one half of every second channel block, into its own accumulator: one thread needs 54 cycles
    // and more for an MMA and as much as several for a commit, the tensor core 16 for an MMA.
    if (lane == 0) {
      const uint32_t idesc = attn::instr_desc(128, false, false, kTok), d = tmem + kDCol + uint32_t(warp) * kTok;
      const uint32_t half = uint32_t(warp) >> 1;
      const uint64_t x0 = attn::smem_desc(smem_u32(smem) + half * (kTok * 128), 0, 1024);
      uint32_t buf = uint32_t(warp) & 1u, use = 0;
      int k = warp & 1;
      for (int step = 0; step < n_steps; ++step, k -= nk) {
        if (step > 0) wait(&sm.d_empty, uint32_t(step - 1));
        for (bool first = true; k < nk; k += 2, first = false) {
          wait(&sm.a_full[buf], use);
          attn::tc_fence_after();
          const uint32_t a = tmem + buf * kACols + half * (kACols / 2);
          const uint64_t xk = x0 + uint64_t(uint32_t(2 * k) * (kTok * 128 / 16));
#pragma unroll
          for (uint32_t i = 0; i < kChan / 32; ++i) umma_ts(d, a + i * 8u, xk + uint64_t(i * 2u), idesc, !first || i > 0);
          attn::umma_commit(smem_u32(&sm.a_empty[buf]));
          buf += 2;
          if (buf >= kABufs) buf -= kABufs, ++use;
        }
        attn::umma_commit(smem_u32(&sm.d_full));
      }
    }
  } else if (warp >= 4 && grp < kGroups) {
    const uint32_t lanes = uint32_t(32 * q) << 16, n_it = uint32_t(n_steps) * uint32_t(nk);
    uint32_t buf = uint32_t(grp), use = 0;  // buffer, and how often it has been used
    int k = grp, rb = rb0 + q;
    int slot = 0, slot_use = 0;
    for (uint32_t it = uint32_t(grp); it < n_it; it += kGroups) {
      while (k >= nk) k -= nk, rb += kStep;
      Row r;
      if (rb < rb1) {
        wait(&sm.full[me][slot], uint32_t(slot_use));
        const unsigned char* blk = sm.ring[me][slot];
#pragma unroll
        for (int j = 0; j < 4; ++j) r.c[j] = *reinterpret_cast<const uint4*>(blk + block_place(lane, j));
        r.s = *reinterpret_cast<const uint2*>(blk + kCodeBytes + 8 * lane);
        attn::fence_async_smem();  // what the lanes have read comes before what the copy writes
        __syncwarp();
        if (lane == 0) copy(slot);
        if (++slot == kSlots) slot = 0, ++slot_use;
      }
      if (use > 0) wait(&sm.a_empty[buf], use - 1);
      __syncwarp();
      attn::tc_fence_after();
      if (rb < rb1) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // 64 channels, 32 columns
          const uint32_t sw = hf ? r.s.y : r.s.x;
          const __half2 s01 = attn::bits_h2(attn::e4m3x2_to_f16x2(uint16_t(sw))),
                        s23 = attn::bits_h2(attn::e4m3x2_to_f16x2(uint16_t(sw >> 16)));
          uint32_t v[32];
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const uint4 cw = r.c[2 * hf + (w >> 2)];
            uint32_t* o = v + 4 * w;
            attn::e2m1x8_to_f16x2x4((w & 3) == 0 ? cw.x : (w & 3) == 1 ? cw.y : (w & 3) == 2 ? cw.z : cw.w, o[0], o[1],
                                    o[2], o[3]);
            const __half2 sc = w < 2 ? __low2half2(s01) : w < 4 ? __high2half2(s01) : w < 6 ? __low2half2(s23)
                                                                                          : __high2half2(s23);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = attn::h2_bits(__hmul2(attn::bits_h2(o[j]), sc));
          }
          tmem_st32(tmem + lanes + buf * kACols + 32u * hf, v);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
      }
      attn::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.a_full[buf]);
      k += kGroups, buf += kGroups;
      if (buf >= kABufs) buf -= kABufs, ++use;
    }
    if (lane == 0 && late) bar_drain<kSlots>(sm.full[me], copied);
  } else if (warp >= 4) {
    const uint32_t lanes = uint32_t(32 * q) << 16;
    for (int step = 0; step < n_steps; ++step) {
      // the step's sums: this CTA's share of the channels, then the cluster's
      const int rb = rb0 + step * kStep, nb = min(kStep, rb1 - rb);
      wait(&sm.d_full, uint32_t(step));
      __syncwarp();
      attn::tc_fence_after();
      float sum[kTok];
#pragma unroll
      for (int j = 0; j < kTok; j += 16) {
        uint32_t d[kIssuers][16];
#pragma unroll
        for (int c = 0; c < kIssuers; ++c) tmem_ld16(tmem + lanes + kDCol + uint32_t(c * kTok + j), d[c]);
        asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float v = 0.f;
#pragma unroll
          for (int c = 0; c < kIssuers; ++c) v += tmem_value(d[c][i]);
          sum[j + i] = v;
        }
      }
      attn::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.d_empty);  // the next step's products may begin
      if (step > 0 && !late && !bar_wait<true>(smem_u32(&sm.red_empty), uint32_t(step - 1) & 1u)) {
        late = true;
        atomicOr(p.flags, CSA2_FLAG_TIMEOUT);
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i)
        if (i < p.m) sm.red[i][32 * q + lane] = sum[i] * sm.inv[i];
      __syncwarp();
      asm volatile("bar.sync 1, 128;\n" ::: "memory");  // warps 16 .. 19
      const int t = tid & 127;
      if (t < C) mbar_arrive_cluster(&sm.red_full, uint32_t(t));
      if (!late && !bar_wait<true>(smem_u32(&sm.red_full), uint32_t(step) & 1u)) {
        late = true;
        atomicOr(p.flags, CSA2_FLAG_TIMEOUT);
      }
      // this CTA finishes rows rank * 128 / C .. of the step, four rows of a token at a time
      constexpr int quads = 32 / C;
      for (int e = t; e < quads * p.m; e += 128) {
        const int tok = e / quads, r = (rank * quads + e - tok * quads) * 4;
        if (r >= nb * kRows) continue;
        float4 part[C];  // (all loads before the first sum: one takes several hundred cycles)
        const uint32_t at = smem_u32(&sm.red[tok][r]);
#pragma unroll
        for (int c = 0; c < C; ++c) part[c] = ld_cluster4(at, uint32_t(c));
        float4 v = part[0];
#pragma unroll
        for (int c = 1; c < C; ++c) v.x += part[c].x, v.y += part[c].y, v.z += part[c].z, v.w += part[c].w;
        const int64_t n = int64_t(rb) * kRows + r;
        const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (n + i >= p.n_out) break;
          const float s = p.row_scale ? o[i] * __ldg(p.row_scale + n + i) : o[i];
          if (p.y_fp32) static_cast<float*>(p.y)[int64_t(tok) * p.n_out + n + i] = s;
          else static_cast<__nv_bfloat16*>(p.y)[int64_t(tok) * p.n_out + n + i] = __float2bfloat16_rn(s);
        }
      }
      __syncwarp();
      asm volatile("bar.sync 1, 128;\n" ::: "memory");
      if (t < C) mbar_arrive_cluster(&sm.red_empty, uint32_t(t));
    }
  }
  __syncwarp();
  attn::tc_fence_before();
  cluster_arrive_wait();  // no CTA leaves while its sums are being read
  if (warp == 3) {
    if (lane == 0 && n_steps > 0) bar_wait(smem_u32(&sm.d_full), uint32_t(n_steps - 1) & 1u);  // (done, unless one is late)
    __syncwarp();
    attn::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
}

// Launches the tensor-memory form, for sizes that plan() gives to it.
template <int kTok, int C>
cudaError_t launch_tc(const mv::Params& g, int sms, cudaStream_t st) {
  Params p = {};
  p.x = g.x, p.packed = g.packed, p.row_scale = g.row_scale, p.y = g.y;
  p.n_out = g.n_out, p.n_in = g.n_in, p.m = g.m, p.n_kb = g.n_kb, p.n_rb = g.n_rb, p.y_fp32 = g.y_fp32;
  const int64_t x = x_bytes(g.n_kb, C, kTok);
  if (x > kXBytes || g.n_kb < 2 * C) return cudaErrorInvalidValue;  // (every issuer has a block in every step)
  p.x_bytes = int(x);
  p.flags = g.flags;
  const size_t smem = size_t(p.x_bytes) + sizeof(Tail);
  auto kern = matvec_tc_kernel<kTok, C>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kXBytes + sizeof(Tail), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
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
  cfg.numAttrs = 2;
  // clusters that run at once (one CTA per SM whatever the shared memory), looked up once per device
  static std::atomic<int> room[64];
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int clusters = dev < 64 ? room[dev].load() : 0;
  if (clusters <= 0) {
    cfg.gridDim = dim3(unsigned(C));
    cfg.dynamicSmemBytes = kXBytes + sizeof(Tail);
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1) clusters = sms / C;
    cfg.dynamicSmemBytes = smem;
    if (dev < 64) room[dev] = clusters;
  }
  cfg.gridDim = dim3(unsigned(std::min(clusters, g.n_rb) * C));
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int kTok>
cudaError_t launch_tc(const mv::Params& g, int C, int sms, cudaStream_t st) {
  return C == 4 ? launch_tc<kTok, 4>(g, sms, st) : launch_tc<kTok, 8>(g, sms, st);
}

}  // namespace tc

template <int TG>
cudaError_t launch_wr(const Params& p, int sms, cudaStream_t st) {
  // The most CTAs that run at once and have a block for every warp, of these the widest (a CTA stages x for all its
  // rows).  Measured, us, weights from HBM, at five rows x 8200 x 4112: 264 CTAs of 8 row blocks 9.3, 260 of 4 9.1, 132
  // of 8 9.0, 258 of 2 11.0, 520 of 4 13.1; at one row 8.7, 8.4, 8.2, 9.0, 12.1; at one row x 512 x 4096: 64 CTAs of 2
  // row blocks 3.7, 128 of 1 (half the warps without a block) 3.8, 32 of 2 4.3.
  int best_wr = 1, best_c = 1;
  int64_t best = 0;
  for (int wr = 8; wr >= 1; wr /= 2)
    for (int c = 1; c <= kMaxCluster && c <= p.n_kb; c *= 2) {
      const int64_t ctas = int64_t((p.n_rb + wr - 1) / wr) * c;
      // three or four groups of tokens leave room for one CTA per SM, and for 15 clusters of 8
      const int64_t room = TG <= 2 ? 2 * int64_t(sms) : c == 8 ? int64_t(sms) * 3 / 4 : int64_t(sms) * 15 / 16;
      if (ctas > best && ctas <= room && ctas * kWarps <= std::max<int64_t>(int64_t(p.n_rb) * p.n_kb, kWarps))
        best = ctas, best_wr = wr, best_c = c;
    }
  if (best == 0) best_wr = 8;  // more row blocks than run at once
  switch (best_wr) {
    case 8: return launch<TG, 8>(p, best_c, st);
    case 4: return launch<TG, 4>(p, best_c, st);
    case 2: return launch<TG, 2>(p, best_c, st);
    default: return launch<TG, 1>(p, best_c, st);
  }
}

inline bool sizes_ok(int64_t n_out, int64_t n_in) {
  return n_out >= 0 && n_in >= 0 && n_in % CSA2_GROUP == 0 && n_out <= (int64_t(1) << 28) && n_in <= (int64_t(1) << 28);
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
  const Span spans[] = {span(packed, int64_t(csa2_fp4_packed_bytes(n_out, n_in)), 1), span(codes, n_out, n_in / 2),
                        span(scales, n_out, n_in / CSA2_GROUP)};
  if (any_overlap(spans, 1, 3)) return CSA2_ERR_INVALID_ARG;
  const int64_t n_kb = (n_in + kChan - 1) / kChan, n_blocks = (n_out + kRows - 1) / kRows * n_kb;  // a warp each
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
  const Span spans[] = {span(y, m, n_out * (y_fp32 ? 4 : 2)), span(x, m, n_in * 2),
                        span(packed, int64_t(csa2_fp4_packed_bytes(n_out, n_in)), 1), span(row_scale, n_out, 4)};
  if (any_overlap(spans, 1, 4)) return CSA2_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return CSA2_ERR_CUDA;
  Params p = {};
  p.x = x, p.packed = packed, p.row_scale = row_scale, p.y = y;
  p.n_out = n_out, p.n_in = n_in, p.m = m, p.y_fp32 = y_fp32;
  p.flags = device_flags_ptr();
  if (!p.flags) return CSA2_ERR_CUDA;
  p.n_kb = int((n_in + kChan - 1) / kChan), p.n_rb = int((n_out + kRows - 1) / kRows);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const tc::Plan plan = tc::plan(m, p.n_rb, p.n_kb);
  if (plan.tok == 32) {
    e = tc::launch_tc<32>(p, plan.C, sms, st);
  } else if (plan.tok == 16) {
    for (int r = 0; r < m && e == cudaSuccess; r += 16) {
      Params q = p;
      q.m = std::min(m - r, 16), q.x = x + int64_t(r) * n_in;
      q.y = static_cast<char*>(y) + int64_t(r) * n_out * (y_fp32 ? 4 : 2);
      e = tc::launch_tc<16>(q, plan.C, sms, st);
    }
  } else {
    switch ((m + 7) / 8) {
      case 1: e = launch_wr<1>(p, sms, st); break;
      case 2: e = launch_wr<2>(p, sms, st); break;
      case 3: e = launch_wr<3>(p, sms, st); break;
      default: e = launch_wr<4>(p, sms, st); break;
    }
  }
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
