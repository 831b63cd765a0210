// Log probabilities of given tokens, log-sum-exp, entropy and the n likeliest tokens of rows of logits, in one pass.
//
// With x the logits, c = inv_temp and M their largest: s = sum exp(c (x - M)), t = sum exp(c (x - M)) c (x - M), then
// lse = c M + log s, log p(x) = c (x - M) - log s and the entropy log s - t / s, a sum of two parts that are not
// negative.  Every lane keeps its own running (M, s, t), in units of log2, and the row's are put together at the end.
//
// The likeliest tokens without a second pass.  A row is cut into groups of consecutive tokens (four 16-byte loads of
// a warp); the pass keeps each group's largest value.  Order the groups by (largest value, first group first): all n
// winners by (value, lowest token first) lie in the first n groups, since each group before a winner's own holds an
// element that beats it.  Likewise the group in place r holds at most n - r of them, as r elements beat all of it.  So
// the n groups are read again (from L2), at most n (n + 1) / 2 candidates are kept, each counts those that beat it, and
// that is its place: whole numbers throughout, whatever the number of ties.
//
// Bound: one read of the logits.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "cluster.cuh"

namespace csa2 {
namespace lp {

constexpr int kLoads = 4;             // 16-byte loads of a lane per group
constexpr int kTop = CSA2_MAX_TOP;    // 32
constexpr int kCand = kTop * (kTop + 1) / 2;
constexpr int kMaxCluster = 8;
constexpr int kParts = 64;            // of a CTA's lanes; at least kTop
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -10000.f;   // exponents are cut off here: 2^-10000 is 0, and 0 times it is 0
constexpr float kNear = 1048576.f;
constexpr float kFloor = -1e30f;      // logits are cut off here: with inv_temp in [1e-20, 1e8] its exponent is finite and 2^ it 0

struct Params {
  const void* logits;
  int64_t ld;
  int rows, V, n_tok, n_top, max_groups;
  float inv_temp;
  const int32_t* tokens;
  float *logprobs, *lse, *entropy, *top_logprobs;
  int32_t* top_ids;
  unsigned int* flags;
};

// Exponents are relative to ref = m * c2 as rounded, wherever they are added, so that its rounding drops out; far from
// zero, where that rounding is no longer small, to m itself.
struct Stat {
  float m, s, t;  // exponents in log2
};
__device__ __forceinline__ bool near(float ref) { return fabsf(ref) < kNear; }
__device__ __forceinline__ float below(float a, float m, float c2) {  // of a's reference, below m's
  return fmaxf(near(m * c2) ? __fsub_rn(__fmul_rn(a, c2), __fmul_rn(m, c2)) : (a - m) * c2, kLowest);
}
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c2) {
  const float m = fmaxf(a.m, b.m);
  Stat r = {m, 0.f, 0.f};
  // (a part whose m is -inf is empty)
  if (a.m > -INFINITY) {
    const float d = below(a.m, m, c2), f = attn::ex2(d);
    r.s = a.s * f, r.t = (a.t + a.s * d) * f;
  }
  if (b.m > -INFINITY) {
    const float d = below(b.m, m, c2), f = attn::ex2(d);
    r.s += b.s * f, r.t += (b.t + b.s * d) * f;
  }
  return r;
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <bool kBf16>
struct Row {
  static constexpr int E = kBf16 ? 8 : 4;         // tokens of a 16-byte load
  static constexpr int kGroup = kLoads * 32 * E;  // tokens of a group
  const unsigned char* at;  // the row, back to a 16-byte boundary
  int shift, V;             // tokens before the row there
  __device__ __forceinline__ Row(const Params& p, int r) {
    const unsigned char* row = static_cast<const unsigned char*>(p.logits) + int64_t(r) * p.ld * (kBf16 ? 2 : 4);
    const int off = int(reinterpret_cast<uintptr_t>(row) & 15u);
    at = row - off, shift = off / (kBf16 ? 2 : 4), V = p.V;
  }
  __device__ __forceinline__ int groups() const { return (V + shift + kGroup - 1) / kGroup; }
  __device__ __forceinline__ float one(int i) const {
    if (kBf16) return bf16f(reinterpret_cast<const uint16_t*>(at)[shift + i]);
    return reinterpret_cast<const float*>(at)[shift + i];
  }
  // the first token of load j of group g for a lane
  __device__ __forceinline__ int first(int g, int j, int lane) const { return g * kGroup + (j * 32 + lane) * E - shift; }
  // the values at tokens i .. i + E - 1, -inf outside of the row
  __device__ __forceinline__ void load(int i, uint4& v) const {
    if (i >= 0 && i + E <= V) {
      v = __ldg(reinterpret_cast<const uint4*>(at + int64_t(i + shift) * (kBf16 ? 2 : 4)));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (kBf16) {
          const int a = i + 2 * e;
          const uint16_t* q = reinterpret_cast<const uint16_t*>(at) + shift;
          const uint32_t lo = a >= 0 && a < V ? q[a] : 0xFF80u, hi = a + 1 >= 0 && a + 1 < V ? q[a + 1] : 0xFF80u;
          w[e] = lo | hi << 16;
        } else {
          w[e] = i + e >= 0 && i + e < V ? reinterpret_cast<const uint32_t*>(at)[shift + i + e] : 0xFF800000u;
        }
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  static __device__ __forceinline__ float value(const uint4& v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (kBf16) return (e & 1) ? bf16hi(w[e >> 1]) : bf16lo(w[e >> 1]);
    return __uint_as_float(w[e]);
  }
};

// Two fp32 values at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The largest of a lane's values of a group; bf16 two at a time.
template <bool kBf16>
__device__ __forceinline__ float group_max(const uint4 (&v)[kLoads]) {
  if (kBf16) {
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&v[0].x);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[e]));
    }
    return fmaxf(__low2float(m), __high2float(m));
  }
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
    m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(v[j].x), __uint_as_float(v[j].y))),
              fmaxf(__uint_as_float(v[j].z), __uint_as_float(v[j].w)));
  return m;
}

// Adds a lane's values of a group to its sums.
template <bool kBf16>
__device__ __forceinline__ void add_group(const uint4 (&v)[kLoads], float top, float c2, Stat& st) {
  if (top > st.m) {
    const float d = below(st.m, top, c2), f = attn::ex2(d);
    st.t = (st.t + st.s * d) * f, st.s *= f, st.m = top;
  }
  if (!(st.m > -INFINITY)) return;
  const float ref = __fmul_rn(st.m, c2);
  if (near(ref)) {
    // one rounding per exponent; what lies below kFloor (-inf among it) weighs nothing
    const uint64_t cc = pair(c2, c2), mm = pair(-ref, -ref);
    uint64_t s = pair(st.s, 0.f), t = pair(st.t, 0.f);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int e = 0; e < (kBf16 ? 4 : 2); ++e) {
        uint64_t x;
        if (kBf16) {
          const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), __float2bfloat162_rn(kFloor));
          const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
          x = pair(bf16lo(u), bf16hi(u));
        } else {
          x = pair(fmaxf(__uint_as_float(w[2 * e]), kFloor), fmaxf(__uint_as_float(w[2 * e + 1]), kFloor));
        }
        const uint64_t d = fma2(x, cc, mm);
        float d0, d1;
        unpair(d, d0, d1);
        const uint64_t p = pair(attn::ex2(d0), attn::ex2(d1));
        s = add2(s, p);
        t = fma2(p, d, t);
      }
    }
    float a, b;
    unpair(s, a, b), st.s = a + b;
    unpair(t, a, b), st.t = a + b;
  } else {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int e = 0; e < Row<kBf16>::E; ++e) {
        const float d = fmaxf((Row<kBf16>::value(v[j], e) - st.m) * c2, kLowest), x = attn::ex2(d);
        st.s += x;
        st.t = fmaf(x, d, st.t);
      }
  }
}

template <bool kBf16, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : kThreads == 256 ? 4 : 8) logprobs_kernel(const Params p, int C) {
  constexpr int kWarps = kThreads / 32;
  using R = Row<kBf16>;
  extern __shared__ float gmax[];  // the groups' largest values; behind them the numbers of those that are looked at
  int* group = reinterpret_cast<int*>(gmax + p.max_groups);
  __shared__ Stat part[kWarps];
  __shared__ Stat whole[kMaxCluster];
  __shared__ int sel[kTop];
  __shared__ float cv[kCand];
  __shared__ int ci[kCand];
  __shared__ int n_cand, n_group;
  __shared__ __align__(16) float pmax[kParts];  // the largest values of parts of a warp's lanes
  __shared__ float bound;
  __shared__ float lv[kMaxCluster * kTop];  // the CTAs' winners, at the cluster's first CTA
  __shared__ int li[kMaxCluster * kTop];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.n_top;
  if (n) {
    for (int i = tid; i < kMaxCluster * kTop; i += kThreads) li[i] = -1;
    if (tid < kTop) sel[tid] = -1;
    if (tid == 0) n_cand = n_group = 0;
  }
  if (C > 1) cluster_arrive();
  const int rank = C > 1 ? int(blockIdx.x % unsigned(C)) : 0;
  const int r = int(blockIdx.x / unsigned(C));
  const R row(p, r);
  const int ng = row.groups(), g0 = ng * rank / C, g1 = ng * (rank + 1) / C;
  const float c2 = p.inv_temp * kLog2e;

  Stat st = {-INFINITY, 0.f, 0.f};
  {
    uint4 v[kLoads], next[kLoads];
    if (g0 + warp < g1) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) row.load(row.first(g0 + warp, j, lane), next[j]);
    }
    for (int g = g0 + warp; g < g1; g += kWarps) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = next[j];
      if (g + kWarps < g1) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) row.load(row.first(g + kWarps, j, lane), next[j]);
      }
      const float top = group_max<kBf16>(v);
      if (n) {
        const float m = warp_max(top);
        if (lane == 0) gmax[g - g0] = m;
      }
      add_group<kBf16>(v, top, c2, st);
    }
  }
  if (n) {
    float v = st.m;
#pragma unroll
    for (int o = 1; o < kThreads / kParts; o *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tid % (kThreads / kParts) == 0) pmax[tid / (kThreads / kParts)] = v;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const Stat b = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                    __shfl_xor_sync(0xffffffffu, st.t, o)};
    st = join(st, b, c2);
  }
  if (lane == 0) part[warp] = st;
  if (C > 1) cluster_wait();  // the cluster's CTAs have all started
  __syncthreads();
  if (tid == 0) {
    Stat a = part[0];
    for (int w = 1; w < kWarps; ++w) a = join(a, part[w], c2);
    const uint32_t to = C > 1 ? cluster_addr(smem_u32(&whole[rank]), 0) : smem_u32(&whole[0]);
    st_cluster(to, a.m), st_cluster(to + 4, a.s), st_cluster(to + 8, a.t);
  }

  if (n) {
    // n values reach the n-th largest of the parts' largest ones: nothing below it is among the n, and no group whose
    // largest value is below it is looked at
    if (tid < kParts) {
      const float v = pmax[tid];
      int place = 0;
#pragma unroll
      for (int j = 0; j < kParts; j += 4) {
        const float4 u = *reinterpret_cast<const float4*>(pmax + j);
        place += (u.x > v || (u.x == v && j < tid)) + (u.y > v || (u.y == v && j + 1 < tid)) +
                 (u.z > v || (u.z == v && j + 2 < tid)) + (u.w > v || (u.w == v && j + 3 < tid));
      }
      if (place == n - 1) bound = v;
    }
    __syncthreads();
    const float low = bound;
    for (int i = tid; i < g1 - g0; i += kThreads)
      if (gmax[i] >= low) group[atomicAdd(&n_group, 1)] = i;  // (in any order)
    __syncthreads();
    const int G = n_group;
    for (int i = tid; i < G; i += kThreads) {
      const int at = group[i];
      const float v = gmax[at];
      int place = 0;
#pragma unroll 4
      for (int j = 0; j < G; ++j) {
        const int o = group[j];
        const float u = gmax[o];
        place += u > v || (u == v && o < at);
      }
      if (place < n) sel[place] = at;
    }
    __syncthreads();
    for (int place = warp; place < min(n, G); place += kWarps) {
      const int g = g0 + sel[place];
      uint4 v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) row.load(row.first(g, j, lane), v[j]);
      uint32_t left = 0;  // this lane's values that reach the bound and are not taken yet
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int i = row.first(g, j, lane);
#pragma unroll
        for (int e = 0; e < R::E; ++e)
          if (i + e >= 0 && i + e < p.V && R::value(v[j], e) >= low) left |= 1u << (j * R::E + e);
      }
      const int most = n - place;
      const int mine = __popc(left), all = int(__reduce_add_sync(0xffffffffu, unsigned(mine)));
      if (all <= most) {  // (the candidates' order does not matter)
        int at = 0;
        if (mine) at = atomicAdd(&n_cand, mine);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
          for (int e = 0; e < R::E; ++e)
            if (left >> (j * R::E + e) & 1u) cv[at] = R::value(v[j], e), ci[at] = row.first(g, j, lane) + e, ++at;
      } else {  // ties: the best of the group, one after the other
        for (int k = 0; k < most; ++k) {
          float best = -INFINITY;
          int where = -1;
#pragma unroll
          for (int j = 0; j < kLoads; ++j)
#pragma unroll
            for (int e = 0; e < R::E; ++e) {
              const float x = R::value(v[j], e);
              if ((left >> (j * R::E + e) & 1u) && (where < 0 || x > best)) best = x, where = j * R::E + e;
            }
          const float m = warp_max(best);
          const int id = where >= 0 && best == m ? row.first(g, where / R::E, lane) + where % R::E : 0x7FFFFFFF;
          const int first = int(__reduce_min_sync(0xffffffffu, unsigned(id)));
          if (id == first) {  // (some lane has one: fewer are taken than there are)
            const int at = atomicAdd(&n_cand, 1);
            cv[at] = m, ci[at] = id, left &= ~(1u << where);
          }
          __syncwarp();
        }
      }
    }
    __syncthreads();
    // the winners' places; into the list of the cluster's first CTA
    const int total = n_cand;
    const uint32_t to_v = C > 1 ? cluster_addr(smem_u32(&lv[rank * kTop]), 0) : smem_u32(&lv[0]);
    const uint32_t to_i = C > 1 ? cluster_addr(smem_u32(&li[rank * kTop]), 0) : smem_u32(&li[0]);
    for (int i = tid; i < total; i += kThreads) {
      const int id = ci[i];
      const float v = cv[i];
      int place = 0;
#pragma unroll 4
      for (int j = 0; j < total; ++j) {
        const float u = cv[j];
        place += u > v || (u == v && ci[j] < id);
      }
      if (place < n) st_cluster(to_v + 4u * place, v), st_cluster_u32(to_i + 4u * place, uint32_t(id));
    }
  }
  if (C > 1) cluster_arrive(), cluster_wait();
  else __syncthreads();
  if (rank != 0) return;

  Stat a = whole[0];
  for (int i = 1; i < C; ++i) a = join(a, whole[i], c2);
  const bool empty = !(a.m > -INFINITY);
  const float log_s = logf(a.s), ref = __fmul_rn(a.m, c2);
  auto logprob = [&](float x) {
    if (x == -INFINITY || empty) return -INFINITY;
    const float d = fmaf(x, c2, -ref);  // (-inf where the product with log2 e alone passes the type's end)
    return near(ref) && d > -INFINITY ? fmaf(d, attn::kLn2, -log_s) : (x - a.m) * p.inv_temp - log_s;
  };
  if (tid == 0) {
    if (p.lse) p.lse[r] = empty ? -INFINITY : near(ref) ? fmaf(ref, attn::kLn2, log_s) : fmaf(a.m, p.inv_temp, log_s);
    if (p.entropy) p.entropy[r] = empty ? 0.f : log_s - a.t / a.s * attn::kLn2;
  }
  for (int i = tid; i < p.n_tok; i += kThreads) {
    const int tok = p.tokens[int64_t(r) * p.n_tok + i];
    float v = 0.f;
    if (tok >= p.V) v = -INFINITY, atomicOr(p.flags, CSA2_FLAG_INDEX_OOB);
    else if (tok >= 0) v = logprob(row.one(tok));
    p.logprobs[int64_t(r) * p.n_tok + i] = v;
  }
  if (n) {
    int32_t* ids = p.top_ids ? p.top_ids + int64_t(r) * n : nullptr;
    float* vals = p.top_logprobs ? p.top_logprobs + int64_t(r) * n : nullptr;
    for (int e = tid; e < C * n; e += kThreads) {
      const int at = e / n * kTop + e % n, id = li[at];
      if (id < 0) continue;
      const float v = lv[at];
      int place = 0;
#pragma unroll 4
      for (int o = 0; o < C * n; ++o) {
        const int i = o / n * kTop + o % n;
        const float u = lv[i];
        place += li[i] >= 0 && (u > v || (u == v && li[i] < id));
      }
      if (place >= n) continue;
      if (ids) ids[place] = id;
      if (vals) vals[place] = logprob(v);
    }
    for (int i = min(n, p.V) + tid; i < n; i += kThreads) {  // fewer tokens than that
      if (ids) ids[i] = -1;
      if (vals) vals[i] = -INFINITY;
    }
  }
}

template <bool kBf16, int kThreads>
cudaError_t launch(Params p, int C, cudaStream_t st) {
  p.max_groups = ((p.V + 15) / Row<kBf16>::kGroup + 2 + C - 1) / C + 1;  // groups of a CTA, whatever the alignment
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.rows) * unsigned(C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.n_top ? size_t(p.max_groups) * 8 : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<kBf16, kThreads>, p, C);
}

}  // namespace lp
}  // namespace csa2

extern "C" csa2_status csa2_token_logprobs(const void* logits, int logits_fp32, int rows, int V, int64_t ld,
                                           const int32_t* tokens, int n_tok, float inv_temp, float* logprobs, float* lse,
                                           float* entropy, int n_top, int32_t* top_ids, float* top_logprobs,
                                           csa2_stream_t stream) {
  using namespace csa2;
  using namespace csa2::lp;
  if (rows < 0 || rows > (1 << 24) || V < 1 || V > CSA2_MAX_VOCAB || ld < V || n_tok < 0 || n_tok > CSA2_MAX_TREE ||
      n_top < 0 || n_top > kTop || !(inv_temp >= 1e-20f && inv_temp <= 1e8f))
    return CSA2_ERR_INVALID_ARG;
  if (rows == 0) return CSA2_OK;
  const int es = logits_fp32 ? 4 : 2;
  if (!logits || !al(logits, uintptr_t(es)) || (n_tok && (!tokens || !logprobs)) || (n_top && !top_ids && !top_logprobs) ||
      !al(tokens, 4) || !al(logprobs, 4) || !al(lse, 4) || !al(entropy, 4) || !al(top_ids, 4) || !al(top_logprobs, 4))
    return CSA2_ERR_INVALID_ARG;
  const Span spans[] = {span(n_tok ? logprobs : nullptr, rows, 4ll * n_tok), span(lse, rows, 4), span(entropy, rows, 4),
                        span(n_top ? top_ids : nullptr, rows, 4ll * n_top), span(n_top ? top_logprobs : nullptr, rows, 4ll * n_top),
                        span(n_tok ? tokens : nullptr, rows, 4ll * n_tok),
                        span(logits, 1, (int64_t(rows - 1) * ld + V) * es)};
  if (ld > (int64_t(1) << 40) || any_overlap(spans, 5, 7)) return CSA2_ERR_INVALID_ARG;
  Params p = {};
  p.logits = logits, p.ld = ld, p.rows = rows, p.V = V, p.n_tok = n_tok, p.n_top = n_top, p.inv_temp = inv_temp;
  p.tokens = tokens, p.logprobs = logprobs, p.lse = lse, p.entropy = entropy, p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.flags = device_flags_ptr();
  const int sms = sm_count();
  if (!p.flags || sms <= 0) return CSA2_ERR_CUDA;
  const int groups = V / (logits_fp32 ? Row<false>::kGroup : Row<true>::kGroup) + 1;
  int C = 1;
  while (C < kMaxCluster && int64_t(rows) * C * 2 <= 2 * sms && groups >= 16 * C) C *= 2;
  const int threads = groups <= 16 ? 128 : C > 1 ? 512 : 256;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_fp32 ? (threads == 128 ? launch<false, 128>(p, C, st) : threads == 256 ? launch<false, 256>(p, C, st)
                                                                                             : launch<false, 512>(p, C, st))
                                    : (threads == 128 ? launch<true, 128>(p, C, st) : threads == 256 ? launch<true, 256>(p, C, st)
                                                                                           : launch<true, 512>(p, C, st));
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
