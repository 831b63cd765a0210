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
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -10000.f;   // exponents are cut off here: 2^-10000 is 0, and 0 times it is 0

struct Params {
  const void* logits;
  int64_t ld;
  int rows, V, n_tok, n_top;
  float inv_temp;
  const int32_t* tokens;
  float *logprobs, *lse, *entropy, *top_logprobs;
  int32_t* top_ids;
  unsigned int* flags;
};

struct Stat {  // exponents in log2, relative to m
  float m, s, t;
};
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c2) {
  const float m = fmaxf(a.m, b.m);
  Stat r = {m, 0.f, 0.f};
  // (a part whose m is -inf is empty)
  if (a.m > -INFINITY) {
    const float d = fmaxf((a.m - m) * c2, kLowest), f = attn::ex2(d);
    r.s = a.s * f, r.t = (a.t + a.s * d) * f;
  }
  if (b.m > -INFINITY) {
    const float d = fmaxf((b.m - m) * c2, kLowest), f = attn::ex2(d);
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

template <bool kBf16, int kThreads>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const Params p, int C) {
  constexpr int kWarps = kThreads / 32;
  using R = Row<kBf16>;
  extern __shared__ float gmax[];  // the groups' largest values
  __shared__ Stat part[kWarps];
  __shared__ Stat whole[kMaxCluster];
  __shared__ int sel[kTop];
  __shared__ float cv[kCand];
  __shared__ int ci[kCand];
  __shared__ float lv[kMaxCluster * kTop];  // the CTAs' winners, at the cluster's first CTA
  __shared__ int li[kMaxCluster * kTop];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (C > 1) cluster_arrive();
  const int rank = C > 1 ? int(blockIdx.x % unsigned(C)) : 0;
  const int r = int(blockIdx.x / unsigned(C));
  const R row(p, r);
  const int ng = row.groups(), g0 = ng * rank / C, g1 = ng * (rank + 1) / C;
  const float c2 = p.inv_temp * kLog2e;
  const int n = p.n_top;

  Stat st = {-INFINITY, 0.f, 0.f};
  for (int g = g0 + warp; g < g1; g += kWarps) {
    uint4 v[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) row.load(row.first(g, j, lane), v[j]);
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int e = 0; e < R::E; ++e) top = fmaxf(top, R::value(v[j], e));
    if (n) {
      const float m = warp_max(top);
      if (lane == 0) gmax[g - g0] = m;
    }
    if (top > st.m) {
      const float d = fmaxf((st.m - top) * c2, kLowest), f = attn::ex2(d);
      st.t = (st.t + st.s * d) * f, st.s *= f, st.m = top;
    }
    if (st.m > -INFINITY) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
          const float d = fmaxf((R::value(v[j], e) - st.m) * c2, kLowest), x = attn::ex2(d);
          st.s += x;
          st.t = fmaf(x, d, st.t);
        }
    }
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
    const int G = g1 - g0;
    for (int i = tid; i < n; i += kThreads) sel[i] = -1;
    for (int i = tid; i < kCand; i += kThreads) ci[i] = -1;
    __syncthreads();
    for (int i = tid; i < G; i += kThreads) {
      const float v = gmax[i];
      int place = 0;
      for (int j = 0; j < G; ++j) {
        const float u = gmax[j];
        place += u > v || (u == v && j < i);
      }
      if (place < n) sel[place] = i;
    }
    __syncthreads();
    // what is below the n-th group's largest value is not among the n
    const float bound = G >= n ? gmax[sel[n - 1]] : -INFINITY;
    for (int place = warp; place < min(n, G); place += kWarps) {
      const int g = g0 + sel[place], slots = place * n - place * (place - 1) / 2;
      uint4 v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) row.load(row.first(g, j, lane), v[j]);
      uint32_t gone = 0;  // of this lane's values: taken, or outside of the row
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
          const int i = row.first(g, j, lane) + e;
          if (i < 0 || i >= p.V) gone |= 1u << (j * R::E + e);
        }
      float best;
      int where;
      auto find = [&]() {  // the largest value left, the lowest token first
        best = -INFINITY, where = -1;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
          for (int e = 0; e < R::E; ++e) {
            const float x = R::value(v[j], e);
            if (!(gone >> (j * R::E + e) & 1u) && (where < 0 || x > best)) best = x, where = j * R::E + e;
          }
      };
      find();
      for (int k = 0; k < n - place; ++k) {
        const float m = warp_max(best);
        const int mine = where >= 0 && best == m ? row.first(g, where / R::E, lane) + where % R::E : 0x7FFFFFFF;
        const int id = int(__reduce_min_sync(0xffffffffu, unsigned(mine)));
        if (id == 0x7FFFFFFF || m < bound) break;
        if (lane == 0) cv[slots + k] = m, ci[slots + k] = id;
        if (mine == id) gone |= 1u << where, find();
        __syncwarp();
      }
    }
    __syncthreads();
    // the winners' places; into the list of the cluster's first CTA
    const int total = min(n, G) * n - min(n, G) * (min(n, G) - 1) / 2;
    const uint32_t to_v = C > 1 ? cluster_addr(smem_u32(&lv[rank * kTop]), 0) : smem_u32(&lv[0]);
    const uint32_t to_i = C > 1 ? cluster_addr(smem_u32(&li[rank * kTop]), 0) : smem_u32(&li[0]);
    int left = 0;  // candidates, counted alike by every thread
    for (int i = 0; i < total; ++i) left += ci[i] >= 0;
    for (int i = tid; i < total; i += kThreads) {
      const int id = ci[i];
      if (id < 0) continue;
      const float v = cv[i];
      int place = 0;
      for (int j = 0; j < total; ++j) {
        const float u = cv[j];
        place += ci[j] >= 0 && (u > v || (u == v && ci[j] < id));
      }
      if (place < n) st_cluster(to_v + 4u * place, v), st_cluster_u32(to_i + 4u * place, uint32_t(id));
    }
    for (int i = left + tid; i < n; i += kThreads) st_cluster_u32(to_i + 4u * i, 0xFFFFFFFFu);
  }
  if (C > 1) cluster_arrive(), cluster_wait();
  else __syncthreads();
  if (rank != 0) return;

  Stat a = whole[0];
  for (int i = 1; i < C; ++i) a = join(a, whole[i], c2);
  const bool empty = !(a.m > -INFINITY);
  const float log_s = logf(a.s);
  auto logprob = [&](float x) { return x == -INFINITY || empty ? -INFINITY : (x - a.m) * p.inv_temp - log_s; };
  if (tid == 0) {
    if (p.lse) p.lse[r] = empty ? -INFINITY : fmaf(a.m, p.inv_temp, log_s);
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
    int have = 0;
    for (int c = 0; c < C; ++c)
      for (int i = 0; i < n; ++i) have += li[c * kTop + i] >= 0;
    for (int e = tid; e < C * n; e += kThreads) {
      const int at = e / n * kTop + e % n, id = li[at];
      if (id < 0) continue;
      const float v = lv[at];
      int place = e % n;
      for (int c = 0; c < C; ++c)
        if (c != e / n)
          for (int j = 0; j < n; ++j) {
            const int o = li[c * kTop + j];
            const float u = lv[c * kTop + j];
            if (o < 0 || !(u > v || (u == v && o < id))) break;  // (each list is in order)
            ++place;
          }
      if (place >= n) continue;
      if (ids) ids[place] = id;
      if (vals) vals[place] = logprob(v);
    }
    for (int i = have + tid; i < n; i += kThreads) {
      if (ids) ids[i] = -1;
      if (vals) vals[i] = -INFINITY;
    }
  }
}

template <bool kBf16, int kThreads>
cudaError_t launch(const Params& p, int C, cudaStream_t st) {
  const int most = ((p.V + 15) / Row<kBf16>::kGroup + 2 + C - 1) / C + 1;  // groups of a CTA, whatever the alignment
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.rows) * unsigned(C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.n_top ? size_t(most) * 4 : 0;
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
      n_top < 0 || n_top > kTop || !(inv_temp > 0.f) || inv_temp > 1e30f)
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
  const bool small = groups <= 16;
  int C = 1;
  while (!small && C < kMaxCluster && int64_t(rows) * C * 2 <= 2 * sms && groups >= 32 * C) C *= 2;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_fp32 ? (small ? launch<false, 128>(p, C, st) : launch<false, 512>(p, C, st))
                                    : (small ? launch<true, 128>(p, C, st) : launch<true, 512>(p, C, st));
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
