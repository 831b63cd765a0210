// Pages of a shared cache pool: block tables and slot maps built on the GPU from request lengths, and the
// slot lists of what a drafted node may attend.  Integer work bound by launch latency for a decode step and
// by the slots written for an admission or a long context.
//
// csa2_block_tables, one launch: sequence b asks for max(want - held, 0) pages and gives back
// max(held - want, 0).  Both counts are summed over the sequences by every CTA for itself (two words per
// sequence), after which the owner of the j-th page asked for, and the page it gets, follow from a search in
// the sums: pages are handed out from the list's end and from those given back, never from what the same
// launch writes (list entries at or past n_free, table entries of pages newly held).  So CTAs share
// nothing but the count of free pages, which the last of them to finish updates.
#include <algorithm>

#include "common.cuh"

namespace csa2 {
namespace pages {

constexpr int kThreads = 1024;

__device__ __forceinline__ int pages_of(int len, int shift) {  // ceil(len / page), len up to 2^31 - 1
  return (len >> shift) + ((len & ((1 << shift) - 1)) != 0);
}
// first b in [0, n) with incl[b] > v (incl ascending, incl[n - 1] > v)
__device__ __forceinline__ int owner(const int* incl, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > v) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
__device__ __forceinline__ int slot_of(int page, int off, int shift) {  // -1: no such slot
  return page >= 0 && page <= (0x7FFFFFFF >> shift) ? (page << shift) + off : -1;
}

__global__ void __launch_bounds__(kThreads) block_tables_kernel(
    const int32_t* __restrict__ old_lens, const int32_t* __restrict__ new_lens, int B, int shift,
    int32_t* block_table, int max_pages, int32_t* free_pages, int free_cap, int32_t* pool_state, int32_t* granted,
    int32_t* __restrict__ slots, int n_new, bool vec, unsigned int* flags) {
  extern __shared__ int sums[];  // inclusive sums of the pages asked for, then of those given back
  __shared__ unsigned long long warp_sum[2][kThreads / 32];
  int* ask = sums;
  int* back = sums + B;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t gtid = int64_t(blockIdx.x) * kThreads + tid, gthreads = int64_t(gridDim.x) * kThreads;
  const int n_free = min(max(pool_state[0], 0), free_cap);
  const int64_t room = int64_t(max_pages) << shift;
  auto old_of = [&](int b) { return int(min(int64_t(max(old_lens[b], 0)), room)); };
  auto new_of = [&](int b) { return max(new_lens[b], 0); };

  // both sums at once, in the halves of 64 bits (each stays below 2^31: B * max_pages does)
  const int lane = tid & 31, warp = tid >> 5;
  unsigned long long base = 0;
  for (int c = 0, round = 0; c < B; c += kThreads, round ^= 1) {
    const int b = c + tid;
    unsigned long long v = 0;
    if (b < B) {
      const int held = pages_of(old_of(b), shift), want = pages_of(new_of(b), shift);
      if (want > held && want <= max_pages) v = uint32_t(want - held);
      if (want < held) v = static_cast<unsigned long long>(held - want) << 32;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[round][warp] = v;
    __syncthreads();
    // every warp adds up the warps' sums for itself
    unsigned long long w = warp_sum[round][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    const unsigned long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    v += base + (warp > 0 ? before : 0);
    if (b < B) ask[b] = int(uint32_t(v)), back[b] = int(uint32_t(v >> 32));
    base += __shfl_sync(0xffffffffu, w, 31);
  }
  const uint32_t ask0 = uint32_t(base), back0 = uint32_t(base >> 32);
  __syncthreads();
  const int F = int(back0);
  const int64_t budget = int64_t(n_free) + F;
  // sequences ask in order, so the granted pages are a prefix of those asked for
  int A = 0;
  if (int64_t(ask0) <= budget) A = int(ask0);
  else {
    int lo = 0, hi = B - 1;  // first sequence whose sum passes the budget
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (int64_t(ask[mid]) > budget) hi = mid;
      else lo = mid + 1;
    }
    A = lo > 0 ? ask[lo - 1] : 0;
  }
  auto given_back = [&](int f) {  // the f-th page given back
    const int b = owner(back, B, f), first = b > 0 ? back[b - 1] : 0;
    return block_table[int64_t(b) * max_pages + pages_of(new_of(b), shift) + (f - first)];
  };
  auto handed_out = [&](int j) { return j < F ? given_back(j) : free_pages[n_free - 1 - (j - F)]; };
  auto is_granted = [&](int b) {
    const int want = pages_of(new_of(b), shift), held = pages_of(old_of(b), shift);
    return want <= held || (want <= max_pages && ask[b] <= A);
  };

  for (int64_t b = gtid; b < B; b += gthreads) {
    const bool ok = is_granted(int(b));
    granted[b] = ok ? new_of(int(b)) : old_of(int(b));
    if (!ok) atomicOr(flags, CSA2_FLAG_PAGES_OUT);
  }
  // pages handed out, and pages put back: four at a time, so that their loads overlap
  for (int64_t j0 = gtid; j0 < A; j0 += 4 * gthreads) {
    int64_t to[4];
    int32_t page[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t j = j0 + i * gthreads;
      to[i] = -1;
      if (j >= A) continue;
      const int b = owner(ask, B, int(j)), first = b > 0 ? ask[b - 1] : 0;
      to[i] = int64_t(b) * max_pages + pages_of(old_of(b), shift) + (j - first);
      page[i] = handed_out(int(j));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (to[i] >= 0) block_table[to[i]] = page[i];
  }
  for (int64_t f0 = A + gtid; f0 < F; f0 += 4 * gthreads) {
    int32_t page[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) page[i] = f0 + i * gthreads < F ? given_back(int(f0 + i * gthreads)) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t f = f0 + i * gthreads, at = int64_t(n_free) + F - 1 - f;
      if (f >= F) continue;
      if (at < free_cap) free_pages[at] = page[i];
      else atomicOr(flags, CSA2_FLAG_INDEX_OOB);  // no room in the list: the page is lost
    }
  }
  // four columns a thread: most of them lie in one page, whose number is looked up once
  const int quads = n_new / 4 + (n_new % 4 != 0);  // (n_new goes up to 2^31 - 1)
  for (int64_t i = gtid; i < int64_t(B) * quads; i += gthreads) {
    const int b = int(uint32_t(i) / uint32_t(quads)), c = (int(i) - b * quads) * 4;
    const int o = old_of(b), end = is_granted(b) ? new_of(b) : o, held = pages_of(o, shift);
    const int first = b > 0 ? ask[b - 1] : 0;
    int s[4], pg = -1, page = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = -1;
      if (c + j >= end - o) continue;
      const int pos = o + c + j;
      if ((pos >> shift) != pg) {
        pg = pos >> shift;
        page = pg < held ? block_table[int64_t(b) * max_pages + pg] : handed_out(first + pg - held);
      }
      s[j] = slot_of(page, pos & ((1 << shift) - 1), shift);
      if (s[j] < 0) atomicOr(flags, CSA2_FLAG_INDEX_OOB);
    }
    int32_t* dst = slots + int64_t(b) * n_new + c;
    if (vec) {
      *reinterpret_cast<int4*>(dst) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < n_new) dst[j] = s[j];
    }
  }

  // the last CTA to get here has seen every other read the old count
  __syncthreads();
  if (tid == 0) {
    const unsigned int done = gridDim.x > 1 ? atomicAdd(reinterpret_cast<unsigned int*>(pool_state + 1), 1u) : 0u;
    if (done == gridDim.x - 1) {
      pool_state[0] = int(min(budget - A, int64_t(free_cap)));
      pool_state[1] = 0;
    }
  }
}

constexpr int kCtxThreads = 256;

// A thread lists four columns for every node of its sequence: up to the committed length a column is the
// same slot for all of them, so the block table is read once per page and thread.  kVec: rows are stored as
// 16-byte pieces (ld a multiple of 4).
template <bool kVec>
__global__ void __launch_bounds__(kCtxThreads) context_slots_kernel(
    const int32_t* __restrict__ lens, const int32_t* __restrict__ parent, const int32_t* __restrict__ n_nodes, int N,
    const int32_t* __restrict__ block_table, int max_pages, int shift, int32_t* __restrict__ slots, int64_t ld,
    int32_t* __restrict__ n_slots, unsigned int* flags) {
  __shared__ unsigned long long anc[CSA2_MAX_TREE];
  __shared__ int par[CSA2_MAX_TREE];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t c0 = (int64_t(blockIdx.x) * kCtxThreads + tid) * 4;
  // everything that depends on the place alone is asked for at once
  const int32_t* table = block_table ? block_table + int64_t(b) * max_pages : nullptr;
  const int page0 = table && (c0 >> shift) < max_pages ? table[c0 >> shift] : -1;
  const int up0 = parent && tid < N ? parent[int64_t(b) * N + tid] : -1;
  const int nn = n_nodes ? min(max(n_nodes[b], 0), N) : N;
  const int len = max(lens[b], 0);
  const int64_t cta0 = int64_t(blockIdx.x) * kCtxThreads * 4;
  // the CTAs that hold drafted rows (and the first, which counts them) walk the tree
  if (blockIdx.x == 0 || (cta0 + kCtxThreads * 4 > len && cta0 < int64_t(len) + CSA2_MAX_TREE)) {
    if (tid < N) par[tid] = up0;
    __syncthreads();
    if (tid < N) {
      unsigned long long m = 0;
      bool bad = false;
      if (parent && tid < nn)
        for (int cur = tid; cur >= 0;) {
          m |= 1ull << cur;
          const int up = par[cur];
          if (up < -1 || up >= cur) {
            bad = true;
            break;
          }
          cur = up;
        }
      anc[tid] = m;
      if (blockIdx.x == 0) {
        const int64_t n = tid < nn ? int64_t(len) + __popcll(m) : 0;
        n_slots[int64_t(b) * N + tid] = int32_t(min(n, ld));
        if (bad || n > ld) atomicOr(flags, CSA2_FLAG_INDEX_OOB);
      }
    }
    __syncthreads();
  }
  auto slot = [&](int64_t pos) -> int {
    if (!table) return pos <= 0x7FFFFFFF ? int(pos) : -1;
    const int64_t pg = pos >> shift;
    const int s = pg < max_pages ? slot_of(table[pg], int(pos & ((1 << shift) - 1)), shift) : -1;
    if (s < 0) atomicOr(flags, CSA2_FLAG_INDEX_OOB);
    return s;
  };
  if (c0 >= ld) return;
  const bool tail = c0 + 3 >= len && c0 < int64_t(len) + CSA2_MAX_TREE;  // may hold drafted rows
  int common[4];  // pages are multiples of four rows: the four columns lie in one
  {
    const int s = table ? slot_of(page0, int(c0 & ((1 << shift) - 1)), shift) : (c0 <= 0x7FFFFFFC ? int(c0) : -1);
    if (s < 0 && c0 < len && nn > 0) atomicOr(flags, CSA2_FLAG_INDEX_OOB);
#pragma unroll
    for (int i = 0; i < 4; ++i) common[i] = s >= 0 && c0 + i < len ? s + i : -1;
  }
  int32_t* dst = slots + int64_t(b) * N * ld + c0;
  for (int r = 0; r < N; ++r, dst += ld) {
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r < nn ? common[i] : -1;
    if (tail && r < nn) {
      unsigned long long m = anc[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t nth = c0 + i - len;  // the nth drafted row of the list
        if (nth < 0 || nth >= __popcll(m)) continue;
        unsigned long long w = m;
        for (int64_t j = 0; j < nth; ++j) w &= w - 1;
        v[i] = slot(int64_t(len) + __ffsll(static_cast<long long>(w)) - 1);
      }
    }
    if (kVec) {
      *reinterpret_cast<int4*>(dst) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i < ld) dst[i] = v[i];
    }
  }
}

inline int page_shift(int page_size) {  // -1: not a power of two in 16..1024
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

}  // namespace pages
}  // namespace csa2

extern "C" csa2_status csa2_block_tables(const int32_t* old_lens, const int32_t* new_lens, int B, int page_size,
                                         int32_t* block_table, int max_pages, int32_t* free_pages, int free_cap,
                                         int32_t* pool_state, int32_t* granted, int32_t* slots, int n_new,
                                         csa2_stream_t stream) {
  using namespace csa2;
  using namespace csa2::pages;
  const int shift = page_shift(page_size);
  if (shift < 0 || B < 0 || B > CSA2_MAX_SEQS || max_pages < 1 || free_cap < 0 || n_new < 0 ||
      int64_t(B) * max_pages > 0x7FFFFFFFll || int64_t(B) * n_new > 0x7FFFFFFFll ||
      (int64_t(max_pages) << shift) > 0x7FFFFFFFll)
    return CSA2_ERR_INVALID_ARG;
  if (B == 0) return CSA2_OK;
  if (!old_lens || !new_lens || !block_table || (free_cap > 0 && !free_pages) || !pool_state || !granted || (n_new > 0 && !slots))
    return CSA2_ERR_INVALID_ARG;
  const void* all[] = {old_lens, new_lens, block_table, free_pages, pool_state, granted, slots};
  for (const void* p : all)
    if (!al(p, 4)) return CSA2_ERR_INVALID_ARG;
  const Span all_spans[] = {span(granted, B, 4),   span(slots, int64_t(B) * n_new, 4), span(block_table, int64_t(B) * max_pages, 4),
                            span(pool_state, 4, 4), span(free_pages, free_cap, 4),      span(old_lens, B, 4),
                            span(new_lens, B, 4)};
  if (any_overlap(all_spans, 5, 7)) return CSA2_ERR_INVALID_ARG;  // (the two lengths may be one array)
  unsigned int* flags = device_flags_ptr();
  const int sms = sm_count();
  if (!flags || sms <= 0) return CSA2_ERR_CUDA;
  // a quad of slots or an entry of the tables a thread; how many pages change hands is known on the device alone.  64
  // sequences x 512 pages, granted and given back: 13.6, 9.7, 7.7, 6.8 us with eight, four, two entries a thread and one
  const int64_t items = std::max(int64_t(B) * ((int64_t(n_new) + 3) / 4), int64_t(B) * max_pages);
  const int grid = int(std::min<int64_t>(std::max<int64_t>(items / kThreads, 1), sms));
  const size_t smem = size_t(B) * 8;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(reinterpret_cast<const void*>(block_tables_kernel), size_t(CSA2_MAX_SEQS) * 8, done) != cudaSuccess)
    return CSA2_ERR_CUDA;
  return launch_pdl(block_tables_kernel, dim3(grid), dim3(kThreads), smem, reinterpret_cast<cudaStream_t>(stream),
                    old_lens, new_lens, B, shift, block_table, max_pages, free_pages, free_cap, pool_state, granted,
                    slots, n_new, n_new % 4 == 0 && al(slots, 16), flags) == cudaSuccess
             ? CSA2_OK
             : CSA2_ERR_CUDA;
}

extern "C" csa2_status csa2_context_slots(const int32_t* lens, const int32_t* parent, const int32_t* n_nodes, int B,
                                          int N, const int32_t* block_table, int max_pages, int page_size,
                                          int32_t* slots, int64_t ld, int32_t* n_slots, csa2_stream_t stream) {
  using namespace csa2;
  using namespace csa2::pages;
  int shift = 4;
  if (B < 0 || B > 65535 || N < 0 || N > CSA2_MAX_TREE || ld < 0 || ld > 0x7FFFFFFFll) return CSA2_ERR_INVALID_ARG;
  if (block_table && (max_pages < 1 || (shift = page_shift(page_size)) < 0)) return CSA2_ERR_INVALID_ARG;
  if (int64_t(B) * N == 0) return CSA2_OK;
  if (!lens || (ld > 0 && !slots) || !n_slots || !al(lens, 4) || !al(parent, 4) || !al(n_nodes, 4) || !al(block_table, 4) ||
      !al(slots, 16) || !al(n_slots, 4))
    return CSA2_ERR_INVALID_ARG;
  const Span spans[] = {span(slots, int64_t(B) * N * ld, 4), span(n_slots, int64_t(B) * N, 4), span(lens, B, 4),
                        span(parent, int64_t(B) * N, 4),     span(n_nodes, B, 4),
                        span(block_table, int64_t(B) * max_pages, 4)};
  if (any_overlap(spans, 2, 6)) return CSA2_ERR_INVALID_ARG;
  unsigned int* flags = device_flags_ptr();
  if (!flags) return CSA2_ERR_CUDA;
  const unsigned gx = unsigned(std::max<int64_t>((ld + 4 * kCtxThreads - 1) / (4 * kCtxThreads), 1));
  auto kern = ld % 4 == 0 ? context_slots_kernel<true> : context_slots_kernel<false>;
  return launch_pdl(kern, dim3(gx, unsigned(B)), dim3(kCtxThreads), 0, reinterpret_cast<cudaStream_t>(stream), lens,
                    parent, n_nodes, N, block_table, max_pages, shift, slots, ld, n_slots, flags) == cudaSuccess
             ? CSA2_OK
             : CSA2_ERR_CUDA;
}
