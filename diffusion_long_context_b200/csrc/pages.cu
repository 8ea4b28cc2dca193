// Care of the cache's pages: reserve, fork, own (copy on write), release, compact.
//
// Reference counts, tables and lists are a few thousand integers that sit in L2, and every
// decision depends on the ones before it, so one CTA of 1024 threads plans a whole call: the
// time is that of a few dependent memory round trips and barriers, not of bytes: 2.0 us a
// release, 2.6 a fork (of 8 branches of 64 pages), 4.5 an own, and compacting 512 pages; 6.9 us a
// reserve of 8 times 64 pages and their release. Nothing
// returns to the host; counts and the pairs that focus_pages_copy has to copy stay on the
// device. Free pages are ranked by block-wide scans in ascending order, so that the result
// never depends on which thread came first.
#include <algorithm>

#include "focus_common.cuh"

namespace focus {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kMaxList = 1024;
constexpr int kScanItems = 4;            // pages a thread looks at in each round of a scan

struct PageArgs {
  int32_t* refs;
  int32_t* table;
  int32_t* held;
  int n_pages, n_seq, cols;
  const int32_t* list[3];
  int n;
  int32_t* pairs;
  int pair_cap;
  int32_t* n_pairs;
  int32_t* status;
  int32_t* remap;
  int* dev_err;
};

// Exclusive prefix sum of v over the CTA; *total receives the sum. Three barriers.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = lane_id(), warp = warp_id();
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();                       // s_warp of an earlier scan has been read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return x - v + (warp > 0 ? s_warp[warp - 1] : 0);
}

// Calls take(rank, page) for the first `need` pages of [0, n_pages) that `want(refs)` accepts,
// ranked in ascending order; returns how many there are (all of them when need < 0, which
// only counts).
template <typename Want, typename Take>
__device__ __forceinline__ int ranked_pages(const PageArgs& a, int lo, int hi, int need, int* s_warp, Want want,
                                            Take take) {
  int base = 0;
  for (int p0 = lo; p0 < hi; p0 += kPageThreads * kScanItems) {
    if (need >= 0 && base >= need) break;          // uniform: base is the same in every thread
    bool hit[kScanItems];
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < kScanItems; ++i) {
      const int p = p0 + static_cast<int>(threadIdx.x) * kScanItems + i;
      hit[i] = p < hi && want(a.refs[p]);
      cnt += hit[i] ? 1 : 0;
    }
    int total = 0;
    int rank = base + block_scan(cnt, s_warp, &total);
    if (need >= 0) {
#pragma unroll
      for (int i = 0; i < kScanItems; ++i)
        if (hit[i]) {
          if (rank < need) take(rank, p0 + static_cast<int>(threadIdx.x) * kScanItems + i);
          ++rank;
        }
    }
    base += total;
  }
  return base;
}

__device__ __forceinline__ void flag(const PageArgs& a) { record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX); }

// Gives up table entry `slot`; threads of different entries may share a page.
__device__ __forceinline__ void drop_entry(const PageArgs& a, size_t slot) {
  const int p = a.table[slot];
  a.table[slot] = -1;
  if (p < 0 || p >= a.n_pages) {
    flag(a);
  } else if (atomicSub(&a.refs[p], 1) <= 0) {
    atomicAdd(&a.refs[p], 1);                      // it was free already: the counts do not match the tables
    flag(a);
  }
}

// ------------------------------------------------------------------ reserve
__global__ void __launch_bounds__(kPageThreads) pages_reserve_kernel(const PageArgs a) {
  __shared__ int s_seq[kMaxList], s_want[kMaxList], s_have[kMaxList], s_pre[kMaxList + 1], s_warp[32];
  griddep_wait();
  griddep_launch_dependents();
  const int i = threadIdx.x;
  int seq = -1, want = 0, have = 0;
  if (i < a.n) {
    seq = a.list[0][i];
    want = a.list[1][i];
    if (seq < 0 || seq >= a.n_seq || want > a.cols) {
      flag(a);
      seq = -1;
    } else {
      have = max(0, min(a.held[seq], a.cols));
    }
    s_seq[i] = seq;
    s_want[i] = want;
  }
  __syncthreads();
  // a sequence that is listed again has what its earlier entries got it
  if (seq >= 0)
    for (int j = 0; j < i; ++j)
      if (s_seq[j] == seq) have = max(have, s_want[j]);
  const int need_i = seq >= 0 ? max(0, want - have) : 0;
  int need = 0;
  const int pre = block_scan(need_i, s_warp, &need);
  if (i < a.n) {
    s_have[i] = have;
    s_pre[i] = pre;
  }
  if (i == 0) s_pre[a.n] = need;
  auto is_free = [](int r) { return r == 0; };
  const int free_n = ranked_pages(a, 0, a.n_pages, -1, s_warp, is_free, [](int, int) {});
  if (need > free_n) {
    if (i == 0) *a.status = need - free_n;
    return;
  }
  if (i == 0) *a.status = 0;
  __syncthreads();                       // every thread has read held, s_pre is complete
  ranked_pages(a, 0, a.n_pages, need, s_warp, is_free, [&](int rank, int page) {
    int lo = 0, hi = a.n - 1;            // the last entry whose prefix is <= rank
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] <= rank) lo = mid;
      else hi = mid - 1;
    }
    a.table[static_cast<size_t>(s_seq[lo]) * a.cols + s_have[lo] + (rank - s_pre[lo])] = page;
    a.refs[page] = 1;
  });
  if (need_i > 0) atomicMax(&a.held[seq], want);
}

// ------------------------------------------------------------------ fork
// Entry i by `nt` threads, of which this is number t.
__device__ __forceinline__ void fork_one(const PageArgs& a, int i, int t, int nt) {
  const int src = a.list[0][i], dst = a.list[1][i];
  if (src < 0 || src >= a.n_seq || dst < 0 || dst >= a.n_seq || src == dst || a.held[dst] != 0) {
    if (t == 0) flag(a);
    return;
  }
  const int keep = max(0, min(a.list[2][i], min(a.held[src], a.cols)));
  for (int j = t; j < keep; j += nt) {
    const int p = a.table[static_cast<size_t>(src) * a.cols + j];
    a.table[static_cast<size_t>(dst) * a.cols + j] = p;
    if (p < 0 || p >= a.n_pages) flag(a);
    else atomicAdd(&a.refs[p], 1);
  }
}

__global__ void __launch_bounds__(kPageThreads) pages_fork_kernel(const PageArgs a) {
  __shared__ int s_dst[kMaxList];
  griddep_wait();
  griddep_launch_dependents();
  const int i = threadIdx.x;
  if (i < a.n) s_dst[i] = a.list[1][i];
  __syncthreads();
  // Entries that name another entry's target (as source or target) have to follow the order
  // of the list; all others are forked side by side, one warp each.
  bool chained = false;
  if (i < a.n) {
    const int src = a.list[0][i];
    for (int j = 0; j < a.n; ++j) chained |= s_dst[j] == src || (j != i && s_dst[j] == s_dst[i]);
  }
  if (__syncthreads_or(chained)) {
    for (int e = 0; e < a.n; ++e) {
      fork_one(a, e, threadIdx.x, kPageThreads);
      __syncthreads();                   // everyone has seen held[dst] before it changes
      if (threadIdx.x == 0) {
        const int src = a.list[0][e], dst = s_dst[e];
        if (src >= 0 && src < a.n_seq && dst >= 0 && dst < a.n_seq && src != dst && a.held[dst] == 0)
          a.held[dst] = max(0, min(a.list[2][e], min(a.held[src], a.cols)));
      }
      __syncthreads();
    }
    return;
  }
  for (int e = warp_id(); e < a.n; e += kPageThreads / 32) {
    fork_one(a, e, lane_id(), 32);
    __syncwarp();
    if (lane_id() == 0) {
      const int src = a.list[0][e], dst = s_dst[e];
      if (src >= 0 && src < a.n_seq && dst >= 0 && dst < a.n_seq && a.held[dst] == 0)
        a.held[dst] = max(0, min(a.list[2][e], min(a.held[src], a.cols)));
    }
  }
}

// ------------------------------------------------------------------ release
__global__ void __launch_bounds__(kPageThreads) pages_release_kernel(const PageArgs a) {
  __shared__ int s_seq[kMaxList], s_keep[kMaxList];
  griddep_wait();
  griddep_launch_dependents();
  const int i = threadIdx.x;
  if (i < a.n) {
    const int seq = a.list[0][i];
    const bool ok = seq >= 0 && seq < a.n_seq;
    if (!ok) flag(a);
    s_seq[i] = ok ? seq : -1;
    s_keep[i] = max(0, a.list[1][i]);
  }
  __syncthreads();
  // of a sequence that is listed more than once the smallest keep counts, at its first entry
  for (int e = warp_id(); e < a.n; e += kPageThreads / 32) {
    const int seq = s_seq[e];
    int keep = 0x7fffffff;
    bool first = seq >= 0;
    for (int j = lane_id(); j < a.n; j += 32)
      if (s_seq[j] == seq) {
        keep = min(keep, s_keep[j]);
        first = first && j >= e;
      }
    first = __all_sync(0xffffffffu, first);
    keep = __reduce_min_sync(0xffffffffu, keep);
    if (!first) continue;
    const int held = max(0, min(a.held[seq], a.cols));
    for (int j = keep + lane_id(); j < held; j += 32) drop_entry(a, static_cast<size_t>(seq) * a.cols + j);
    __syncwarp();
    if (lane_id() == 0 && keep < held) a.held[seq] = keep;
  }
}

// ------------------------------------------------------------------ own
// The listed ranges are walked as one list of entries, 1024 at a time. An entry with page x
// needs a copy when enough others keep x: its rank among this chunk's entries of x is below
// refs[x] - 1, refs[x] already reduced by the chunks before. Until enough free pages are known
// to exist, pairs[r] holds (x, table slot) and can be undone.
struct OwnLists {
  int seq[kMaxList], first[kMaxList], last[kMaxList], pre[kMaxList + 1];   // pre: entries of the ranges before
};

// Place in the table of entry e of the listed ranges, -1 if an earlier range holds it too.
__device__ __forceinline__ int listed_entry(const PageArgs& a, const OwnLists& l, int e) {
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.pre[mid] <= e) lo = mid;
    else hi = mid - 1;
  }
  const int j = l.first[lo] + (e - l.pre[lo]);
  bool again = false;
  for (int o = 0; o < lo; ++o) again |= l.seq[o] == l.seq[lo] && j >= l.first[o] && j < l.last[o];
  return again ? -1 : l.seq[lo] * a.cols + j;
}

// The copies that a call without room for all its pairs needs (this thread's part of their number).
// Copies without a pair have not lowered their page's count, so what the walk found behind them is
// too high. All m entries of a page are taken off its count R and put back one by one; min(m, R - 1)
// of them, the copies, find another one there. (Not inlined: in the kernel's path it cost 2 us.)
__device__ __noinline__ int count_copies(const PageArgs& a, const OwnLists& l, int entries) {
  int copies = 0;
  for (int back = 0; back < 2; ++back) {
    for (int e = threadIdx.x; e < entries; e += kPageThreads) {
      const int slot = listed_entry(a, l, e);
      const int x = slot >= 0 ? a.table[slot] : -1;
      if (x < 0 || x >= a.n_pages) continue;
      const int was = atomicAdd(&a.refs[x], back ? 1 : -1);
      if (back && was >= 1) ++copies;
    }
    __syncthreads();
  }
  return copies;
}

__global__ void __launch_bounds__(kPageThreads) pages_own_kernel(const PageArgs a) {
  __shared__ OwnLists l;
  __shared__ int s_x[kPageThreads], s_warp[32];
  griddep_wait();
  griddep_launch_dependents();
  const int i = threadIdx.x;
  int cnt = 0;
  if (i < a.n) {
    const int seq = a.list[0][i];
    const bool ok = seq >= 0 && seq < a.n_seq;
    if (!ok) flag(a);
    const int first = max(0, a.list[1][i]);
    const int last = ok ? min(a.list[2][i], min(a.held[seq], a.cols)) : 0;
    l.seq[i] = ok ? seq : -1;
    l.first[i] = first;
    l.last[i] = last;
    cnt = max(0, last - first);
  }
  int entries = 0;
  const int pre = block_scan(cnt, s_warp, &entries);
  if (i < a.n) l.pre[i] = pre;
  if (i == 0) l.pre[a.n] = entries;
  __syncthreads();
  int found = 0;                         // copies needed so far (the same in every thread)
  for (int e0 = 0; e0 < entries; e0 += kPageThreads) {
    const int e = e0 + i;
    int x = -1, slot = -1;
    if (e < entries) {
      slot = listed_entry(a, l, e);
      if (slot >= 0) {
        x = a.table[slot];
        if (x < 0 || x >= a.n_pages) {
          flag(a);
          x = -1;
        }
      }
    }
    s_x[i] = x;
    __syncthreads();
    bool copies = false;
    if (x >= 0) {
      int rank = 0;
      for (int j = 0; j < i; ++j) rank += s_x[j] == x ? 1 : 0;
      copies = rank < a.refs[x] - 1;
    }
    int total = 0;
    const int r = found + block_scan(copies ? 1 : 0, s_warp, &total);   // (its barriers follow the reads of refs)
    if (copies && r < a.pair_cap) {
      a.pairs[2 * r] = x;
      a.pairs[2 * r + 1] = slot;
      atomicSub(&a.refs[x], 1);
    }
    found += total;
    __syncthreads();
  }
  auto is_free = [](int r) { return r == 0; };
  const int room = min(a.pair_cap, ranked_pages(a, 0, a.n_pages, -1, s_warp, is_free, [](int, int) {}));
  __syncthreads();
  if (found > room) {
    for (int r = i; r < min(found, a.pair_cap); r += kPageThreads) atomicAdd(&a.refs[a.pairs[2 * r]], 1);
    if (found > a.pair_cap) {            // (counted too high, see count_copies)
      __syncthreads();
      block_scan(count_copies(a, l, entries), s_warp, &found);
    }
    if (i == 0) {
      *a.status = found - room;
      *a.n_pairs = 0;
    }
    return;
  }
  ranked_pages(a, 0, a.n_pages, found, s_warp, is_free, [&](int rank, int page) {
    a.table[a.pairs[2 * rank + 1]] = page;
    a.pairs[2 * rank + 1] = page;
    a.refs[page] = 1;
  });
  if (i == 0) {
    *a.status = 0;
    *a.n_pairs = found;
  }
}

// ------------------------------------------------------------------ compact
__global__ void __launch_bounds__(kPageThreads) pages_compact_kernel(const PageArgs a) {
  __shared__ int s_warp[32];
  griddep_wait();
  griddep_launch_dependents();
  auto is_free = [](int r) { return r <= 0; };
  auto is_live = [](int r) { return r > 0; };
  const int live = ranked_pages(a, 0, a.n_pages, -1, s_warp, is_live, [](int, int) {});
  // as many holes before `live` as live pages behind it
  const int moves = ranked_pages(a, 0, live, live, s_warp, is_free, [&](int rank, int page) { a.pairs[2 * rank + 1] = page; });
  ranked_pages(a, live, a.n_pages, moves, s_warp, is_live, [&](int rank, int page) { a.pairs[2 * rank] = page; });
  __syncthreads();
  for (int p = threadIdx.x; p < a.n_pages; p += kPageThreads) a.remap[p] = a.refs[p] > 0 ? p : -1;
  __syncthreads();
  for (int r = threadIdx.x; r < moves; r += kPageThreads) {
    const int src = a.pairs[2 * r], dst = a.pairs[2 * r + 1];
    a.remap[src] = dst;
    a.refs[dst] = a.refs[src];
    a.refs[src] = 0;
  }
  if (threadIdx.x == 0) *a.n_pairs = moves;
}

// Table entries follow their pages; the entries behind held stay as they are.
__global__ void __launch_bounds__(256) pages_remap_kernel(const PageArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const long long total = static_cast<long long>(a.n_seq) * a.cols;
  for (long long x = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * 256) {
    const int seq = static_cast<int>(x / a.cols);
    if (x - static_cast<long long>(seq) * a.cols >= a.held[seq]) continue;
    const int p = a.table[x];
    if (p < 0 || p >= a.n_pages) flag(a);
    else a.table[x] = a.remap[p];
  }
}

int check_pages(const focus_pages* p, int n) {
  FOCUS_CHECK_ARG(p && p->refs && p->table && p->held, "null pointer argument (pages)");
  FOCUS_CHECK_ARG(p->n_pages >= 1 && p->n_seq >= 1 && p->table_cols >= 1, "bad sizes (n_pages=%d n_seq=%d table_cols=%d)",
                  p->n_pages, p->n_seq, p->table_cols);
  FOCUS_CHECK_ARG(static_cast<long long>(p->n_seq) * p->table_cols < (1LL << 31) && p->n_pages < (1 << 30),
                  "tables of 2^31 entries or more");
  FOCUS_CHECK_ARG(n >= 0, "negative list length %d", n);
  if (n > kMaxList) {
    set_error("pages: lists of up to %d entries (got %d)", kMaxList, n);
    return FOCUS_ERR_UNSUPPORTED;
  }
  return FOCUS_OK;
}

PageArgs page_args(const focus_pages* p, const int32_t* l0, const int32_t* l1, const int32_t* l2, int n) {
  PageArgs a{};
  a.refs = p->refs;
  a.table = p->table;
  a.held = p->held;
  a.n_pages = p->n_pages;
  a.n_seq = p->n_seq;
  a.cols = p->table_cols;
  a.list[0] = l0;
  a.list[1] = l1;
  a.list[2] = l2;
  a.n = n;
  a.dev_err = device_error_word();
  return a;
}

int plan(void (*kern)(const PageArgs), const PageArgs& a, void* stream, const char* what) {
  const cudaError_t e =
      launch_k(kern, dim3(1), dim3(kPageThreads), 0, static_cast<cudaStream_t>(stream), a);
  note_launch();
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("%s launch: %s", what, cudaGetErrorString(e));
    return FOCUS_ERR_CUDA;
  }
  return FOCUS_OK;
}

}  // namespace
}  // namespace focus

using namespace focus;

extern "C" int focus_pages_reserve(const focus_pages* pages, const int32_t* seqs, const int32_t* want, int n,
                                   int32_t* status, void* stream) {
  if (const int st = check_pages(pages, n)) return st;
  FOCUS_CHECK_ARG(status && (n == 0 || (seqs && want)), "null pointer argument");
  PageArgs a = page_args(pages, seqs, want, nullptr, n);
  a.status = status;
  return plan(pages_reserve_kernel, a, stream, "pages_reserve");
}

extern "C" int focus_pages_fork(const focus_pages* pages, const int32_t* src, const int32_t* dst, const int32_t* keep,
                                int n, void* stream) {
  if (const int st = check_pages(pages, n)) return st;
  FOCUS_CHECK_ARG(n == 0 || (src && dst && keep), "null pointer argument");
  if (n == 0) return FOCUS_OK;
  return plan(pages_fork_kernel, page_args(pages, src, dst, keep, n), stream, "pages_fork");
}

extern "C" int focus_pages_own(const focus_pages* pages, const int32_t* seqs, const int32_t* first,
                               const int32_t* last, int n, int32_t* pairs, int pair_cap, int32_t* n_pairs,
                               int32_t* status, void* stream) {
  if (const int st = check_pages(pages, n)) return st;
  FOCUS_CHECK_ARG(n_pairs && status && (n == 0 || (seqs && first && last)), "null pointer argument");
  FOCUS_CHECK_ARG(pair_cap >= 0 && (pair_cap == 0 || pairs), "bad pairs");
  if (static_cast<long long>(n) * pages->table_cols >= (1LL << 31) - kPageThreads) {
    // (entries are counted in 32 bits, and a pass behind the last)
    set_error("pages_own: %d ranges of up to %d entries, nearly 2^31 or more in all", n, pages->table_cols);
    return FOCUS_ERR_UNSUPPORTED;
  }
  PageArgs a = page_args(pages, seqs, first, last, n);
  a.pairs = pairs;
  a.pair_cap = pair_cap;
  a.n_pairs = n_pairs;
  a.status = status;
  return plan(pages_own_kernel, a, stream, "pages_own");
}

extern "C" int focus_pages_release(const focus_pages* pages, const int32_t* seqs, const int32_t* keep, int n,
                                   void* stream) {
  if (const int st = check_pages(pages, n)) return st;
  FOCUS_CHECK_ARG(n == 0 || (seqs && keep), "null pointer argument");
  if (n == 0) return FOCUS_OK;
  return plan(pages_release_kernel, page_args(pages, seqs, keep, nullptr, n), stream, "pages_release");
}

extern "C" int focus_pages_compact(const focus_pages* pages, int32_t* pairs, int pair_cap, int32_t* n_pairs,
                                   int32_t* remap, void* stream) {
  if (const int st = check_pages(pages, 0)) return st;
  FOCUS_CHECK_ARG(n_pairs && remap && pair_cap >= 0 && (pair_cap == 0 || pairs), "null pointer argument");
  if (pair_cap < pages->n_pages / 2) {
    set_error("pages_compact: pair_cap %d < n_pages / 2 = %d", pair_cap, pages->n_pages / 2);
    return FOCUS_ERR_CAPACITY;
  }
  PageArgs a = page_args(pages, nullptr, nullptr, nullptr, 0);
  a.pairs = pairs;
  a.pair_cap = pair_cap;
  a.n_pairs = n_pairs;
  a.remap = remap;
  if (const int st = plan(pages_compact_kernel, a, stream, "pages_compact")) return st;
  const long long total = static_cast<long long>(a.n_seq) * a.cols;
  const long long grid = std::min<long long>((total + 255) / 256, static_cast<long long>(device_sm_count()) * 8);
  const cudaError_t e = launch_k(pages_remap_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0,
                                 static_cast<cudaStream_t>(stream), a);
  note_launch();
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("pages_remap launch: %s", cudaGetErrorString(e));
    return FOCUS_ERR_CUDA;
  }
  return FOCUS_OK;
}
