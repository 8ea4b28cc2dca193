// Rows of the 8-bit paged cache: storing whole prompts, replacing single rows, reading back,
// copying pages.
//
// All four only move bytes: a store reads 2 bytes and writes 1 per element, a load the other
// way round, a copy 1 and 1. The scale of a page needs the largest magnitude of its rows
// before the first code can be written, so a group of threads holds a whole page of one head
// in registers between the two: page * d / 32 threads with four 16-byte vectors each.
//
// Measured (graph replay, of 6.55 TB/s that a copy reaches): 268M elements in e4m3, pages of 64,
// stored in 154 us (5.2 TB/s) and loaded in 157 us (5.1 TB/s), from memory's side bound by the
// mix of reads and writes; 32 rows of 32 layers of 32 heads replaced in 16.5 us and read back in
// 11.5 us: 2048 CTAs of 256 threads and 64 registers, four to an SM, so 3.5 rounds of a few
// dependent loads each; a page copy 5.7 TB/s.
#include <algorithm>

#include "cache.cuh"

namespace focus {

int check_cache(const focus_cache* c, const int32_t* table, int table_cols, bool n_mat_one) {
  FOCUS_CHECK_ARG(c && c->k && c->v && c->k_scale && c->v_scale, "null pointer argument (cache)");
  FOCUS_CHECK_ARG(c->format == FOCUS_CACHE_E4M3 || c->format == FOCUS_CACHE_INT8, "unknown cache format %d", c->format);
  FOCUS_CHECK_ARG(c->n_mat >= 0 && c->n_pages >= 1 && c->Hkv >= 1, "bad cache sizes (n_mat=%d n_pages=%d Hkv=%d)",
                  c->n_mat, c->n_pages, c->Hkv);
  FOCUS_CHECK_ARG(!n_mat_one || c->n_mat == 1, "attention reads the cache of one layer (n_mat=%d)", c->n_mat);
  if (c->d != 64 && c->d != 128) {
    set_error("cache: d must be 64 or 128 (got %d)", c->d);
    return FOCUS_ERR_UNSUPPORTED;
  }
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) {
    set_error("cache: page must be 16, 32, 64 or 128 (got %d)", c->page);
    return FOCUS_ERR_UNSUPPORTED;
  }
  FOCUS_CHECK_ARG(static_cast<long long>(c->n_pages) * c->Hkv < (1LL << 31), "cache: n_pages * Hkv must be below 2^31");
  FOCUS_CHECK_ARG(aligned16(c->k) && aligned16(c->v), "cache codes must be 16-byte aligned");
  FOCUS_CHECK_ARG((reinterpret_cast<uintptr_t>(c->k_scale) & 3u) == 0 && (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) == 0,
                  "cache scales must be 4-byte aligned");
  FOCUS_CHECK_ARG(table && table_cols >= 1, "null table or no columns");
  return FOCUS_OK;
}

namespace {

struct RowArgs {
  const uint4* X[2];           // K, V (bf16 rows)
  uint2* code[2];              // codes, eight to a vector
  float* scale[2];
  uint4* out[2];               // load: bf16 rows
  const int32_t* lens;
  const int32_t* table;
  const int32_t* rows;         // scatter
  const int32_t* n_rows;
  int table_cols, B, H, L, d, page, n_pages, cap, start;
  int cols;                    // store: pages of L positions
  int page_shift, vec_shift;   // log2 of page, and of the vectors (of 8 elements) of a row
  int* dev_err;
};

// Largest of the eight |x| of a vector of bf16, as the bits of its magnitude (a NaN's bits are
// above infinity's, which are above every number's, so both come through).
__device__ __forceinline__ uint32_t absmax_bits(uint4 v, uint32_t m) {
  uint32_t a = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m, max(a & 0xffffu, a >> 16));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The codes of eight bf16 under scale s, those of the IEEE quotient x / s (exact ties between two
// codes exist in plenty: bf16 has few mantissas).
//
// As divisions the eight were most of a store's instructions. With r the rounded reciprocal,
// q = x r is off by less than 2 ulp, and q + (x - q s) r, one step of residual correction
// (Markstein 1990), by less than 2^-45 of x / s before its own rounding. So its code can differ
// from the quotient's only where x / s lies that close to a midpoint of two floats next to a tie
// t of two codes. With mantissas as integers that is x = (T 2^a +- 1) s to within 16 units, with
// T 2^a of 25 bits, T (the tie) of 5 or 8 bits, s of 24, x a multiple of 2^40: s is then
// u 2^a -+ c with |c| <= 16, and u = T c. But u has one bit less than T, so no s does that (nor
// below a tie that is a power of two, where s would have to be -c).
// The bounds on s keep r, q s and every residual that matters normal numbers.
template <int FMT>
__device__ __forceinline__ uint2 encode8(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
  if (s > 0x1p-90f && s < 0x1p90f) {
    const float r = 1.f / s;
    const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
      const float2 q = mul2(x, r2);
      const float2 y = fma2(fma2(q, s2, x), r2, q);
      if constexpr (FMT == FOCUS_CACHE_E4M3) {
        c[i] = code2<FMT>(y.x, y.y);
      } else {
        // rounded to an integer by adding 1.5 * 2^23
        const float2 n = add2(y, make_float2(12582912.f, 12582912.f));
        c[i] = __byte_perm(__float_as_uint(n.x), __float_as_uint(n.y), 0x0040);
      }
    }
    uint2 out = make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
    if constexpr (FMT == FOCUS_CACHE_E4M3) {
      // the sign of a zero, which the correction drops
      out.x |= __byte_perm(w[0], w[1], 0x7531) & 0x80808080u;
      out.y |= __byte_perm(w[2], w[3], 0x7531) & 0x80808080u;
    }
    return out;
  }
  if (s == 0.f) return make_uint2(0u, 0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = code2<FMT>(bf16_lo(w[i]) / s, bf16_hi(w[i]) / s);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Eight held codes under a grown scale: the codes of the IEEE quotients (code * s_old) / s. Two
// residual corrections here: the first leaves a faithful quotient, from which the second gives
// the IEEE one (Markstein 1990), since the dividend has all 24 bits.
template <int FMT>
__device__ __forceinline__ uint2 recode8(uint2 held, float s_old, float s) {
  const uint32_t w[2] = {held.x, held.y};
  uint32_t out[2];
  const bool scaled = s_old > 0x1p-60f && s < 0x1p60f;     // (s_old < s; every step a normal number)
  const float r = 1.f / s;
  const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s), o2 = make_float2(s_old, s_old);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[4];
    decode4<FMT>(w[i], x);
    uint32_t c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 y = mul2(make_float2(x[2 * e], x[2 * e + 1]), o2);
      if (scaled) {
        float2 q = mul2(y, r2);
        q = fma2(fma2(q, s2, y), r2, q);
        q = fma2(fma2(q, s2, y), r2, q);
        c[e] = code2<FMT>(q.x, q.y);
      } else {
        c[e] = code2<FMT>(y.x / s, y.y / s);
      }
    }
    out[i] = c[0] | (c[1] << 16);
    if (FMT == FOCUS_CACHE_E4M3 && scaled) out[i] |= w[i] & 0x80808080u;      // the sign of a zero
  }
  return make_uint2(out[0], out[1]);
}

// Largest of `m` over the group of `gt` threads (whole warps) that works on one page; every
// thread of the CTA calls it. s_red holds a word for each warp.
__device__ __forceinline__ uint32_t group_max(uint32_t m, int gt, uint32_t* s_red) {
  m = __reduce_max_sync(0xffffffffu, m);
  if (gt == 32) return m;
  __syncthreads();                       // the words of an earlier call have been read
  if (lane_id() == 0) s_red[warp_id()] = m;
  __syncthreads();
  const int w0 = warp_id() / (gt / 32) * (gt / 32);
  for (int w = 0; w < gt / 32; ++w) m = max(m, s_red[w0 + w]);
  return m;
}

// ------------------------------------------------------------------ store
// A group of page * d / 32 threads stores one page of one head; a CTA holds 256 threads or one
// group. blockIdx.y: head, of the keys and then of the values; blockIdx.z: matrix and sequence (as
// grid dimensions: the divisions of one number cost as many instructions as the codes).
// The rows are requested before the page is looked up.
template <int FMT>
__global__ void __launch_bounds__(512) cache_store_kernel(const RowArgs a) {
  __shared__ uint32_t s_red[16];
  griddep_wait();
  griddep_launch_dependents();
  const int kv = blockIdx.y >= a.H ? 1 : 0, h = blockIdx.y - kv * a.H;
  const int gshift = a.page_shift + a.vec_shift - 2, gt = 1 << gshift;   // threads of a group
  const int t = threadIdx.x & (gt - 1);
  const int mat = blockIdx.z / a.B, b = blockIdx.z - mat * a.B;
  const int j = blockIdx.x * (blockDim.x >> gshift) + (threadIdx.x >> gshift);   // page of the sequence
  const int len = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
  const int n = j < a.cols ? stored_vectors(len, j, a.page_shift, a.vec_shift) : 0;
  const long long mbh = static_cast<long long>(blockIdx.z) * a.H + h;
  const uint4* src = a.X[kv] + ((mbh * a.L + (static_cast<long long>(j) << a.page_shift)) << a.vec_shift);
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = t + i * gt;
    v[i] = c < n ? __ldcs(src + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int page = n > 0 ? checked_page(a.table, a.table_cols, b, j, a.n_pages, a.dev_err) : -1;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = absmax_bits(v[i], m);
  m = group_max(m, gt, s_red);
  if (page < 0) return;
  const float s = __uint_as_float(m << 16) / CodeTop<FMT>::value;
  const long long ph = (static_cast<long long>(mat) * a.n_pages + page) * a.H + h;   // page and head
  uint2* dst = a.code[kv] + (ph << (a.page_shift + a.vec_shift));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = t + i * gt;
    if (c < n) dst[c] = encode8<FMT>(v[i], s);
  }
  if (t == 0) a.scale[kv][ph] = s;
}

// ------------------------------------------------------------------ scatter_rows
constexpr int kMaxCap = 4096;

// The CTAs (x = split, y = (mat, b, h), z = keys/values) of one head share the pages that its
// rows fall in: the first listed row of a page leads, leader number n goes to split n mod
// gridDim.x. A page is then rebuilt as in the store, from the new rows and the held codes.
//
// Bound by its chain of dependent steps, not by bytes. A list of 32 rows at most (one denoising
// block, SHORT) is a register of each warp: leaders by a match, the row of a position by a
// ballot, no shared memory and no barriers but those of the largest magnitude (32 rows of 32
// layers of 32 heads: 16.5 us against 19.3 by the way for longer lists). Longer lists lie
// in dynamic shared memory, as long as the call's cap (with room for the longest always, six
// CTAs fitted an SM): 40 rows of 32 layers of 32 heads 26 us, 128 rows 40, 512 rows 124.
struct PageRows {                        // what a thread writes of a page: vectors t, t + gt, ...
  int src[4];                            // listed rows, -1 = none
};

// Rebuilds one page from the new rows src; the whole CTA.
template <int FMT>
__device__ __forceinline__ void rebuild_page(const RowArgs& a, int kv, int mbh, long long ph, int p0, int len, PageRows& w,
                                             uint32_t* s_red) {
  const int gt = blockDim.x, t = threadIdx.x;
  const bool held = p0 < len;
  const float s_old = held ? a.scale[kv][ph] : 0.f;
  const uint4* X = a.X[kv] + ((static_cast<long long>(mbh) * a.cap) << a.vec_shift);
  const int in_row = t & ((1 << a.vec_shift) - 1);         // (gt is a multiple of a row's vectors)
  uint4 v[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (w.src[i] >= 0) v[i] = __ldg(X + (static_cast<long long>(w.src[i]) << a.vec_shift) + in_row);
    m = absmax_bits(v[i], m);
  }
  m = group_max(m, gt, s_red);
  const float s_new = __uint_as_float(m << 16) / CodeTop<FMT>::value;
  const bool grown = !(s_new <= s_old) && s_old == s_old;      // a NaN stays what it is
  const float s = grown ? s_new : s_old;
  uint2* dst = a.code[kv] + (ph << (a.page_shift + a.vec_shift));
  uint2 old[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = t + i * gt;
    const bool again = w.src[i] < 0 && held && grown && p0 + (c >> a.vec_shift) < len;
    if (again) old[i] = dst[c];
    else if (w.src[i] < 0) w.src[i] = -2;                  // stays as it is
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (w.src[i] >= 0) dst[t + i * gt] = encode8<FMT>(v[i], s);
    else if (w.src[i] == -1) dst[t + i * gt] = recode8<FMT>(old[i], s_old, s);
  }
  __syncthreads();                       // every thread has read s_old
  if (t == 0) a.scale[kv][ph] = s;
}

template <int FMT, bool SHORT>
__global__ void __launch_bounds__(512) cache_scatter_kernel(const RowArgs a) {
  extern __shared__ int s_pos[];         // [cap] position of each listed row, -1 = not written
  int* const s_lead = s_pos + a.cap;     // [cap] the leaders of this CTA
  __shared__ uint32_t s_red[16];
  __shared__ int s_src[128];             // row of the page -> listed row, -1 = none
  __shared__ int s_nlead, s_count[16], s_base;
  griddep_wait();
  griddep_launch_dependents();
  const int kv = blockIdx.z;
  const int mbh = blockIdx.y;
  const int mb = mbh / a.H, h = mbh - mb * a.H, mat = mb / a.B, b = mb - mat * a.B;
  const int n = max(0, min(a.n_rows[b], a.cap));
  const int len = a.lens[b];
  const int32_t* rows = a.rows + static_cast<size_t>(b) * a.cap;
  const int gt = blockDim.x, t = threadIdx.x, ps = a.page_shift;
  const long long heads = static_cast<long long>(mat) * a.n_pages;
  if constexpr (SHORT) {
    const int lane = lane_id();
    int pos = -1;
    if (lane < n) {
      pos = rows[lane];
      if (pos < 0 || (pos >> ps) >= a.table_cols) {
        record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
        pos = -1;
      }
    }
    const int col_of = pos >> ps;                          // (-1 for what is not written)
    const unsigned same = __match_any_sync(0xffffffffu, col_of);
    unsigned leaders = __ballot_sync(0xffffffffu, pos >= 0 && __ffs(same) - 1 == lane);
    int page_of = -1;
    if ((leaders >> lane) & 1u) page_of = checked_page(a.table, a.table_cols, b, col_of, a.n_pages, a.dev_err);
    for (int l = 0; leaders; ++l, leaders &= leaders - 1) {
      if (l % static_cast<int>(gridDim.x) != static_cast<int>(blockIdx.x)) continue;
      const int first = __ffs(leaders) - 1;
      const int p0 = __shfl_sync(0xffffffffu, col_of, first) << ps, page = __shfl_sync(0xffffffffu, page_of, first);
      if (page < 0) continue;                              // the same for the whole CTA
      // a warp's 32 vectors are of 2 rows, or with d = 64 of 4
      PageRows w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = p0 + ((t + i * gt) >> a.vec_shift);
        w.src[i] = -1;
        for (int k = 0; k < 32; k += 1 << a.vec_shift) {
          const int r = __shfl_sync(0xffffffffu, row, k);
          const unsigned listed = __ballot_sync(0xffffffffu, pos == r);
          if (row == r && listed) w.src[i] = 31 - __clz(listed);      // the last listed row of the position
        }
      }
      rebuild_page<FMT>(a, kv, mbh, (heads + page) * a.H + h, p0, len, w, s_red);
    }
    return;
  }
  bool sorted = true;
  for (int i = t; i < n; i += gt) {
    const int r = rows[i];
    const bool ok = r >= 0 && (r >> ps) < a.table_cols;
    if (!ok) record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
    s_pos[i] = ok ? r : -1;
    sorted = sorted && ok && (i == 0 || rows[i - 1] < r);
  }
  if (t == 0) {
    s_nlead = 0;
    s_base = 0;
  }
  sorted = __syncthreads_and(sorted);
  // leaders in the order of the list, numbered by a scan over chunks of the CTA
  for (int i0 = 0; i0 < n; i0 += gt) {
    const int i = i0 + t;
    bool lead = i < n && s_pos[i] >= 0;
    if (lead && sorted) lead = i == 0 || s_pos[i - 1] >> ps != s_pos[i] >> ps;
    else if (lead)
      for (int j = 0; j < i && lead; ++j) lead = s_pos[j] < 0 || s_pos[j] >> ps != s_pos[i] >> ps;
    const unsigned bal = __ballot_sync(0xffffffffu, lead);
    if (lane_id() == 0) s_count[warp_id()] = __popc(bal);
    __syncthreads();
    int at = s_base;
    for (int w = 0; w < warp_id(); ++w) at += s_count[w];
    at += __popc(bal & ((1u << lane_id()) - 1u));
    if (lead && at % static_cast<int>(gridDim.x) == static_cast<int>(blockIdx.x)) s_lead[at / gridDim.x] = i;
    __syncthreads();
    if (t == 0) {
      for (int w = 0; w < (gt + 31) / 32; ++w) s_base += s_count[w];
      const int own = s_base - static_cast<int>(blockIdx.x);
      s_nlead = own <= 0 ? 0 : (own + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    }
    __syncthreads();
  }
  const int nlead = s_nlead;
  for (int l = 0; l < nlead; ++l) {
    const int first = s_lead[l], col = s_pos[first] >> ps, p0 = col << ps;
    __syncthreads();                     // the previous page's s_src has been read
    // the last listed row of each position
    if (sorted) {
      for (int r = t; r < a.page; r += gt) s_src[r] = -1;
      __syncthreads();
      for (int i = first + t; i < min(n, first + a.page); i += gt)
        if (s_pos[i] >> ps == col) s_src[s_pos[i] - p0] = i;
    } else {
      for (int r = t; r < a.page; r += gt) {
        int src = -1;
        for (int i = first; i < n; ++i)
          if (s_pos[i] == p0 + r) src = i;
        s_src[r] = src;
      }
    }
    const int page = checked_page(a.table, a.table_cols, b, col, a.n_pages, a.dev_err);
    __syncthreads();
    if (page < 0) continue;              // the same for the whole CTA
    PageRows w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w.src[i] = s_src[(t + i * gt) >> a.vec_shift];
    rebuild_page<FMT>(a, kv, mbh, (heads + page) * a.H + h, p0, len, w, s_red);
  }
}

// ------------------------------------------------------------------ load
// A CTA loads 2048 vectors of eight codes (128 rows of 128 elements) of one head, eight to a
// thread, all requested before the first is used. Eight codes are 16 bytes of the output: with
// sixteen to a vector, each store of a warp wrote half of the 32-byte sectors it touched.
constexpr int kLoadThreads = 256, kLoadVecs = 8;
template <int FMT>
__global__ void __launch_bounds__(kLoadThreads) cache_load_kernel(const RowArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int kv = blockIdx.y >= a.H ? 1 : 0, h = blockIdx.y - kv * a.H;
  const int mat = blockIdx.z / a.B, b = blockIdx.z - mat * a.B;
  const int n = min(a.L, max(0, a.lens[b]) - a.start);                   // rows of this sequence
  const long long x0 = static_cast<long long>(blockIdx.x) * (kLoadThreads * kLoadVecs) + threadIdx.x;
  uint2 c[kLoadVecs];
  float s[kLoadVecs];
#pragma unroll
  for (int i = 0; i < kLoadVecs; ++i) {
    const long long x = x0 + i * kLoadThreads;
    const int row = static_cast<int>(x >> a.vec_shift);
    c[i] = make_uint2(0u, 0u);
    s[i] = 0.f;
    if (row < n) {
      const int pos = a.start + row;
      const int page = checked_page(a.table, a.table_cols, b, pos >> a.page_shift, a.n_pages, a.dev_err);
      if (page >= 0) {
        const long long ph = (static_cast<long long>(mat) * a.n_pages + page) * a.H + h;
        c[i] = __ldcs(a.code[kv] + (((ph << a.page_shift) + (pos & (a.page - 1))) << a.vec_shift) +
                      (x & ((1 << a.vec_shift) - 1)));
        s[i] = a.scale[kv][ph];
      }
    }
  }
  uint4* dst = a.out[kv] + (((static_cast<long long>(blockIdx.z) * a.H + h) * a.L) << a.vec_shift);
#pragma unroll
  for (int i = 0; i < kLoadVecs; ++i) {
    const long long x = x0 + i * kLoadThreads;
    if (static_cast<int>(x >> a.vec_shift) >= n) continue;
    float f[4], g[4];
    decode4<FMT>(c[i].x, f);
    decode4<FMT>(c[i].y, g);
    __stcs(dst + x, make_uint4(pack_bf16x2(f[0] * s[i], f[1] * s[i]), pack_bf16x2(f[2] * s[i], f[3] * s[i]),
                               pack_bf16x2(g[0] * s[i], g[1] * s[i]), pack_bf16x2(g[2] * s[i], g[3] * s[i])));
  }
}

// ------------------------------------------------------------------ copy of pages
// The page of one layer is Hkv * page * d contiguous codes, keys and values alike. A CTA copies
// 16 KB pieces (four vectors a thread in flight); the last piece number of a page stands for
// its scales. How many pairs there are is known on the device only, so a grid that fills the
// GPU walks over them.
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(uint4* k, uint4* v, float* ks, float* vs, int n_mat,
                                                                  int n_pages, int H, long long page_vecs,
                                                                  const int32_t* pairs, const int32_t* n_pairs,
                                                                  int pair_cap, int* dev_err) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = max(0, min(*n_pairs, pair_cap));
  const int pieces = static_cast<int>((page_vecs + 4 * kCopyThreads - 1) / (4 * kCopyThreads));
  const int per_page = 2 * pieces + 1;
  const int total = per_page * n * n_mat;
  for (int w = blockIdx.x; w < total; w += gridDim.x) {
    const int pm = w / per_page, piece = w - pm * per_page;
    const int r = pm / n_mat, m = pm - r * n_mat;
    const int src = pairs[2 * r], dst = pairs[2 * r + 1];
    if (src < 0 || src >= n_pages || dst < 0 || dst >= n_pages) {
      if (threadIdx.x == 0) record_dev_error(dev_err, DEV_ERR_BAD_INDEX);
      continue;
    }
    const long long so = static_cast<long long>(m) * n_pages + src, dn = static_cast<long long>(m) * n_pages + dst;
    if (piece == 2 * pieces) {
      for (int h = threadIdx.x; h < H; h += kCopyThreads) {
        ks[dn * H + h] = ks[so * H + h];
        vs[dn * H + h] = vs[so * H + h];
      }
      continue;
    }
    uint4* base = piece < pieces ? k : v;
    const long long off = static_cast<long long>(piece < pieces ? piece : piece - pieces) * (4 * kCopyThreads) + threadIdx.x;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (off + i * kCopyThreads < page_vecs) x[i] = __ldcs(base + so * page_vecs + off + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (off + i * kCopyThreads < page_vecs) base[dn * page_vecs + off + i * kCopyThreads] = x[i];
  }
}

RowArgs row_args(const focus_cache* c, const int32_t* table, int table_cols, const int32_t* lens, int B) {
  RowArgs a{};
  a.code[0] = static_cast<uint2*>(c->k);
  a.code[1] = static_cast<uint2*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.lens = lens;
  a.table = table;
  a.table_cols = table_cols;
  a.B = B;
  a.H = c->Hkv;
  a.d = c->d;
  a.page = c->page;
  a.n_pages = c->n_pages;
  a.page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  a.vec_shift = c->d == 128 ? 4 : 3;
  a.dev_err = device_error_word();
  return a;
}

// Grids of (positions, keys' and values' heads, matrix and sequence).
int check_grid(long long units, int H, const char* what) {
  if (units <= 65535 && H <= 32767) return FOCUS_OK;
  set_error("%s: n_mat * B = %lld exceeds 65535 or Hkv = %d 32767", what, units, H);
  return FOCUS_ERR_UNSUPPORTED;
}

int launched(cudaError_t e, const char* what) {
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

extern "C" int focus_cache_store(const focus_bf16* K, const focus_bf16* V, int B, int L, const int32_t* lens,
                                 const int32_t* table, int table_cols, const focus_cache* cache, void* stream) {
  FOCUS_CHECK_ARG(K && V, "null pointer argument");
  if (const int st = check_cache(cache, table, table_cols, false)) return st;
  FOCUS_CHECK_ARG(B >= 0 && L >= 1, "bad sizes (B=%d L=%d)", B, L);
  FOCUS_CHECK_ARG(aligned16(K) && aligned16(V), "tensors must be 16-byte aligned");
  const long long units = static_cast<long long>(cache->n_mat) * B;
  if (units == 0) return FOCUS_OK;
  if (const int st = check_grid(units, cache->Hkv, "cache_store")) return st;
  RowArgs a = row_args(cache, table, table_cols, lens, B);
  a.X[0] = reinterpret_cast<const uint4*>(K);
  a.X[1] = reinterpret_cast<const uint4*>(V);
  a.L = L;
  a.cols = (L - 1) / a.page + 1;
  const int gt = a.page * a.d / 32, threads = std::max(256, gt), per = threads / gt;
  auto kern = cache->format == FOCUS_CACHE_E4M3 ? cache_store_kernel<FOCUS_CACHE_E4M3> : cache_store_kernel<FOCUS_CACHE_INT8>;
  return launched(launch_k(kern, dim3((a.cols + per - 1) / per, 2 * a.H, static_cast<unsigned>(units)), dim3(threads), 0,
                           static_cast<cudaStream_t>(stream), a),
                  "cache_store");
}

extern "C" int focus_cache_scatter_rows(const focus_bf16* K_rows, const focus_bf16* V_rows, const int32_t* rows,
                                        const int32_t* n_rows, int B, int cap, const int32_t* lens,
                                        const int32_t* table, int table_cols, const focus_cache* cache, void* stream) {
  FOCUS_CHECK_ARG(K_rows && V_rows && rows && n_rows && lens, "null pointer argument");
  if (const int st = check_cache(cache, table, table_cols, false)) return st;
  FOCUS_CHECK_ARG(B >= 0 && cap >= 1, "bad sizes (B=%d cap=%d)", B, cap);
  if (cap > kMaxCap) {
    set_error("cache_scatter_rows: cap %d exceeds %d", cap, kMaxCap);
    return FOCUS_ERR_UNSUPPORTED;
  }
  FOCUS_CHECK_ARG(aligned16(K_rows) && aligned16(V_rows), "tensors must be 16-byte aligned");
  const long long units = static_cast<long long>(cache->n_mat) * B * cache->Hkv;
  if (units == 0) return FOCUS_OK;
  if (units > 65535) {
    set_error("cache_scatter_rows: n_mat * B * Hkv = %lld exceeds 65535", units);
    return FOCUS_ERR_UNSUPPORTED;
  }
  RowArgs a = row_args(cache, table, table_cols, lens, B);
  a.X[0] = reinterpret_cast<const uint4*>(K_rows);
  a.X[1] = reinterpret_cast<const uint4*>(V_rows);
  a.rows = rows;
  a.n_rows = n_rows;
  a.cap = cap;
  // rows next to each other fall in cap / page + 1 pages or fewer; no more CTAs to a head than fill
  // the GPU eight times
  const long long fill = (static_cast<long long>(device_sm_count()) * 8 + 2 * units - 1) / (2 * units);
  const int splits = static_cast<int>(std::min<long long>(std::min(16, (cap + a.page - 1) / a.page + 1), fill));
  const bool e4m3 = cache->format == FOCUS_CACHE_E4M3, few = cap <= 32;
  auto kern = few ? (e4m3 ? cache_scatter_kernel<FOCUS_CACHE_E4M3, true> : cache_scatter_kernel<FOCUS_CACHE_INT8, true>)
                  : (e4m3 ? cache_scatter_kernel<FOCUS_CACHE_E4M3, false> : cache_scatter_kernel<FOCUS_CACHE_INT8, false>);
  return launched(launch_k(kern, dim3(splits, static_cast<unsigned>(units), 2), dim3(a.page * a.d / 32),
                           few ? 0 : 2 * sizeof(int) * static_cast<size_t>(cap),
                           static_cast<cudaStream_t>(stream), a),
                  "cache_scatter_rows");
}

extern "C" int focus_cache_load(const focus_cache* cache, const int32_t* table, int table_cols, const int32_t* lens,
                                int B, int start, int L, focus_bf16* K, focus_bf16* V, void* stream) {
  FOCUS_CHECK_ARG(K && V && lens, "null pointer argument");
  if (const int st = check_cache(cache, table, table_cols, false)) return st;
  FOCUS_CHECK_ARG(B >= 0 && L >= 1 && start >= 0 && static_cast<long long>(start) + L < (1LL << 31),
                  "bad sizes (B=%d start=%d L=%d)", B, start, L);
  FOCUS_CHECK_ARG(aligned16(K) && aligned16(V), "tensors must be 16-byte aligned");
  const long long units = static_cast<long long>(cache->n_mat) * B;
  if (units == 0) return FOCUS_OK;
  if (const int st = check_grid(units, cache->Hkv, "cache_load")) return st;
  RowArgs a = row_args(cache, table, table_cols, lens, B);
  a.out[0] = reinterpret_cast<uint4*>(K);
  a.out[1] = reinterpret_cast<uint4*>(V);
  a.start = start;
  a.L = L;
  const long long vecs = static_cast<long long>(L) << a.vec_shift;
  const int per = kLoadThreads * kLoadVecs;
  auto kern = cache->format == FOCUS_CACHE_E4M3 ? cache_load_kernel<FOCUS_CACHE_E4M3> : cache_load_kernel<FOCUS_CACHE_INT8>;
  return launched(launch_k(kern, dim3(static_cast<unsigned>((vecs + per - 1) / per), 2 * a.H, static_cast<unsigned>(units)),
                           dim3(kLoadThreads), 0, static_cast<cudaStream_t>(stream), a),
                  "cache_load");
}

extern "C" int focus_pages_copy(const focus_cache* cache, const int32_t* pairs, const int32_t* n_pairs, int pair_cap,
                                void* stream) {
  FOCUS_CHECK_ARG(pairs && n_pairs && pair_cap >= 0, "null pointer argument");
  if (const int st = check_cache(cache, pairs, 2, false)) return st;
  if (cache->n_mat == 0 || pair_cap == 0) return FOCUS_OK;
  const long long page_vecs = static_cast<long long>(cache->Hkv) * cache->page * cache->d / 16;
  const long long most = static_cast<long long>(pair_cap) * cache->n_mat * (2 * ((page_vecs + 1023) / 1024) + 1);
  const long long grid = std::min<long long>(most, static_cast<long long>(device_sm_count()) * 8);
  if (most + grid >= (1LL << 31)) {              // (a CTA's next piece, too, is counted in 32 bits)
    set_error("pages_copy: %d pairs of %d layers are too many for one call", pair_cap, cache->n_mat);
    return FOCUS_ERR_UNSUPPORTED;
  }
  return launched(launch_k(pages_copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(kCopyThreads), 0,
                           static_cast<cudaStream_t>(stream), static_cast<uint4*>(cache->k),
                           static_cast<uint4*>(cache->v), cache->k_scale, cache->v_scale, cache->n_mat, cache->n_pages,
                           cache->Hkv, page_vecs, pairs, n_pairs, pair_cap, device_error_word()),
                  "pages_copy");
}
