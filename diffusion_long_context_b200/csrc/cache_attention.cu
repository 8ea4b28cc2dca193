// Attention of few queries over the 8-bit paged cache, on the sm_100a tensor cores.
//
// Bound by the bytes of the codes: 2 d per key and head, against 4 d operations per key and
// query. So the codes go into the tensor cores as they are, and the other operands are brought
// to 8 bits without losing what bf16 holds:
//   * a query row is the sum of two 8-bit rows, hi + lo. e4m3: scaled by a power of two so that
//     its largest element lies in [128, 256), rounded to e4m3, and the rest rounded again; both
//     carry 4 bits, together the 8 of a bf16 (elements below 2^-9 of the largest keep less, but
//     never worse than 2^-17 of it). int8: 15-bit fixed point, hi * 128 + lo.
//   * a probability the same way: p in [0, 1] as e4m3 hi + lo of 256 p (error 2^-8 p, or 2^-18),
//     or as hi * 128 + lo of 16256 p (error 2^-15). With one 8-bit number only, a probability
//     would be off by 2^-4, far above what a bf16 result shows.
// The keys of a tile of 128 are the M side, the queries the N side (swap-AB):
//   S^T[key, q] = K_tile . Q^T        (M = 128 keys, N = queries, K = d)
//   O^T[dim, q] = V_tile^T . P^T      (M = d,        N = queries, K = 128 keys)
// hi and lo stand side by side in N, so a product of both is one MMA and their sums are added
// when they are read (as two MMAs into one accumulator, which e4m3 could do, a tile took 1550
// cycles of MMA instead of half that: at these widths an MMA costs about 100 cycles whatever
// its N). V_tile^T is the row-major tile and P^T the rows of a key each, both MN-major.
//
// Scales: a key's scale multiplies its row of S^T (a thread owns a key). A value's scale goes
// into P, relative to the largest of the tile, and that largest into the sum of O over tiles,
// which is kept in registers (a thread owns a dim): O^T of a tile is read back from tensor
// memory and added with the factors that bring it to the running maximum.
//
// Work is cut evenly: the 128-key tiles of all (sequence, KV head, slice of query rows) in a
// row, gridDim.x contiguous shares of them, one CTA per SM. A share that begins or ends inside
// a unit leaves (m, l, O) of its part in the workspace; cache_combine_kernel joins those and
// writes zeros for the units without keys. So one long sequence among short ones still fills
// the GPU, and a sequence's length is only read on the device.
//
// Warps: 0-3 and 4-7 two softmax groups, 8 producer (TMA for pages, cp.async for sink rows),
// 9 tcgen05.mma issuer and TMEM owner, 10-11 query rows. Up to 32 query rows the two groups
// take tiles in turn, each with its own running maximum, and join at the end of a unit; with
// 64 rows both work on every tile, 32 columns each.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "cache.cuh"

namespace focus {
namespace {

constexpr int kThreads = 384;
constexpr int kProducer = 8, kMma = 9, kQuery = 10;
constexpr int kMaxList = 1024;          // sinks, kept blocks
constexpr int kDescs = 4;

struct CacheAttnArgs {
  const __nv_bfloat16* Q;
  const int32_t* n_q;
  const uint8_t* code[2];
  const float* scale[2];
  const int32_t* table;
  const int32_t* lens;       // dense
  const int32_t* P;          // sparse
  const int32_t* g0;
  const int32_t* sinks;
  const int32_t* blocks;
  __nv_bfloat16* O;
  float* part_o;             // [2 grid][NQ][d]
  float2* part_ml;           // [2 grid][NQ]
  int table_cols, n_pages, page, B, Hq, Hkv, g, qcap, G, S, C;
  int n_slices, slice_rows;  // the g * qcap query rows of a KV head in slices
  int grid;
  float scale_log2;          // |scale| log2(e); the sign goes into the queries
  int negative;
  int* dev_err;
};

// ------------------------------------------------------------------ tiles of a unit
// The key slots of a unit are whole pages, then sinks one by one; a tile is 128 of them.
struct Sequence {
  int tiles;
  int n_pages;          // page slots
  int gs, ge, P, n_gen; // sparse: current block [gs, ge), prompt, its pages
  int len;              // dense
};

template <bool SPARSE>
__device__ __forceinline__ Sequence sequence_of(const CacheAttnArgs& a, int b) {
  Sequence s{};
  const int top = a.table_cols * a.page;
  if (SPARSE) {
    const int g0 = a.g0[b];
    s.gs = max(0, min(g0, top));
    s.ge = static_cast<int>(max(0LL, min(static_cast<long long>(g0) + a.G, static_cast<long long>(top))));
    s.P = max(0, min(a.P[b], s.gs));
    s.n_gen = s.ge > s.gs ? (s.ge - 1) / a.page - s.gs / a.page + 1 : 0;
    s.n_pages = s.n_gen + a.C;
    s.tiles = (s.n_pages * a.page + a.S + 127) >> 7;
  } else {
    s.len = max(0, min(a.lens[b], top));
    s.n_pages = (s.len + a.page - 1) / a.page;
    s.tiles = (s.len + 127) >> 7;
  }
  return s;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Tiles of the units of one head slice of all sequences (a warp; the same in every lane).
template <bool SPARSE>
__device__ __forceinline__ int tiles_of_all(const CacheAttnArgs& a) {
  int n = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) n += warp_sum(b0 + lane_id() < a.B ? sequence_of<SPARSE>(a, b0 + lane_id()).tiles : 0);
  return n;
}

// Tiles of sequences before b.
template <bool SPARSE>
__device__ __forceinline__ int tiles_before(const CacheAttnArgs& a, int b) {
  int n = 0;
  for (int b0 = 0; b0 < b; b0 += 32) n += warp_sum(b0 + lane_id() < b ? sequence_of<SPARSE>(a, b0 + lane_id()).tiles : 0);
  return n;
}

// Share i of `shares` contiguous shares of T tiles begins at tile i * T / shares.
__device__ __forceinline__ int share_begin(int i, int T, int shares) {
  return static_cast<int>(static_cast<long long>(i) * T / shares);
}
// The share that tile x falls in.
__device__ __forceinline__ int share_of(int x, int T, int shares) {
  return static_cast<int>((static_cast<long long>(x + 1) * shares - 1) / T);
}

// ------------------------------------------------------------------ shared memory
struct Desc {               // a run of tiles of one unit that this CTA works on
  int n;                    // tiles, 0 = the end
  int j0;                   // number of the first, counted over the CTA's runs
  int b, kvh, row0, rows, nq;
  int slot;                 // where the partial result goes, -1 = straight into O
};

template <int NQ, int STAGES>
struct __align__(16) Book {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t s_full[4], p_full[2], o_full[2];
  uint64_t q_full[2], q_empty[2];
  uint64_t d_full[kDescs], d_empty[kDescs];
  uint64_t x_full, x_done, drain;
  uint32_t tmem_base;
  int abort_flag;
  Desc desc[kDescs];
  // (arrays that are read four floats at a time start on 16 bytes)
  alignas(16) float2 key[STAGES][128];  // (scale of the key, factor of the value relative to the tile's largest)
  alignas(16) uint8_t valid[STAGES][128];
  float vmax[STAGES];                   // largest scale of a value in the tile
  int masked[STAGES];                   // some key of the tile is masked
  float q_scale[2][NQ];
  float red[2][2][4][32];               // [group][parity][warp][column]
  alignas(16) float2 pre[8][32];        // [warp][column]: (query scale, -reference)
  alignas(16) float be[8][32];          // [warp][column]: factor of the tile's row sum
  alignas(16) float post[8][2][32];     // [warp][buffer][column]: factor of the tile's O
  alignas(16) float2 xml[2][32];        // (m, l) of the other group's columns
  int blk[kMaxList], snk[kMaxList];
};

template <int FMT, int D, int NQ>
struct Lay {
  static constexpr int kStages = NQ == 64 ? 4 : 5;
  static constexpr uint32_t kTile = 128 * D;                       // bytes of a K or V tile
  static constexpr uint32_t kQ = kStages * 2 * kTile;              // 2 buffers of hi, lo rows
  static constexpr uint32_t kQBuf = 2 * NQ * D;
  static constexpr uint32_t kP = kQ + 2 * kQBuf;
  static constexpr uint32_t kPRow = 2 * NQ;                        // bytes of a key's row of P: hi, lo
  static constexpr uint32_t kPBuf = 128 * kPRow;
  static constexpr uint32_t kBook = kP + 2 * kPBuf;
  static constexpr uint32_t kBytes = kBook + sizeof(Book<NQ, kStages>) + 1024;
  static constexpr int kAcc = 2 * NQ;                              // accumulator columns of a product: hi, lo
  static constexpr int kS = NQ == 64 ? 2 : 4;                      // buffers of S^T
  static constexpr uint32_t kTmemUsed = (kS + 2) * kAcc;
  static constexpr uint32_t kTmem = kTmemUsed <= 256 ? 256 : 512;
  static_assert(kBytes <= 232448, "exceeds the 227 KB of shared memory per CTA");
  static_assert(kTmemUsed <= 512, "exceeds tensor memory");
  using Bk = Book<NQ, kStages>;
  static_assert(kBook % 16 == 0 && alignof(Bk) == 16, "shared-memory alignment");
};

// ------------------------------------------------------------------ small pieces
// Byte offset of 16-byte chunk c of row r of a tile whose rows are W bytes, in the swizzle of
// that width (128, 64 or 32 bytes) that the copies and the tensor cores use: bits 4 and up of
// the address are combined with bits 7 and up.
template <int W>
__device__ __forceinline__ uint32_t row_chunk(int r, int c) {
  static_assert(W == 128 || W == 64 || W == 32, "row width");
  const int x = W == 128 ? (r & 7) : W == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
  return static_cast<uint32_t>(r * W + ((c ^ x) << 4));
}

// Matrix descriptor of such a tile (8-row groups every 8 * W bytes), for a K-major operand whose
// K is the row's bytes and for an MN-major one whose K is the rows. For the MN-major read of V
// with d = 64, M = 128 needs two 64-wide columns of atoms: a leading stride of 0 reads the one
// there is twice (dims 64 .. 127 of O^T repeat 0 .. 63 and are not used).
template <int W>
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr) {
  const uint64_t layout = W == 128 ? 2ull : W == 64 ? 4ull : 6ull;   // SWIZZLE_128B, _64B, _32B
  const uint64_t leading = W == 128 ? 1ull : 0ull;     // not used where one column of atoms is all there is
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (leading << 16) |
         (static_cast<uint64_t>((8 * W) >> 4) << 32) | (1ull << 46) | (layout << 61);
}

template <int FMT>
__device__ constexpr uint32_t idesc8(int N, bool mn_major) {
  // D format (1 = f32, 2 = s32) | A, B format (e4m3 = 0 of kind::f8f6f4, s8 = 1 of kind::i8)
  const uint32_t d = FMT == FOCUS_CACHE_E4M3 ? 1u : 2u, f = FMT == FOCUS_CACHE_E4M3 ? 0u : 1u;
  return (d << 4) | (f << 7) | (f << 10) | ((mn_major ? 3u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (128u >> 4 << 24);
}

template <int FMT>
__device__ __forceinline__ void mma8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                     uint32_t accumulate) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// Largest of a float over the warp, NaN if any is NaN.
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 1 in one lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e;
}

// n arrivals at once.
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// Whether phase `parity` is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// hi and lo of four probabilities p times f (256 for e4m3, 16256 for int8, times the value's
// relative scale), a byte each, column 0 lowest.
template <int FMT>
__device__ __forceinline__ void split4(const float (&p)[4], float f, uint32_t& hi, uint32_t& lo) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // in half precision: 11 bits hold p to 2^-12, and p - hi is exact
      const __half2 x = __floats2half2_rn(p[2 * i] * f, p[2 * i + 1] * f);
      h[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
      const __half2 r = __hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h[i]), __NV_E4M3)));
      l[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E4M3);
    }
    hi = __byte_perm(h[0], h[1], 0x5410);
    lo = __byte_perm(l[0], l[1], 0x5410);
  } else {
    // v = round(p f) + 64 by adding 1.5 * 2^23 + 64: v = 128 hi + (lo + 64) with lo + 64 in
    // [0, 128), in the low 15 bits of the sum
    uint32_t h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __float_as_uint(fmaf(p[2 * i], f, 12582976.f)), b = __float_as_uint(fmaf(p[2 * i + 1], f, 12582976.f));
      const uint32_t w = __byte_perm(a, b, 0x5410);
      h[i] = (w >> 7) & 0x00ff00ffu;
      l[i] = (w & 0x007f007fu) + 0x00c000c0u;      // lo mod 256 in bits 0-7 and 16-23
    }
    hi = __byte_perm(h[0], h[1], 0x6420);
    lo = __byte_perm(l[0], l[1], 0x6420);
  }
}

// The product of hi and lo from their accumulators.
template <int FMT>
__device__ __forceinline__ float both(uint32_t hi, uint32_t lo) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) return __uint_as_float(hi) + __uint_as_float(lo);
  else return static_cast<float>(static_cast<int>(hi) * 128 + static_cast<int>(lo));
}

template <int FMT>
constexpr float prob_top() {
  return FMT == FOCUS_CACHE_E4M3 ? 256.f : 16256.f;
}

// Query q of the slice (head kvh * g + r / qcap, row r % qcap of r = row0 + q) as hi and lo rows
// of the K-major B operand: a warp, rows first, first + step, ...
template <int FMT, int D, int NQ>
__device__ __noinline__ void split_queries(const CacheAttnArgs& a, const Desc& d, uint8_t* dst, float* q_scale, int first,
                                           int step) {
  constexpr int E = D / 32;                  // elements of a lane
  constexpr int UN = 4;                      // rows in flight
  const int lane = lane_id();
  for (int q0 = first; q0 < NQ; q0 += step * UN) {
    float x[UN][E];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int q = q0 + step * i, r = d.row0 + q;
      const int qh = r / a.qcap, qi = r - qh * a.qcap;
      const bool real = q < d.rows && qi < d.nq;
      const __nv_bfloat16* src = a.Q + ((static_cast<size_t>(d.b) * a.Hq + d.kvh * a.g + qh) * a.qcap + qi) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        uint32_t w = 0u;
        if (real) w = __ldg(reinterpret_cast<const uint32_t*>(src) + e / 2);
        x[i][e] = __uint_as_float(w << 16);
        x[i][e + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int q = q0 + step * i;
      if (q >= NQ) break;
      float m = 0.f;
      bool bad = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        m = fmaxf(m, fabsf(x[i][e]));
        bad |= !(fabsf(x[i][e]) <= 3.4e38f);
      }
      m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
      bad = __any_sync(0xffffffffu, bad);
      float back;                            // what a unit of the row's codes stands for
      uint32_t hi = 0, lo = 0;
      if constexpr (FMT == FOCUS_CACHE_E4M3) {
        // power of two that brings the largest element into [128, 256), from its exponent bits
        const int ex = m > 0.f ? max(-120, min(120, 7 - (static_cast<int>(__float_as_uint(m) >> 23) - 127))) : 0;
        const float up = __int_as_float((127 + ex) << 23);
        back = __int_as_float((127 - ex) << 23);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float y0 = (a.negative ? -x[i][e] : x[i][e]) * up, y1 = (a.negative ? -x[i][e + 1] : x[i][e + 1]) * up;
          const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
          const float2 hf = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
          hi |= static_cast<uint32_t>(h) << (8 * e);
          lo |= static_cast<uint32_t>(
                    __nv_cvt_float2_to_fp8x2(make_float2(y0 - hf.x, y1 - hf.y), __NV_SATFINITE, __NV_E4M3))
                << (8 * e);
        }
      } else {
        const float up = m > 1e-30f ? 16256.f / m : 0.f;
        back = m > 1e-30f ? m / 16256.f : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int v = __float2int_rn((a.negative ? -x[i][e] : x[i][e]) * up), vh = (v + 64) >> 7;
          hi |= static_cast<uint32_t>(vh & 0xff) << (8 * e);
          lo |= static_cast<uint32_t>((v - (vh << 7)) & 0xff) << (8 * e);
        }
      }
      const uint32_t at = row_chunk<D>(q, lane * E / 16) + (lane * E & 15);
      if constexpr (E == 4) {
        *reinterpret_cast<uint32_t*>(dst + at) = hi;
        *reinterpret_cast<uint32_t*>(dst + NQ * D + at) = lo;
      } else {
        *reinterpret_cast<uint16_t*>(dst + at) = static_cast<uint16_t>(hi);
        *reinterpret_cast<uint16_t*>(dst + NQ * D + at) = static_cast<uint16_t>(lo);
      }
      if (lane == 0) q_scale[q] = bad ? NAN : back * a.scale_log2;
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int FMT, int D, int NQ, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CacheAttnArgs a) {
  using SM = Lay<FMT, D, NQ>;
  constexpr int STAGES = SM::kStages;
  constexpr bool kBoth = NQ == 64;               // both groups work on every tile
  constexpr int NC = kBoth ? 32 : NQ;            // columns of a softmax thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  auto* bk = reinterpret_cast<Book<NQ, STAGES>*>(smem + SM::kBook);
  volatile int* abort_flag = &bk->abort_flag;
  const int warp = warp_id(), lane = lane_id();

  if (warp == kProducer && lane == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bk->full[i], 2);                // the copies' bytes, the keys' scales
      mbar_init(&bk->empty[i], 1);
    }
    for (int i = 0; i < SM::kS; ++i) mbar_init(&bk->s_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bk->p_full[i], kBoth ? 8 : 4);
      mbar_init(&bk->o_full[i], 1);
      mbar_init(&bk->q_full[i], 10);             // the query and the softmax warps
      mbar_init(&bk->q_empty[i], 9);             // the last QK, and the softmax warps that read the scales
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&bk->d_full[i], 1);
      mbar_init(&bk->d_empty[i], 11);            // softmax, query and MMA warps
    }
    mbar_init(&bk->x_full, 8);
    mbar_init(&bk->x_done, 8);
    mbar_init(&bk->drain, 1);
    bk->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMma) {
    tmem_alloc(&bk->tmem_base, SM::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t tmem = bk->tmem_base;
  const uint32_t tS = tmem, tO = tmem + SM::kS * SM::kAcc;

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    const int all = tiles_of_all<SPARSE>(a);
    const int heads = a.Hkv * a.n_slices;
    const int T = all * heads;
    const int shares = min(static_cast<int>(gridDim.x), T);
    int issued = 0;                              // tiles whose copies are under way or done
    bool ok = true;
    int n_desc = 0;
    auto push = [&](const Desc& d) {             // lane 0 publishes a run
      const int s = n_desc % kDescs;
      if (n_desc >= kDescs)
        ok = __all_sync(0xffffffffu, mbar_wait(&bk->d_empty[s], ((n_desc / kDescs) - 1) & 1, abort_flag, a.dev_err,
                                               DEV_ERR_TIMEOUT_PRODUCER));
      if (!ok) return;
      if (lane == 0) {
        bk->desc[s] = d;
        mbar_arrive(&bk->d_full[s]);
      }
      __syncwarp();
      ++n_desc;
    };
    if (static_cast<int>(blockIdx.x) < shares) {
      const int t0 = share_begin(blockIdx.x, T, shares), t1 = share_begin(blockIdx.x + 1, T, shares);
      // the sequence that tile t0 falls in
      int b = 0, base = 0;                       // base: tiles of the sequences before b, all heads
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int n = b0 + lane < a.B ? sequence_of<SPARSE>(a, b0 + lane).tiles * heads : 0;
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > t0);
        if (past) {
          const int l = __ffs(past) - 1;
          b = b0 + l;
          base += __shfl_sync(0xffffffffu, incl - n, l);
          break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
      Sequence q = sequence_of<SPARSE>(a, b);
      const uint64_t policy = l2_evict_first_policy();
      const bool once = a.n_slices == 1;         // the codes are read by this unit alone
      const int ppt = 128 / a.page;              // pages of a tile
      const int32_t* trow = a.table + static_cast<size_t>(b) * a.table_cols;
      bool lists_sorted = true;
      int n_snk = 0;
      for (int t = t0; t < t1 && ok;) {
        while (q.tiles * heads <= t - base) {    // on to the next sequence that has tiles
          base += q.tiles * heads;
          ++b;
          q = sequence_of<SPARSE>(a, b);
          trow = a.table + static_cast<size_t>(b) * a.table_cols;
        }
        const int u = (t - base) / q.tiles;      // KV head and slice
        const int first = t - base - u * q.tiles, last = min(q.tiles, first + t1 - t);
        const int kvh = u / a.n_slices, slice = u - kvh * a.n_slices;
        Desc d;
        d.n = last - first;
        d.j0 = issued;
        d.b = b;
        d.kvh = kvh;
        d.row0 = slice * a.slice_rows;
        d.rows = min(a.slice_rows, a.g * a.qcap - d.row0);
        d.nq = a.n_q ? max(0, min(a.n_q[b], a.qcap)) : a.qcap;
        d.slot = d.n == q.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (first == 0 ? 1 : 0);
        push(d);
        if (!ok) break;
        t += d.n;

        if (SPARSE) {
          // the kept blocks: repeated entries are dropped (in an ascending list they are neighbours)
          const int32_t* blk = a.blocks + (static_cast<size_t>(b) * a.Hkv + kvh) * a.C;
          bool up = true;
          int before = -1;
          for (int i0 = 0; i0 < a.C; i0 += 32) {
            const int i = i0 + lane;
            const int v = i < a.C ? blk[i] : -1;
            const int prev = __shfl_up_sync(0xffffffffu, v, 1);
            const int pv = lane == 0 ? before : prev;
            up = up && (v < 0 || v > pv) && !(v >= 0 && pv < 0 && i > 0);
            if (i < a.C) bk->blk[i] = v;
            before = __shfl_sync(0xffffffffu, v, 31);
          }
          lists_sorted = __all_sync(0xffffffffu, up);
          __syncwarp();
          if (!lists_sorted) {
            // drop repeats, the later ones: entry by entry over the list, 32 at a time
            for (int i0 = (a.C - 1) & ~31; i0 >= 0; i0 -= 32) {
              const int i = i0 + lane;
              bool again = false;
              if (i < a.C)
                for (int j = 0; j < i && !again; ++j) again = bk->blk[j] == bk->blk[i];
              __syncwarp();
              if (again) bk->blk[i] = -1;
              __syncwarp();
            }
          }
          n_snk = -1;                            // the sinks are looked up when a tile needs them
        }
        // A batch of 32 page slots, one to a lane: what its table entry names, rows [lo, hi) of
        // it that are keys, and its scales. The next batch's table entries are requested a
        // batch ahead, its scales when the entries have come.
        struct Batch {
          int raw, lo, hi, pg;
          float ks, vs;
        };
        auto look_up = [&](int slot) {
          Batch x{-1, 0, 0, -1, 0.f, 0.f};
          int col = -1;
          if (!SPARSE) {
            if (slot < q.n_pages) {
              col = slot;
              x.hi = min(a.page, q.len - slot * a.page);
            }
          } else if (slot < q.n_gen) {
            col = q.gs / a.page + slot;
            x.lo = max(0, q.gs - col * a.page);
            x.hi = min(a.page, q.ge - col * a.page);
          } else if (slot < q.n_pages) {
            const int j = bk->blk[slot - q.n_gen];
            if (j >= 0 && j < a.table_cols && j * a.page < q.P) {
              col = j;
              x.hi = min(a.page, q.P - j * a.page);
            }
          }
          if (col >= 0) x.raw = trow[col];
          else x.hi = 0;
          return x;
        };
        auto resolve = [&](Batch& x) {
          if (x.hi > x.lo) {
            if (x.raw >= 0 && x.raw < a.n_pages) {
              x.pg = x.raw;
              const long long ph = static_cast<long long>(x.pg) * a.Hkv + kvh;
              x.ks = __ldg(a.scale[0] + ph);
              x.vs = __ldg(a.scale[1] + ph);
            } else {
              record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
              x.hi = x.lo;
            }
          }
        };
        if (SPARSE && lane == 0) {
          const long long g0 = a.g0[b];          // a current block that leaves the table
          if (g0 < 0 || g0 + a.G > static_cast<long long>(a.table_cols) * a.page) record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
        }
        if (!SPARSE && lane == 0 && a.lens[b] > a.table_cols * a.page) record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
        int bbase = first * ppt;
        Batch cur = look_up(bbase + lane);
        resolve(cur);
        for (int tile = first; tile < last && ok;) {
          const int b_end = min(last, (bbase + 32) / ppt);
          Batch nxt{-1, 0, 0, -1, 0.f, 0.f};
          if (b_end < last) nxt = look_up(bbase + 32 + lane);
          bool resolved = false;
          int done = tile;                       // tiles whose scales are published
          while (done < b_end && ok) {
            // copies of every tile of the batch that finds a free stage, at least one
            while (tile < b_end) {
              const int s = issued % STAGES;
              if (issued >= STAGES) {
                const uint32_t ph = ((issued / STAGES) - 1) & 1;
                bool got;
                if (tile == done) {
                  got = ok = __all_sync(0xffffffffu, mbar_wait(&bk->empty[s], ph, abort_flag, a.dev_err,
                                                               DEV_ERR_TIMEOUT_PRODUCER));
                } else {
                  got = __all_sync(0xffffffffu, mbar_test(&bk->empty[s], ph));
                }
                if (!got) break;
              }
              const int rel = bbase + lane - tile * ppt;             // this lane's page of the tile
              const bool mine = rel >= 0 && rel < ppt && cur.pg >= 0;
              const unsigned any = __ballot_sync(0xffffffffu, mine);
              if (lane == 0) mbar_arrive_expect_tx(&bk->full[s], static_cast<uint32_t>(__popc(any) * 2 * a.page * D));
              __syncwarp();
              if (mine) {
                const uint32_t dst = smem_u32(smem) + s * 2 * SM::kTile + rel * a.page * D;
                const int z = static_cast<int>(static_cast<long long>(cur.pg) * a.Hkv + kvh);
                if (once) {
                  tma_load_3d_hint(dst, &tmK, &bk->full[s], 0, 0, z, policy);
                  tma_load_3d_hint(dst + SM::kTile, &tmV, &bk->full[s], 0, 0, z, policy);
                } else {
                  tma_load_3d(dst, &tmK, &bk->full[s], 0, 0, z);
                  tma_load_3d(dst + SM::kTile, &tmV, &bk->full[s], 0, 0, z);
                }
              }
              __syncwarp();
              ++issued;
              ++tile;
            }
            if (!ok) break;
            for (; done < tile; ++done) {
              const int s = (issued - (tile - done)) % STAGES;
              // keys 4 lane .. 4 lane + 3 lie in one page slot, or among the sinks
              const int k0 = done * 128 + 4 * lane;
              const int slot = k0 / a.page, from = (slot - bbase) & 31;
              float ks[4], vs[4];
              bool on[4];
              {
                const int lo = __shfl_sync(0xffffffffu, cur.lo, from), hi = __shfl_sync(0xffffffffu, cur.hi, from);
                const float k = __shfl_sync(0xffffffffu, cur.ks, from), v = __shfl_sync(0xffffffffu, cur.vs, from);
                const int r = k0 - slot * a.page;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  on[e] = slot < q.n_pages && r + e >= lo && r + e < hi;
                  ks[e] = on[e] ? k : 0.f;
                  vs[e] = on[e] ? v : 0.f;
                }
              }
              if (SPARSE && done * 128 + 128 > q.n_pages * a.page) {
                if (n_snk < 0) {
                  // the sinks that no other slot holds: a sink is dropped inside the current
                  // block, inside a kept block, and when it was listed before
                  const int32_t* snk = a.sinks + (static_cast<size_t>(b) * a.Hkv + kvh) * a.S;
                  bool up = true;
                  int before = -1;
                  for (int i0 = 0; i0 < a.S; i0 += 32) {
                    const int v = i0 + lane < a.S ? snk[i0 + lane] : -1;
                    const int prev = __shfl_up_sync(0xffffffffu, v, 1);
                    const int pv = lane == 0 ? before : prev;
                    up = up && (v < 0 || v > pv) && !(v >= 0 && pv < 0 && i0 + lane > 0);
                    if (i0 + lane < a.S) bk->snk[i0 + lane] = v;
                    before = __shfl_sync(0xffffffffu, v, 31);
                  }
                  up = __all_sync(0xffffffffu, up);
                  __syncwarp();
                  for (int i0 = (a.S - 1) & ~31; i0 >= 0; i0 -= 32) {
                    const int i = i0 + lane, v = i < a.S ? bk->snk[i] : -1;
                    bool drop = v < 0 || (v >= q.gs && v < q.ge);
                    if (!up)
                      for (int j = 0; j < i && !drop; ++j) drop = bk->snk[j] == v;
                    if (!drop && v < q.P) {
                      const int col = v / a.page;
                      if (lists_sorted) {        // ascending, then -1
                        int lo = 0, hi = a.C;
                        while (lo < hi) {
                          const int mid = (lo + hi) >> 1, x = bk->blk[mid];
                          if (x >= 0 && x < col) lo = mid + 1;
                          else hi = mid;
                        }
                        drop = lo < a.C && bk->blk[lo] == col;
                      } else {
                        for (int j = 0; j < a.C && !drop; ++j) drop = bk->blk[j] == col;
                      }
                    }
                    __syncwarp();
                    if (drop && i < a.S) bk->snk[i] = -1;
                    __syncwarp();
                  }
                  n_snk = a.S;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int i = k0 + e - q.n_pages * a.page;
                  const int pos = i >= 0 && i < n_snk ? bk->snk[i] : -1;
                  if (pos < 0) continue;
                  const int pg = checked_page(a.table, a.table_cols, b, pos / a.page, a.n_pages, a.dev_err);
                  if (pg < 0) continue;
                  const long long ph = static_cast<long long>(pg) * a.Hkv + kvh;
                  on[e] = true;
                  ks[e] = __ldg(a.scale[0] + ph);
                  vs[e] = __ldg(a.scale[1] + ph);
                  const long long off = (ph * a.page + pos % a.page) * D;
                  const uint32_t dst = smem_u32(smem) + s * 2 * SM::kTile;
#pragma unroll
                  for (int c = 0; c < D / 16; ++c) {
                    cp_async16(dst + row_chunk<D>(4 * lane + e, c), a.code[0] + off + c * 16, 16);
                    cp_async16(dst + SM::kTile + row_chunk<D>(4 * lane + e, c), a.code[1] + off + c * 16, 16);
                  }
                }
                cp_async_wait_all();
                fence_proxy_async_smem();
              }
              float vm = fmaxf(fmaxf(fabsf(vs[0]), fabsf(vs[1])), fmaxf(fabsf(vs[2]), fabsf(vs[3])));
              if (vs[0] != vs[0] || vs[1] != vs[1] || vs[2] != vs[2] || vs[3] != vs[3]) vm = NAN;
              vm = warp_max_nan(vm);
              float2* key = &bk->key[s][4 * lane];
              const float c = vm == 0.f ? 0.f : prob_top<FMT>();
#pragma unroll
              for (int e = 0; e < 4; ++e) key[e] = make_float2(ks[e], vm == 0.f ? 0.f : vs[e] / vm * c);
              *reinterpret_cast<uchar4*>(&bk->valid[s][4 * lane]) = make_uchar4(on[0], on[1], on[2], on[3]);
              const bool part = !__all_sync(0xffffffffu, on[0] && on[1] && on[2] && on[3]);
              if (lane == 0) {
                bk->vmax[s] = vm / prob_top<FMT>();
                bk->masked[s] = part ? 1 : 0;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&bk->full[s]);
              if (!resolved && b_end < last) {
                resolve(nxt);
                resolved = true;
              }
            }
          }
          cur = nxt;
          bbase += 32;
        }
      }
    }
    if (ok) {
      Desc d{};
      push(d);
    }
    if (!ok) {
      // a wait ran out: the copies under way still have to land before the CTA may leave
      for (int j = max(0, issued - STAGES); j < issued; ++j) {
        const unsigned long long w0 = globaltimer();
        if (lane == 0) mbar_arrive(&bk->full[j % STAGES]);
        while (!mbar_try_wait(&bk->full[j % STAGES], (j / STAGES) & 1) && globaltimer() - w0 < 500000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp takes every step and one elected thread issues: the descriptors then stay
    // in uniform registers. (Inside a branch on lane == 0 an MMA cost 110 cycles to issue, with
    // the elected thread about 60.)
    const uint32_t elected = elect_one();
    const uint32_t id_qk = idesc8<FMT>(2 * NQ, false), id_pv = idesc8<FMT>(2 * NQ, true);
    const uint64_t k0 = tile_desc<D>(smem_u32(smem));
    const uint64_t q0 = tile_desc<D>(smem_u32(smem) + SM::kQ);
    const uint64_t p0 = tile_desc<SM::kPRow>(smem_u32(smem) + SM::kP);
    // QK runs ahead of PV by as many tiles as there are buffers of S^T; whichever product has its
    // operands goes next, so that neither a late tile holds up a finished P nor the other way.
    int di = -1, left = 0;                 // descriptor, tiles left in it
    int j_qk = 0, j_pv = 0;                // next tile of either product
    bool ended = false, fresh = false;     // no more tiles; the run's queries are still to come
    auto test = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0; };
    unsigned long long idle = 0;           // since when neither could go on
    while (!ended || j_pv < j_qk) {
      bool did = false;
      if (!ended && left == 0 && test(&bk->d_full[(di + 1) % kDescs], ((di + 1) / kDescs) & 1)) {
        if (di >= 0 && lane == 0) mbar_arrive(&bk->d_empty[di % kDescs]);
        ++di;
        left = bk->desc[di % kDescs].n;
        __syncwarp();
        ended = left == 0;
        fresh = true;
        did = true;
      }
      const int s = j_qk % STAGES;
      if (left > 0 && j_qk - j_pv < SM::kS && (!fresh || test(&bk->q_full[di & 1], (di >> 1) & 1)) &&
          test(&bk->full[s], (j_qk / STAGES) & 1)) {
        tc_fence_after();
        const int qb = di & 1, sb = j_qk % SM::kS;
        const uint64_t kd = k0 + static_cast<uint64_t>(s * 2 * SM::kTile / 16);
        const uint64_t qd = q0 + static_cast<uint64_t>(qb * SM::kQBuf / 16);
        fresh = false;
        --left;
        if (elected) {
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks)
            mma8<FMT>(tS + sb * SM::kAcc, kd + ks * 2, qd + ks * 2, id_qk, ks > 0 ? 1u : 0u);
          mma_commit(&bk->s_full[sb]);
          if (left == 0) mma_commit(&bk->q_empty[qb]);
        }
        __syncwarp();
        ++j_qk;
        did = true;
      }
      const int buf = j_pv & 1;
      if (j_pv < j_qk && test(&bk->p_full[buf], (j_pv >> 1) & 1)) {
        tc_fence_after();
        const int sv = j_pv % STAGES;
        const uint64_t vd = k0 + static_cast<uint64_t>((sv * 2 + 1) * SM::kTile / 16);
        const uint64_t pd = p0 + static_cast<uint64_t>(buf * SM::kPBuf / 16);
        if (elected) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma8<FMT>(tO + buf * SM::kAcc, vd + ks * (32 * D / 16), pd + ks * (32 * SM::kPRow / 16), id_pv, ks > 0 ? 1u : 0u);
          mma_commit(&bk->o_full[buf]);
          mma_commit(&bk->empty[sv]);
        }
        __syncwarp();
        ++j_pv;
        did = true;
      }
      if (did) {
        idle = 0;
      } else {
        const unsigned long long now = globaltimer();
        if (idle == 0) idle = now;
        bool stop = *abort_flag != 0;
        if (now - idle > kWaitLimitNs) {
          if (lane == 0) {
            *abort_flag = 1;
            record_dev_error(a.dev_err, DEV_ERR_TIMEOUT_MMA);
          }
          stop = true;
        }
        if (__any_sync(0xffffffffu, stop)) break;
      }
    }
    if (elected) mma_commit(&bk->drain);
    __syncwarp();
    const unsigned long long w0 = globaltimer();
    while (!mbar_try_wait(&bk->drain, 0) && globaltimer() - w0 < 500000000ull) {
    }
    __syncwarp();
  } else if (warp >= kQuery) {
    // ------------------------------------------------------------ query rows
    bool ok = true;
    for (int di = 0; ok; ++di) {
      const int ds = di % kDescs, qb = di & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&bk->d_full[ds], (di / kDescs) & 1, abort_flag, a.dev_err,
                                             DEV_ERR_TIMEOUT_PRODUCER));
      if (!ok) break;
      const Desc d = bk->desc[ds];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bk->d_empty[ds]);
      if (d.n == 0) break;
      if (di >= 2)
        ok = __all_sync(0xffffffffu, mbar_wait(&bk->q_empty[qb], ((di >> 1) - 1) & 1, abort_flag, a.dev_err,
                                               DEV_ERR_TIMEOUT_PRODUCER));
      if (!ok) break;
      // the first run's rows are shared with the softmax warps, which have nothing else to do yet
      split_queries<FMT, D, NQ>(a, d, smem + SM::kQ + qb * SM::kQBuf, bk->q_scale[qb], warp - kQuery, di == 0 ? 10 : 2);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_n(&bk->q_full[qb], di == 0 ? 1 : 5);
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    const int grp = warp >> 2, wq = warp & 3;
    const int t = threadIdx.x & 127;             // key of the tile == TMEM lane == dim of O^T
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const int c0 = kBoth ? grp * 32 : 0;         // first column
    const int bar = 1 + grp;
    const int lc = lane < NC ? lane : 0;         // the column whose maximum this lane follows
    bool ok = true;
    int n_x = 0;                                 // exchanges so far
    int par = 0;
    // A warp whose wait ran out goes on without waits or tensor memory to the next barrier of its
    // group, where the whole group leaves: the four warps always take the same barriers.
    for (int di = 0;; ++di) {
      const int ds = di % kDescs, qb = di & 1;
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait(&bk->d_full[ds], (di / kDescs) & 1, abort_flag, a.dev_err,
                                               DEV_ERR_TIMEOUT_SOFTMAX));
      Desc d{};
      if (ok) d = bk->desc[ds];
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bk->d_empty[ds]);
      if (ok && d.n > 0 && di == 0) {
        split_queries<FMT, D, NQ>(a, d, smem + SM::kQ, bk->q_scale[0], 2 + warp, 10);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bk->q_full[0]);
      }
      if (ok && d.n > 0)
        ok = __all_sync(0xffffffffu, mbar_wait(&bk->q_full[qb], (di >> 1) & 1, abort_flag, a.dev_err,
                                               DEV_ERR_TIMEOUT_SOFTMAX));
      if (bar_red_or(bar, 128, !ok) || d.n == 0) break;      // the whole group leaves together
      // (a zero query or scale: with the smallest normal number instead, every finite score is
      // still 0, and a masked key's -infinity stays what it is)
      const float qs_read = bk->q_scale[qb][c0 + lc];
      const float qs = qs_read == 0.f ? 1.17549435e-38f : qs_read;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bk->q_empty[qb]);
      // Sums over tiles are relative to 2^m_ref, which is the largest score of the run's first
      // tile and moves up only when another tile's is 2^30 times as large: fp32 has the range, and
      // no sum is rescaled tile by tile.
      float acc[NC], lsum[NC], m_ref = -INFINITY;
#pragma unroll
      for (int n = 0; n < NC; ++n) acc[n] = lsum[n] = 0.f;
      // adds O^T of tile j, in its buffer, to the sums
      auto collect = [&](int j) {
        const int buf = j & 1;
        if (ok)
          ok = __all_sync(0xffffffffu, mbar_wait(&bk->o_full[buf], (j >> 1) & 1, abort_flag, a.dev_err,
                                                 DEV_ERR_TIMEOUT_SOFTMAX));
        if (!ok) return;
        tc_fence_after();
        uint32_t r[NC], r2[NC];
        tmem_ld_cols<NC>(tO + buf * SM::kAcc + lane_addr + c0, r);
        tmem_ld_cols<NC>(tO + buf * SM::kAcc + NQ + lane_addr + c0, r2);
        tmem_ld_wait();
        const float4* f = reinterpret_cast<const float4*>(bk->post[warp][buf]);
#pragma unroll
        for (int n = 0; n < NC; n += 4) {
          const float4 v = f[n / 4];
          acc[n] += v.x * both<FMT>(r[n], r2[n]);
          acc[n + 1] += v.y * both<FMT>(r[n + 1], r2[n + 1]);
          acc[n + 2] += v.z * both<FMT>(r[n + 2], r2[n + 2]);
          acc[n + 3] += v.w * both<FMT>(r[n + 3], r2[n + 3]);
        }
        tc_fence_before();
      };
      const int jb = d.j0, je = d.j0 + d.n;
      constexpr int kStep = kBoth ? 1 : 2;
      const int j_first = kBoth ? jb : jb + ((jb ^ grp) & 1);
      bool left_early = false;
      for (int j = j_first; j < je; j += kStep) {
        const int buf = j & 1, s = j % STAGES, sb = j % SM::kS;
        if (j - 2 >= jb) collect(j - 2);
        if (ok)
          ok = __all_sync(0xffffffffu, mbar_wait(&bk->full[s], (j / STAGES) & 1, abort_flag, a.dev_err,
                                                 DEV_ERR_TIMEOUT_SOFTMAX));
        float2 key = make_float2(0.f, 0.f);
        bool on = true, masked = false;
        float vmax = 0.f;
        if (ok) {
          key = bk->key[s][t];
          masked = bk->masked[s] != 0;
          vmax = bk->vmax[s];
          if (masked) on = bk->valid[s][t] != 0;
          ok = __all_sync(0xffffffffu, mbar_wait(&bk->s_full[sb], (j / SM::kS) & 1, abort_flag, a.dev_err,
                                                 DEV_ERR_TIMEOUT_SOFTMAX));
        }
        float x[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) x[n] = 0.f;
        if (ok) {
          tc_fence_after();
          uint32_t r[NC], r2[NC];
          tmem_ld_cols<NC>(tS + sb * SM::kAcc + lane_addr + c0, r);
          tmem_ld_cols<NC>(tS + sb * SM::kAcc + NQ + lane_addr + c0, r2);
          tmem_ld_wait();
#pragma unroll
          for (int n = 0; n < NC; ++n) x[n] = both<FMT>(r[n], r2[n]) * key.x;
        }
        if (masked && !on) {
#pragma unroll
          for (int n = 0; n < NC; ++n) x[n] = -INFINITY;
        }
        // the largest of each column: over the warp, then over the group's four warps; lane n of
        // every warp follows column n
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const float m = warp_max_nan(x[n]);
          top[n & 3] = lane == n ? m : top[n & 3];
        }
        const float mine = (lane & 2) ? ((lane & 1) ? top[3] : top[2]) : ((lane & 1) ? top[1] : top[0]);
        par ^= 1;
        if (lane < NC) bk->red[grp][par][wq][lane] = mine;
        if (bar_red_or(bar, 128, !ok)) {
          left_early = true;
          break;
        }
        {
          const float* rd = &bk->red[grp][par][0][0];
          const float mt = max_nan(max_nan(rd[lc], rd[32 + lc]), max_nan(rd[64 + lc], rd[96 + lc]));
          const float ms = mt == -INFINITY ? -INFINITY : mt * qs;      // in units of log2
          // The tile's probabilities are relative to its own largest score. Against the running
          // maximum instead, all that lies 2^-18 below one large key (an attention sink) would be
          // rounded away, and with thousands of such keys a part of the result; so, no more than
          // 128 * 2^-18 of a tile's own largest is.
          float al = 1.f;
          if (ms > m_ref + 30.f || (m_ref == -INFINITY && ms > -INFINITY)) {
            al = exp2_approx(m_ref - ms);
            m_ref = ms;
          }
          const float be = ms == -INFINITY ? 0.f : exp2_approx(ms - m_ref);
          __syncwarp();                                                // the last tile's factors have been read
          if (__any_sync(0xffffffffu, al != 1.f)) {                    // the same in the group's four warps
            if (lane < NC) {
              bk->be[warp][lane] = al;
              bk->post[warp][buf ^ 1][lane] *= al;                     // a product that is still under way
            }
            __syncwarp();
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              const float f = bk->be[warp][n];
              lsum[n] *= f;
              acc[n] *= f;
            }
            __syncwarp();
          }
          if (lane < NC) {
            bk->pre[warp][lane] = make_float2(qs, ms == -INFINITY ? 0.f : -ms);
            bk->be[warp][lane] = be;
            bk->post[warp][buf][lane] = be * vmax;
          }
          __syncwarp();
        }
        const float4* pre = reinterpret_cast<const float4*>(bk->pre[warp]);
        const float4* pbe = reinterpret_cast<const float4*>(bk->be[warp]);
        // P is written as it is held, a key to a row, hi then lo: an MN-major operand. (Stored
        // query-major, a byte at a time, the stores alone took 1500 cycles of a tile.)
        uint8_t* pbuf = smem + SM::kP + buf * SM::kPBuf;
#pragma unroll
        for (int n0 = 0; n0 < NC; n0 += 16) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = n0 + 4 * i;
            const float4 e0 = pre[n / 2], e1 = pre[n / 2 + 1], be = pbe[n / 4];
            float p[4];
            p[0] = exp2_approx(x[n] * e0.x + e0.y);
            p[1] = exp2_approx(x[n + 1] * e0.z + e0.w);
            p[2] = exp2_approx(x[n + 2] * e1.x + e1.y);
            p[3] = exp2_approx(x[n + 3] * e1.z + e1.w);
            lsum[n] += p[0] * be.x;
            lsum[n + 1] += p[1] * be.y;
            lsum[n + 2] += p[2] * be.z;
            lsum[n + 3] += p[3] * be.w;
            split4<FMT>(p, key.y, hi[i], lo[i]);
          }
          *reinterpret_cast<uint4*>(pbuf + row_chunk<SM::kPRow>(t, (c0 + n0) / 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(pbuf + row_chunk<SM::kPRow>(t, (NQ + c0 + n0) / 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        // A masked key's values may be anything, NaN codes included, and 0 * NaN is NaN
        if (FMT == FOCUS_CACHE_E4M3 && masked && !on && (!kBoth || grp == 0)) {
          uint8_t* v = smem + (s * 2 + 1) * SM::kTile;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) *reinterpret_cast<uint4*>(v + row_chunk<D>(t, c)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bk->p_full[buf]);
      }
      if (left_early) break;
      // the products still under way: of this group's last tile, or of the last two
      {
        const int lastj = kBoth ? je - 1 : je - 1 - ((je - 1 - j_first) & 1);
        if (kBoth) {
          if (je - 2 >= jb) collect(je - 2);
          collect(je - 1);
        } else if (lastj >= j_first) {
          collect(lastj);
        }
      }
      // row sums over the 128 keys
      float l;
      {
        if constexpr (NC == 32) {
          warp_sum_scatter<32>(lsum);
          l = lsum[0];
        } else {
          warp_sum_scatter16(lsum);
          l = __shfl_sync(0xffffffffu, lsum[0], (2 * lane) & 31);
        }
        par ^= 1;
        if (lane < NC) bk->red[grp][par][wq][lane] = l;
        if (bar_red_or(bar, 128, !ok)) break;
        const float* rd = &bk->red[grp][par][0][0];
        l = (rd[lc] + rd[32 + lc]) + (rd[64 + lc] + rd[96 + lc]);
      }
      // Up to 32 rows: each group hands the other half of the columns over through the P
      // buffers, which no product reads any more once both groups have collected theirs.
      int n0 = 0;
      if constexpr (!kBoth) {
        constexpr int HC = NC / 2;
        float* xch = reinterpret_cast<float*>(smem + SM::kP);        // [group][HC][128]
        static_assert(2 * HC * 128 * 4 <= 2 * SM::kPBuf, "exchange exceeds the P buffers");
        // both groups are past their last product
        if (lane == 0) mbar_arrive(&bk->x_full);
        ok = __all_sync(0xffffffffu, mbar_wait(&bk->x_full, (2 * n_x) & 1, abort_flag, a.dev_err, DEV_ERR_TIMEOUT_EPILOGUE));
        if (bar_red_or(bar, 128, !ok)) break;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          const float v = grp == 0 ? acc[HC + i] : acc[i];
          xch[(grp * HC + i) * 128 + t] = v;
        }
        if (wq == 0 && lane < NC) bk->xml[grp][lane] = make_float2(m_ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bk->x_full);
        ok = __all_sync(0xffffffffu, mbar_wait(&bk->x_full, (2 * n_x + 1) & 1, abort_flag, a.dev_err, DEV_ERR_TIMEOUT_EPILOGUE));
        if (bar_red_or(bar, 128, !ok)) break;
        const float2 om = bk->xml[1 - grp][lc];
        const float M = max_nan(m_ref, om.x);
        const float ca = l == 0.f ? 0.f : exp2_approx(m_ref - M), cb = om.y == 0.f ? 0.f : exp2_approx(om.x - M);
        l = ca * l + cb * om.y;
        m_ref = M;
        n0 = grp * HC;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          const float fa = __shfl_sync(0xffffffffu, ca, n0 + i), fb = __shfl_sync(0xffffffffu, cb, n0 + i);
          const float v = grp == 0 ? acc[i] : acc[HC + i];
          acc[i] = fa * v + fb * xch[((1 - grp) * HC + i) * 128 + t];
        }
        if (lane == 0) mbar_arrive(&bk->x_done);
        ok = __all_sync(0xffffffffu, mbar_wait(&bk->x_done, n_x & 1, abort_flag, a.dev_err, DEV_ERR_TIMEOUT_EPILOGUE));
        ++n_x;
      }
      // out: columns n0 .. of the slice
      constexpr int OC = kBoth ? NC : NC / 2;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int i = 0; i < OC; ++i) {
        const int n = c0 + n0 + i;
        const float f = __shfl_sync(0xffffffffu, inv, n0 + i);
        if (n < d.rows && t < D) {
          if (d.slot >= 0) {
            a.part_o[(static_cast<size_t>(d.slot) * NQ + n) * D + t] = acc[i];
          } else {
            const int r = d.row0 + n, qh = r / a.qcap, qi = r - qh * a.qcap;
            const size_t row = (static_cast<size_t>(d.b) * a.Hq + d.kvh * a.g + qh) * a.qcap + qi;
            a.O[row * D + t] = __float2bfloat16_rn(qi < d.nq ? acc[i] * f : 0.f);
          }
        }
      }
      if (d.slot >= 0 && wq == 0 && lane >= n0 && lane < n0 + OC && c0 + lane < d.rows)
        a.part_ml[static_cast<size_t>(d.slot) * NQ + c0 + lane] = make_float2(m_ref, l);
    }
    if (!ok) bk->abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, SM::kTmem);
}

// Joins the parts of the units that several CTAs worked on (a warp per query row, a lane holds
// D / 32 dims): weights 2^(m - M) over the parts' (m, l), 32 parts at a time. Units without
// keys get zeros; units of one CTA are done already.
template <int D, bool SPARSE>
__global__ void __launch_bounds__(128) cache_combine_kernel(const CacheAttnArgs a, int NQ) {
  constexpr int E = D / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = lane_id();
  const int rows = a.g * a.qcap;                            // of a KV head
  const long long w = static_cast<long long>(blockIdx.x) * 4 + warp_id();
  if (w >= static_cast<long long>(a.B) * a.Hkv * rows) return;
  const int bh = static_cast<int>(w / rows), r = static_cast<int>(w - static_cast<long long>(bh) * rows);
  const int b = bh / a.Hkv, kvh = bh - b * a.Hkv, slice = r / a.slice_rows, n = r - slice * a.slice_rows;
  const Sequence q = sequence_of<SPARSE>(a, b);
  const int heads = a.Hkv * a.n_slices;
  const int qh = r / a.qcap, qi = r - qh * a.qcap;
  __nv_bfloat16* O = a.O + ((static_cast<size_t>(b) * a.Hq + kvh * a.g + qh) * a.qcap + qi) * D + lane * E;
  const int nq = a.n_q ? max(0, min(a.n_q[b], a.qcap)) : a.qcap;
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  float l = 0.f;
  if (q.tiles > 0) {
    const int T = tiles_of_all<SPARSE>(a) * heads;
    const int shares = min(a.grid, T);
    const int x0 = tiles_before<SPARSE>(a, b) * heads + (kvh * a.n_slices + slice) * q.tiles;
    const int s0 = share_of(x0, T, shares), s1 = share_of(x0 + q.tiles - 1, T, shares);
    if (s0 == s1) return;
    float M = -INFINITY;
    for (int c0 = s0; c0 <= s1; c0 += 32) {
      const int c = c0 + lane;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (c <= s1) ml = a.part_ml[(static_cast<size_t>(2 * c) + (c == s0 ? 1 : 0)) * NQ + n];
      const float mn = max_nan(M, warp_max_nan(ml.x));
      const float back = l == 0.f ? 0.f : exp2_approx(M - mn);
      const float f = ml.y == 0.f ? 0.f : exp2_approx(ml.x - mn);
      float lw = f * ml.y;
#pragma unroll
      for (int off = 16; off; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
      l = l * back + lw;
      M = mn;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= back;
      const int cn = min(32, s1 - c0 + 1);
#pragma unroll 8
      for (int i = 0; i < cn; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        const float* src = a.part_o + ((static_cast<size_t>(2 * (c0 + i)) + (c0 + i == s0 ? 1 : 0)) * NQ + n) * D + lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          o[0] += fi * v.x;
          o[1] += fi * v.y;
          o[2] += fi * v.z;
          o[3] += fi * v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          o[0] += fi * v.x;
          o[1] += fi * v.y;
        }
      }
    }
  }
  const float inv = (qi < nq && l != 0.f) ? 1.f / l : 0.f;
  const bool real = qi < nq;
  uint32_t pk[E / 2];
#pragma unroll
  for (int e = 0; e < E; e += 2) pk[e / 2] = real ? pack_bf16x2(o[e] * inv, o[e + 1] * inv) : 0u;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(O) = make_uint2(pk[0], pk[1]);
  else *reinterpret_cast<uint32_t*>(O) = pk[0];
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Codes as [n_pages * Hkv] pages of [page, d] bytes; a box is one page of one head.
int page_map(CUtensorMap* map, const void* base, const focus_cache* c) {
  auto fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is unavailable (driver entry point lookup failed)");
    return FOCUS_ERR_CUDA;
  }
  const cuuint64_t d = c->d, page = c->page;
  cuuint64_t dims[3] = {d, page, static_cast<cuuint64_t>(c->n_pages) * c->Hkv};
  cuuint64_t strides[2] = {d, d * page};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(page), 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        c->d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
    return FOCUS_ERR_CUDA;
  }
  return FOCUS_OK;
}

// Query rows a CTA works on: 16 for single tokens of grouped heads, 32 for a step's active rows,
// 64 where a KV head has more (each slice reads the codes again, from L2).
int rows_per_cta(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int FMT, int D, int NQ, bool SPARSE>
int launch_attention(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnArgs& a, cudaStream_t stream) {
  auto kern = cache_attn_kernel<FMT, D, NQ, SPARSE>;
  constexpr int bytes = static_cast<int>(Lay<FMT, D, NQ>::kBytes);
  if (const int st = configure_dynamic_smem(reinterpret_cast<const void*>(kern), bytes, "cache attention")) return st;
  cudaError_t e = launch_k(kern, dim3(a.grid), dim3(kThreads), bytes, stream, mk, mv, a);
  note_launch();
  if (e == cudaSuccess) {
    const long long rows = static_cast<long long>(a.B) * a.Hkv * a.g * a.qcap;
    e = launch_k(cache_combine_kernel<D, SPARSE>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream, a, NQ);
    note_launch();
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("cache attention launch: %s", cudaGetErrorString(e));
    return FOCUS_ERR_CUDA;
  }
  return FOCUS_OK;
}

template <int FMT, int D, bool SPARSE>
int launch_rows(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnArgs& a, cudaStream_t stream) {
  switch (rows_per_cta(a.g * a.qcap)) {
    case 16: return launch_attention<FMT, D, 16, SPARSE>(mk, mv, a, stream);
    case 32: return launch_attention<FMT, D, 32, SPARSE>(mk, mv, a, stream);
    default: return launch_attention<FMT, D, 64, SPARSE>(mk, mv, a, stream);
  }
}

template <bool SPARSE>
int run_cache_attention(CacheAttnArgs a, const focus_cache* c, void* ws, cudaStream_t stream) {
  if (a.B == 0) return FOCUS_OK;
  const int rows = a.g * a.qcap, nq = rows_per_cta(rows);
  a.n_slices = (rows + nq - 1) / nq;
  a.slice_rows = (rows + a.n_slices - 1) / a.n_slices;
  // tiles at most, for the grid and for the 32-bit tile numbers
  const long long per_unit = SPARSE ? (static_cast<long long>((a.G + a.page - 2) / a.page + 1 + a.C) * a.page + a.S + 127) / 128
                                    : (static_cast<long long>(a.table_cols) * a.page + 127) / 128;
  const long long most = static_cast<long long>(a.B) * a.Hkv * a.n_slices * per_unit;
  if (most >= (1LL << 31) || static_cast<long long>(a.B) * a.Hkv * rows >= (1LL << 32)) {
    set_error("cache attention: %lld tiles of 128 keys in one call", most);
    return FOCUS_ERR_UNSUPPORTED;
  }
  const int sms = device_sm_count();
  a.grid = static_cast<int>(std::min<long long>(sms, most));
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(2) * sms * nq * c->d);
  CUtensorMap mk, mv;
  if (const int st = page_map(&mk, c->k, c)) return st;
  if (const int st = page_map(&mv, c->v, c)) return st;
  if (c->format == FOCUS_CACHE_E4M3)
    return c->d == 128 ? launch_rows<FOCUS_CACHE_E4M3, 128, SPARSE>(mk, mv, a, stream)
                       : launch_rows<FOCUS_CACHE_E4M3, 64, SPARSE>(mk, mv, a, stream);
  return c->d == 128 ? launch_rows<FOCUS_CACHE_INT8, 128, SPARSE>(mk, mv, a, stream)
                     : launch_rows<FOCUS_CACHE_INT8, 64, SPARSE>(mk, mv, a, stream);
}

int check_attention(const focus_bf16* Q, const focus_cache* cache, const int32_t* table, int table_cols, int B, int Hq,
                    int qcap, float scale, const focus_bf16* O, const void* ws, size_t ws_bytes) {
  FOCUS_CHECK_ARG(Q && O, "null pointer argument");
  if (const int st = check_cache(cache, table, table_cols, true)) return st;
  FOCUS_CHECK_ARG(B >= 0 && Hq >= 1 && qcap >= 1, "bad sizes (B=%d Hq=%d qcap=%d)", B, Hq, qcap);
  FOCUS_CHECK_ARG(Hq % cache->Hkv == 0, "Hq %d is not a multiple of Hkv %d", Hq, cache->Hkv);
  FOCUS_CHECK_ARG(static_cast<long long>(Hq) * qcap < (1LL << 30), "Hq * qcap must be below 2^30");
  FOCUS_CHECK_ARG(aligned16(Q) && aligned16(O), "tensors must be 16-byte aligned");
  FOCUS_CHECK_ARG(static_cast<long long>(table_cols) * cache->page < (1LL << 31), "table of 2^31 positions or more");
  FOCUS_CHECK_ARG(scale - scale == 0.f, "scale must be finite");
  const size_t need = focus_cache_workspace_bytes(B, Hq, cache->Hkv, cache->d, qcap);
  FOCUS_CHECK_ARG(ws, "null workspace (%zu bytes needed)", need);
  FOCUS_CHECK_ARG((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "workspace must be 256-byte aligned");
  if (ws_bytes < need) {
    set_error("workspace of %zu bytes, %zu needed", ws_bytes, need);
    return FOCUS_ERR_CAPACITY;
  }
  return FOCUS_OK;
}

CacheAttnArgs attn_args(const focus_bf16* Q, const int32_t* n_q, const focus_cache* c, const int32_t* table,
                        int table_cols, int B, int Hq, int qcap, float scale, focus_bf16* O) {
  CacheAttnArgs a{};
  a.Q = reinterpret_cast<const __nv_bfloat16*>(Q);
  a.n_q = n_q;
  a.code[0] = static_cast<const uint8_t*>(c->k);
  a.code[1] = static_cast<const uint8_t*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.table = table;
  a.table_cols = table_cols;
  a.n_pages = c->n_pages;
  a.page = c->page;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = c->Hkv;
  a.g = Hq / c->Hkv;
  a.qcap = qcap;
  a.O = reinterpret_cast<__nv_bfloat16*>(O);
  a.scale_log2 = (scale < 0.f ? -scale : scale) * 1.4426950408889634f;
  a.negative = scale < 0.f ? 1 : 0;
  a.dev_err = device_error_word();
  return a;
}

}  // namespace
}  // namespace focus

using namespace focus;

extern "C" size_t focus_cache_workspace_bytes(int B, int Hq, int Hkv, int d, int qcap) {
  if (B <= 0 || Hkv < 1 || Hq < Hkv || d < 1 || qcap < 1) return 256;
  const size_t nq = rows_per_cta(static_cast<int>(std::min<long long>(static_cast<long long>(Hq / Hkv) * qcap, 1 << 20)));
  // two parts of each CTA: O [nq, d] fp32 and (m, l) [nq]
  return (static_cast<size_t>(2) * device_sm_count() * nq * (static_cast<size_t>(d) * 4 + 8) + 255) & ~static_cast<size_t>(255);
}

extern "C" int focus_cache_attention(const focus_bf16* Q, const int32_t* n_q, const focus_cache* cache,
                                     const int32_t* table, int table_cols, const int32_t* lens, int B, int Hq,
                                     int qcap, float scale, focus_bf16* O, void* ws, size_t ws_bytes, void* stream) {
  if (const int st = check_attention(Q, cache, table, table_cols, B, Hq, qcap, scale, O, ws, ws_bytes)) return st;
  FOCUS_CHECK_ARG(lens, "null pointer argument");
  CacheAttnArgs a = attn_args(Q, n_q, cache, table, table_cols, B, Hq, qcap, scale, O);
  a.lens = lens;
  return run_cache_attention<false>(a, cache, ws, static_cast<cudaStream_t>(stream));
}

extern "C" int focus_cache_sparse_attention(const focus_bf16* Q_active, const int32_t* n_active,
                                            const focus_cache* cache, const int32_t* table, int table_cols,
                                            const int32_t* P, const int32_t* g0, int G, const int32_t* sinks, int S,
                                            const int32_t* blocks, int C, int B, int Hq, int qcap, float scale,
                                            focus_bf16* O_active, void* ws, size_t ws_bytes, void* stream) {
  if (const int st = check_attention(Q_active, cache, table, table_cols, B, Hq, qcap, scale, O_active, ws, ws_bytes))
    return st;
  FOCUS_CHECK_ARG(P && g0 && blocks && (S == 0 || sinks), "null pointer argument");
  FOCUS_CHECK_ARG(G >= 1 && S >= 0 && C >= 1, "bad sizes (G=%d S=%d C=%d)", G, S, C);
  if (S > kMaxList || C > kMaxList) {
    set_error("cache sparse attention: S and C up to %d (got %d and %d)", kMaxList, S, C);
    return FOCUS_ERR_UNSUPPORTED;
  }
  CacheAttnArgs a = attn_args(Q_active, n_active, cache, table, table_cols, B, Hq, qcap, scale, O_active);
  a.P = P;
  a.g0 = g0;
  a.G = G;
  a.sinks = sinks;
  a.S = S;
  a.blocks = blocks;
  a.C = C;
  return run_cache_attention<true>(a, cache, ws, static_cast<cudaStream_t>(stream));
}
