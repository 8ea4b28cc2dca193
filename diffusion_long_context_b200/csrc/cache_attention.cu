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
// when they are read (as two MMAs into one accumulator, which e4m3 could do, a tile took twice
// the MMAs, and at these widths one costs about 55 cycles whatever its N). V_tile^T is the row-major tile and P^T the rows of a key each, both MN-major.
//
// Scales: a key's scale multiplies its row of S^T (a thread owns a key). A value's scale goes
// into P, relative to the largest of the tile (so 2^-18 of a tile's largest p times value scale
// is lost), and that largest into the sum of O over tiles, in fp32 in tensor memory: O^T of a
// tile is read back and added with the factor from the tile's reference to the run's.
//
// Work is cut evenly: the 128-key tiles of all (sequence, KV head, slice of query rows) in a
// row, gridDim.x contiguous shares of them, one CTA per SM. A share that begins or ends inside
// a unit leaves (m, l, O) of its part in the workspace; cache_combine_kernel joins those and
// writes zeros for the units without keys. So one long sequence among short ones still fills
// the GPU, and a sequence's length is only read on the device.
//
// Measured (graph replay): 32 heads of 32 rows over 32K keys 63 us, 4.3 TB/s of codes, and per
// doubling of the keys 5.4 TB/s (of 6.5 that a copy reaches); 9.6 us of it are there with a
// single tile: launch, page lookup, first bytes, the chain below, output, join. What bounds a
// long sequence is not one pipe or stage: a tile takes 4 to 5 us through memory and the chain,
// every stage idles for a third of the time, half of the issue slots are used, and more tiles under
// way than the four of keys and six of values in 160 KB (a ring of seven, or five of keys) gained
// nothing. Which hand-over sets the 1700 cycles a tile is not known.
//
// A tile goes through a chain of warps, each of which works on a tile of its own, so that the
// latencies of the hand-overs (mbarriers, tensor memory, shuffles: half of a tile's way) are
// covered by the other tiles (cycles a tile in parentheses, of 1700 at 32 rows over 32K keys):
//   16, 17  producers, a tile each in turn (TMA for pages, cp.async for sink rows)
//   18      issues S^T = K Q^T (330), and sets the references (590); owns tensor memory
//   0-3     the largest score of every column in each warp's 32 keys (760)
//   4-11    two groups, a tile each in turn: exp, row sums, hi and lo of P (2600 a tile of two)
//   19      issues O^T = V^T P^T (320)
//   12-15   sum of O^T over tiles (790); at the end of a unit, the output
// With one group taking a tile from its scores to its sum, and two such groups, a tile took 2200
// cycles, most of them latency. The loops over columns stay short (16 columns, rolled, with what
// lasts from tile to tile in tensor memory instead of registers): the stages run side by side on
// every scheduler, and unrolled over 32 columns their code, together, left the instruction cache
// (3.2 of 13 warp cycles per instruction waited for one, 1.2 of 9.6 as it is).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "cache.cuh"

namespace focus {
namespace {

constexpr int kMaxWarp = 0, kExpWarp = 4, kSumWarp = 12;      // first warps of the stages
constexpr int kSoftmaxWarps = 16;
constexpr int kProducers = 2;
constexpr int kProducer = kSoftmaxWarps, kMmaS = kProducer + kProducers, kMmaO = kMmaS + 1;
constexpr int kThreads = (kMmaO + 1) * 32;
constexpr int kQParts = kSoftmaxWarps;   // warps that prepare the first queries
constexpr int kMaxList = 1024;          // sinks, kept blocks
constexpr int kDescs = 4;
constexpr int kMasked = 1, kByKey = 2;
constexpr int kLead = 6;                // places of a unit before its first tile (see unit_length)

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
  int table_cols, n_pages, page, page_shift, B, Hq, Hkv, g, qcap, G, S, C;
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

// EARLY: before the wait for the kernels in front, past L1, which may hold what an earlier kernel read.
template <bool EARLY>
__device__ __forceinline__ int word(const int32_t* p) {
  if constexpr (EARLY) return __ldcg(p);
  else return *p;
}

template <bool SPARSE, bool EARLY = false>
__device__ __forceinline__ Sequence sequence_of(const CacheAttnArgs& a, int b) {
  Sequence s{};
  const int top = a.table_cols * a.page;
  if (SPARSE) {
    const int g0 = word<EARLY>(a.g0 + b);
    s.gs = max(0, min(g0, top));
    s.ge = static_cast<int>(max(0LL, min(static_cast<long long>(g0) + a.G, static_cast<long long>(top))));
    s.P = max(0, min(word<EARLY>(a.P + b), s.gs));
    s.n_gen = s.ge > s.gs ? ((s.ge - 1) >> a.page_shift) - (s.gs >> a.page_shift) + 1 : 0;
    s.n_pages = s.n_gen + a.C;
    s.tiles = (s.n_pages * a.page + a.S + 127) >> 7;
  } else {
    s.len = max(0, min(word<EARLY>(a.lens + b), top));
    s.n_pages = (s.len + a.page - 1) >> a.page_shift;
    s.tiles = (s.len + 127) >> 7;
  }
  return s;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Tiles lie on an axis on which every unit also takes kLead places before its first tile, for
// what a run costs beyond its tiles (page lists, query rows, filling and draining the chain,
// output): shares of equal length then take about as long, whether they hold one long unit or
// many short ones. With 2, 4, 6 places: kept blocks at 32K 28.5, 28.0, 26.7 us, sixteen ragged
// sequences 63, 57, 57 us, one sequence of 32K 64.5, 64.9, 64.6 us.
__device__ __forceinline__ int unit_length(int tiles) { return tiles > 0 ? tiles + kLead : 0; }

// Length of the axis for one head slice of all sequences (a warp; the same in every lane).
template <bool SPARSE, bool EARLY = false>
__device__ __forceinline__ int length_of_all(const CacheAttnArgs& a) {
  int n = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) n += warp_sum(b0 + lane_id() < a.B ? unit_length(sequence_of<SPARSE, EARLY>(a, b0 + lane_id()).tiles) : 0);
  return n;
}

// The part of it before sequence b.
template <bool SPARSE, bool EARLY>
__device__ __forceinline__ int length_before(const CacheAttnArgs& a, int b) {
  int n = 0;
  for (int b0 = 0; b0 < b; b0 += 32) n += warp_sum(b0 + lane_id() < b ? unit_length(sequence_of<SPARSE, EARLY>(a, b0 + lane_id()).tiles) : 0);
  return n;
}

// Share i of `shares` contiguous shares of an axis of length T begins at i * T / shares (without
// a 64-bit division, which is a few hundred cycles at the head of every call).
__device__ __forceinline__ int share_begin(int i, int T, int shares) {
  const unsigned n = static_cast<unsigned>(shares), whole = static_cast<unsigned>(T) / n;
  return static_cast<int>(i * whole + i * (T - whole * n) / n);
}
// The share that place x falls in.
__device__ __forceinline__ int share_of(int x, int T, int shares) {
  int s = min(shares - 1, static_cast<int>(__fdividef(static_cast<float>(x) * shares, static_cast<float>(T))));
  while (s > 0 && share_begin(s, T, shares) > x) --s;
  while (s + 1 < shares && share_begin(s + 1, T, shares) <= x) ++s;
  return s;
}

// ------------------------------------------------------------------ shared memory
struct Desc {               // a run of tiles of one unit that this CTA works on
  int n;                    // tiles, 0 = the end
  int j0;                   // number of the first, counted over the CTA's runs
  int b, kvh, row0, rows, nq;
  int slot;                 // where the partial result goes, -1 = straight into O
};

// Tiles in the rings of K and of V. A key tile is free once its scores are out, a value tile only
// after the way through the probabilities, so that takes more of them.
constexpr int kK = 4, kV = 6;
constexpr int kS = 4, kO = 2;           // buffers of S^T, of O^T
// Entries for what the later stages need to know of a tile. Tile j's may be overwritten by tile
// j + kE's without a wait: its score product waited for P of tile j + kE - kS, that for the
// product of P of tile j + kE - kS - 2, and that for the sums of tile j + kE - kS - 2 - kO.
constexpr int kE = kS + 2 + kO;

template <int NQ>
struct __align__(16) Book {
  uint64_t k_full[kK], k_empty[kK], v_full[kV], v_empty[kV];
  uint64_t s_full[kS], s_free[kS], t_full[kS], m_full[kS], o_full[kO], o_free[kO];
  uint64_t p_full[2];
  uint64_t q_full[2], q_empty[2];
  uint64_t d_full[kDescs], d_empty[kDescs];
  uint64_t x_full[2], x_done[2], drain[2];
  uint32_t tmem_base;
  int abort_flag;
  Desc desc[kDescs];
  // (arrays that are read four floats at a time start on 16 bytes)
  // scales of a tile: a page's (key scale, value scale relative to the tile's largest, first and
  // last row that are keys), or with sinks among them each key's
  alignas(16) float4 page[kV][8];
  alignas(16) float2 key[kV][128];
  alignas(16) uint8_t valid[kV][128];
  float vmax[kV];              // largest scale of a value in the tile
  int info[kV];                // kMasked: some key is masked, kByKey: scales key by key
  alignas(16) float q_scale[2][NQ];
  alignas(16) float top[kS][4][NQ];            // [S buffer][warp][column]: largest score, without the query's scale
  alignas(16) float qs[8][NQ];                 // [exp warp][column]: scale of the query
  // of a tile's columns, [entry][column]: -reference of its probabilities, the run's reference, and
  // the factor from one to the other, a power of two, in bf16
  alignas(16) float ref[kE][NQ], run[kE][NQ];
  alignas(16) uint16_t be[kE][NQ];
  float o_vmax[kE];                                // and its value scale
  float x_m[2][2][NQ], x_l[2][8][NQ];      // [run parity]: reference, row sums of the exp warps
  int blk[kProducers][kMaxList], snk[kProducers][kMaxList];   // a producer's lists of its unit
};

template <int FMT, int D, int NQ>
struct Lay {
  static constexpr uint32_t kTile = 128 * D;                       // bytes of a K or V tile
  static constexpr uint32_t kVRing = kK * kTile;
  static constexpr uint32_t kQ = kVRing + kV * kTile;              // 2 buffers of hi, lo rows
  static constexpr uint32_t kQBuf = 2 * NQ * D;
  static constexpr uint32_t kP = kQ + 2 * kQBuf;
  static constexpr uint32_t kPRow = 2 * NQ;                        // bytes of a key's row of P: hi, lo
  static constexpr uint32_t kPBuf = 128 * kPRow;
  static constexpr uint32_t kBook = kP + 2 * kPBuf;
  using Bk = Book<NQ>;
  static constexpr uint32_t kBytes = kBook + sizeof(Bk) + 1024;
  static constexpr int kAcc = 2 * NQ;                              // accumulator columns of a product: hi, lo
  static constexpr uint32_t kTmemUsed = (kS + kO) * kAcc + 3 * NQ;    // S^T, O^T, the sum of O^T, two of P's rows
  static constexpr uint32_t kTmem = kTmemUsed <= 256 ? 256 : 512;
  static_assert(kBytes <= 232448, "exceeds the 227 KB of shared memory per CTA");
  static_assert(kTmemUsed <= 512, "exceeds tensor memory");
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

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Largest of a float over the warp, NaN if any is NaN.
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// Waits for phase `parity` (a whole warp), in the barrier as long as the hardware suspends the
// thread (a wait that polls takes issue slots from the warps that have work); false when the
// limit runs out or another warp gave up.
__device__ __forceinline__ bool mbar_sleep(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* dev_err, int code) {
  const unsigned long long t0 = globaltimer();
  while (!__all_sync(0xffffffffu, mbar_sleep(bar, parity))) {
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    if (__any_sync(0xffffffffu, globaltimer() - t0 > kWaitLimitNs)) {
      *abort_flag = 1;
      if (lane_id() == 0) record_dev_error(dev_err, code);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* dev_err, int code) {
  if (__all_sync(0xffffffffu, mbar_sleep(bar, parity))) return true;
  return wait_slow(bar, parity, abort_flag, dev_err, code);
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

// hi and lo of four probabilities (in units of 1/256 for e4m3, 1/16256 for int8), a byte each,
// column 0 lowest.
template <int FMT>
__device__ __forceinline__ void split4(float2 p01, float2 p23, uint32_t& hi, uint32_t& lo) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) {
    // the rest in half precision: 11 bits hold p to 2^-12, and p - hi is exact
    const __half2 x0 = __floats2half2_rn(p01.x, p01.y), x1 = __floats2half2_rn(p23.x, p23.y);
    const __nv_fp8x2_storage_t h0 = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x0), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t h1 = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x1), __NV_SATFINITE, __NV_E4M3);
    const __half2 r0 = __hsub2(x0, __half2(__nv_cvt_fp8x2_to_halfraw2(h0, __NV_E4M3)));
    const __half2 r1 = __hsub2(x1, __half2(__nv_cvt_fp8x2_to_halfraw2(h1, __NV_E4M3)));
    const __nv_fp8x2_storage_t l0 = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r0), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t l1 = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r1), __NV_SATFINITE, __NV_E4M3);
    // (packed by byte_perm: packed by mov.b32 {h0, h1}, ptxas 12.9 read h0 back from the wrong half)
    hi = __byte_perm(h0, h1, 0x5410);
    lo = __byte_perm(l0, l1, 0x5410);
  } else {
    // v = round(p) + 64 by adding 1.5 * 2^23 + 64: v = 128 hi + (lo + 64) with lo + 64 in
    // [0, 128), in the low 15 bits of the sum
    const float2 c = make_float2(12582976.f, 12582976.f);
    const float2 a = add2(p01, c), b = add2(p23, c);
    const uint32_t w0 = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x5410);
    const uint32_t w1 = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x5410);
    hi = __byte_perm((w0 >> 7) & 0x00ff00ffu, (w1 >> 7) & 0x00ff00ffu, 0x6420);
    // lo mod 256 in bits 0-7 and 16-23
    lo = __byte_perm((w0 & 0x007f007fu) + 0x00c000c0u, (w1 & 0x007f007fu) + 0x00c000c0u, 0x6420);
  }
}

// Two scores of a key: the products times its scale, -infinity if it is masked. In int8 the
// products are finite whatever the codes, so that is an addend (a multiply-add instead of a
// multiply and two selects: 224 rows over 16K keys 36.9 -> 35.5 us); in e4m3 a masked key's may
// be NaN.
template <int FMT>
__device__ __forceinline__ float2 key_score(float2 s, float scale, bool off) {
  if constexpr (FMT == FOCUS_CACHE_INT8) {
    const float k = off ? 0.f : scale, add = off ? -INFINITY : 0.f;
    return fma2(s, make_float2(k, k), make_float2(add, add));
  } else {
    const float2 x = mul2(s, make_float2(scale, scale));
    return off ? make_float2(-INFINITY, -INFINITY) : x;
  }
}

// The product of hi and lo from their accumulators.
template <int FMT>
__device__ __forceinline__ float both(uint32_t hi, uint32_t lo) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) return __uint_as_float(hi) + __uint_as_float(lo);
  else return static_cast<float>(static_cast<int>(hi) * 128 + static_cast<int>(lo));
}

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int FMT>
__device__ __forceinline__ float2 both2(const uint32_t* hi, const uint32_t* lo) {
  if constexpr (FMT == FOCUS_CACHE_E4M3)
    return add2(make_float2(__uint_as_float(hi[0]), __uint_as_float(hi[1])),
                make_float2(__uint_as_float(lo[0]), __uint_as_float(lo[1])));
  else
    return make_float2(both<FMT>(hi[0], lo[0]), both<FMT>(hi[1], lo[1]));
}

template <int FMT>
constexpr float prob_top() {
  return FMT == FOCUS_CACHE_E4M3 ? 256.f : 16256.f;
}

// Query q of the slice (head kvh * g + r / qcap, row r % qcap of r = row0 + q) as hi and lo rows
// of the K-major B operand: a warp, rows first, first + step, ...
template <int FMT, int D, int NQ>
__device__ __forceinline__ void split_queries(const CacheAttnArgs& a, const Desc& d, uint8_t* dst, float* q_scale, int first,
                                           int step) {
  constexpr int E = D / 32;                  // elements of a lane
  constexpr int UN = 8;                      // rows in flight
  const int lane = lane_id();
  for (int q0 = first; q0 < NQ; q0 += step * UN) {
    float x[UN][E];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int q = q0 + step * i, r = d.row0 + q;
      const bool real = q < d.rows && (d.nq == a.qcap || r % a.qcap < d.nq);
      const __nv_bfloat16* src = a.Q + ((static_cast<size_t>(d.b) * a.Hq + d.kvh * a.g) * a.qcap + r) * D + lane * E;
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

// NQ fp32 columns of tensor memory times a factor each, that of column n from lane n, or zero.
template <int NQ>
__device__ __forceinline__ void scale_columns(uint32_t taddr, float f, bool zero) {
#pragma unroll 1
  for (int h = 0; h < NQ; h += 16) {
    uint32_t r[16];
    if (!zero) {
      tmem_ld16(taddr + h, r);
      tmem_ld_wait();
    }
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      const float g = __shfl_sync(0xffffffffu, f, h + n);
      r[n] = zero ? 0u : __float_as_uint(__uint_as_float(r[n]) * g);
    }
    tmem_st16(taddr + h, r);
  }
  tmem_st_wait();
}

// ------------------------------------------------------------------ kernel
template <int FMT, int D, int NQ, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CacheAttnArgs a) {
  using SM = Lay<FMT, D, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  auto* bk = reinterpret_cast<Book<NQ>*>(smem + SM::kBook);
  volatile int* abort_flag = &bk->abort_flag;
  const int warp = warp_id(), lane = lane_id();

  if (warp == kProducer && lane == 0) {
    for (int i = 0; i < kK; ++i) {
      mbar_init(&bk->k_full[i], 2);              // the copies' bytes, the tile's scales (and sink rows)
      mbar_init(&bk->k_empty[i], 1);
    }
    for (int i = 0; i < kV; ++i) {
      mbar_init(&bk->v_full[i], 1);              // the copies' bytes
      mbar_init(&bk->v_empty[i], 1);
    }
    for (int i = 0; i < kS; ++i) {
      mbar_init(&bk->s_full[i], 2);              // the product, and the warp that has seen the tile's scales
      mbar_init(&bk->s_free[i], 4);
      mbar_init(&bk->t_full[i], 4);
      mbar_init(&bk->m_full[i], 1);
    }
    for (int i = 0; i < kO; ++i) {
      mbar_init(&bk->o_full[i], 2);              // the product, and the warp that has seen P's entry
      mbar_init(&bk->o_free[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bk->p_full[i], 4);
      mbar_init(&bk->q_full[i], kQParts);
      mbar_init(&bk->q_empty[i], 2 + 8);         // the last QK, and the warps that read the scales
      mbar_init(&bk->x_full[i], 8);
      mbar_init(&bk->x_done[i], 4);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&bk->d_full[i], 1);
      mbar_init(&bk->d_empty[i], kSoftmaxWarps + 2);   // softmax and MMA warps
    }
    mbar_init(&bk->drain[0], 1);
    mbar_init(&bk->drain[1], 1);
    bk->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMmaS) {
    tmem_alloc(&bk->tmem_base, SM::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();                   // (behind the wait: the join reads lengths in front of its own)
  const uint32_t tmem = bk->tmem_base;
  const uint32_t tS = tmem, tO = tS + kS * SM::kAcc, tAcc = tO + kO * SM::kAcc, tSum = tAcc + NQ;

  if (warp >= kProducer && warp < kProducer + kProducers) {
    // ------------------------------------------------------------ producers
    // Both walk over all runs; tile j of the CTA is producer j % 2's: issuing the copies of a 32 KB
    // tile takes 550 to 730 cycles, and with the scales and the wait one alone was slower than the
    // memory.
    const int pw = warp - kProducer;
    int* const blk_s = bk->blk[pw];
    int* const snk_s = bk->snk[pw];
    const int all = length_of_all<SPARSE>(a);
    const int heads = a.Hkv * a.n_slices;
    const int T = all * heads;
    const int shares = min(static_cast<int>(gridDim.x), T);
    int n_tiles = 0;                             // tiles of the runs so far
    int issued = 0;                              // tiles up to here have their copies under way (this producer's)
    bool ok = true;
    int n_desc = 0;
    auto push = [&](const Desc& d) {             // the first producer publishes a run
      if (pw != 0) return;
      const int s = n_desc % kDescs;
      if (n_desc >= kDescs)
        ok = wait_phase(&bk->d_empty[s], ((n_desc / kDescs) - 1) & 1, abort_flag, a.dev_err, DEV_ERR_TIMEOUT_PRODUCER);
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
      // the sequence that place t0 falls in
      int b = 0, base = 0;                       // base: length of the sequences before b, all heads
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int n = b0 + lane < a.B ? unit_length(sequence_of<SPARSE>(a, b0 + lane).tiles) * heads : 0;
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
      const int tp = 7 - a.page_shift;           // a tile is 2^tp pages
      const int ppt = 1 << tp;
      const int32_t* trow = a.table + static_cast<size_t>(b) * a.table_cols;
      bool lists_sorted = true;
      int n_snk = 0;
      for (int t = t0; t < t1 && ok;) {
        while (unit_length(q.tiles) * heads <= t - base) {    // on to the next sequence that has tiles
          base += unit_length(q.tiles) * heads;
          ++b;
          q = sequence_of<SPARSE>(a, b);
          trow = a.table + static_cast<size_t>(b) * a.table_cols;
        }
        const int len = unit_length(q.tiles), u = (t - base) / len;      // KV head and slice
        const int at = base + u * len + kLead;                           // place of the unit's first tile
        const int first = max(0, t - at), last = min(q.tiles, t1 - at);
        t = at + q.tiles;
        if (last <= first) continue;
        const int kvh = u / a.n_slices, slice = u - kvh * a.n_slices;
        Desc d;
        d.n = last - first;
        d.j0 = n_tiles;
        d.b = b;
        d.kvh = kvh;
        d.row0 = slice * a.slice_rows;
        d.rows = min(a.slice_rows, a.g * a.qcap - d.row0);
        d.nq = a.n_q ? max(0, min(a.n_q[b], a.qcap)) : a.qcap;
        d.slot = d.n == q.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (first == 0 ? 1 : 0);
        push(d);
        if (!ok) break;

        if (SPARSE) {
          // the kept blocks: repeated entries are dropped (in an ascending list they are neighbours)
          const int32_t* blk = a.blocks + (static_cast<size_t>(b) * a.Hkv + kvh) * a.C;
          bool up = true;
          int before = -1;
          for (int i0 = 0; i0 < a.C; i0 += 64) {
            int vs[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) vs[u] = i0 + 32 * u + lane < a.C ? blk[i0 + 32 * u + lane] : -1;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int i = i0 + 32 * u + lane, v = vs[u];
              const int prev = __shfl_up_sync(0xffffffffu, v, 1);
              const int pv = lane == 0 ? before : prev;
              up = up && (v < 0 || v > pv) && !(v >= 0 && pv < 0 && i > 0);
              if (i < a.C) blk_s[i] = v;
              before = __shfl_sync(0xffffffffu, v, 31);
            }
          }
          lists_sorted = __all_sync(0xffffffffu, up);
          __syncwarp();
          if (!lists_sorted) {
            // drop repeats, the later ones: entry by entry over the list, 32 at a time
            for (int i0 = (a.C - 1) & ~31; i0 >= 0; i0 -= 32) {
              const int i = i0 + lane;
              bool again = false;
              if (i < a.C)
                for (int j = 0; j < i && !again; ++j) again = blk_s[j] == blk_s[i];
              __syncwarp();
              if (again) blk_s[i] = -1;
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
          float f, vm;                           // value scale relative to the tile's largest, that
          unsigned part;                         // lanes whose page is not all keys
        };
        auto look_up = [&](int slot) {
          Batch x{-1, 0, 0, -1, 0.f, 0.f, 0.f, 0.f, 0u};
          int col = -1;
          if (!SPARSE) {
            if (slot < q.n_pages) {
              col = slot;
              x.hi = min(a.page, q.len - slot * a.page);
            }
          } else if (slot < q.n_gen) {
            col = (q.gs >> a.page_shift) + slot;
            x.lo = max(0, q.gs - col * a.page);
            x.hi = min(a.page, q.ge - col * a.page);
          } else if (slot < q.n_pages) {
            const int j = blk_s[slot - q.n_gen];
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
        // what a tile's entry says, for all tiles of the batch at once: its pages are neighbouring
        // lanes
        auto finish = [&](Batch& x) {
          x.vm = x.hi > x.lo ? fabsf(x.vs) : 0.f;
          for (int off = 1; off < ppt; off <<= 1) x.vm = max_nan(x.vm, __shfl_xor_sync(0xffffffffu, x.vm, off));
          x.f = x.vm == 0.f || x.hi <= x.lo ? 0.f : x.vs / x.vm * prob_top<FMT>();
          x.part = __ballot_sync(0xffffffffu, x.lo > 0 || x.hi < a.page);
        };
        auto find_sinks = [&]() {
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
            if (i0 + lane < a.S) snk_s[i0 + lane] = v;
            before = __shfl_sync(0xffffffffu, v, 31);
          }
          up = __all_sync(0xffffffffu, up);
          __syncwarp();
          for (int i0 = (a.S - 1) & ~31; i0 >= 0; i0 -= 32) {
            const int i = i0 + lane, v = i < a.S ? snk_s[i] : -1;
            bool drop = v < 0 || (v >= q.gs && v < q.ge);
            if (!up)
              for (int j = 0; j < i && !drop; ++j) drop = snk_s[j] == v;
            if (!drop && v < q.P) {
              const int col = v >> a.page_shift;
              if (lists_sorted) {        // ascending, then -1
                int lo = 0, hi = a.C;
                while (lo < hi) {
                  const int mid = (lo + hi) >> 1, x = blk_s[mid];
                  if (x >= 0 && x < col) lo = mid + 1;
                  else hi = mid;
                }
                drop = lo < a.C && blk_s[lo] == col;
              } else {
                for (int j = 0; j < a.C && !drop; ++j) drop = blk_s[j] == col;
              }
            }
            __syncwarp();
            if (drop && i < a.S) snk_s[i] = -1;
            __syncwarp();
          }
          n_snk = a.S;
        };
        if (SPARSE && lane == 0) {
          const long long g0 = a.g0[b];          // a current block that leaves the table
          if (g0 < 0 || g0 + a.G > static_cast<long long>(a.table_cols) * a.page) record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
        }
        if (!SPARSE && lane == 0 && a.lens[b] > a.table_cols * a.page) record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
        const int j0 = n_tiles - first;          // the CTA's number of tile 0 of this unit
        n_tiles += d.n;
        const int mine_first = first + ((j0 + first + pw) & 1);      // this producer's first tile
        int bbase = first << tp;
        Batch cur = look_up(bbase + lane);
        resolve(cur);
        int tile = mine_first;
        for (; tile < last && ok;) {
          const int b_end = min(last, (bbase + 32) >> tp);
          Batch nxt{-1, 0, 0, -1, 0.f, 0.f, 0.f, 0.f, 0u};
          if (b_end < last) nxt = look_up(bbase + 32 + lane);
          bool resolved = false, finished = false, cold = tile == mine_first;
          int done = tile;                       // the next tile whose scales are to be published
          while (done < b_end && ok) {
            // Copies of the next tile; at the start of a run, while its first scales are on their
            // way, of as many as find a free stage (afterwards scales go with each tile, or they
            // would hold up its use)
            do {
              const int j = j0 + tile, sk = j % kK, sv = j % kV;
              auto free_stage = [&](uint64_t* bar, int round) {
                if (round == 0) return true;
                if (tile == done)
                  return ok = wait_phase(bar, (round - 1) & 1, abort_flag, a.dev_err, DEV_ERR_TIMEOUT_PRODUCER);
                return __all_sync(0xffffffffu, mbar_test(bar, (round - 1) & 1)) != 0;
              };
              if (!free_stage(&bk->k_empty[sk], j / kK) || !free_stage(&bk->v_empty[sv], j / kV)) break;
              const int rel = bbase + lane - (tile << tp);           // this lane's page of the tile
              const bool mine = rel >= 0 && rel < ppt && cur.pg >= 0;
              const unsigned any = __ballot_sync(0xffffffffu, mine);
              if (lane == 0) {
                mbar_arrive_expect_tx(&bk->k_full[sk], static_cast<uint32_t>(__popc(any) * a.page * D));
                mbar_arrive_expect_tx(&bk->v_full[sv], static_cast<uint32_t>(__popc(any) * a.page * D));
              }
              __syncwarp();
              if (mine) {
                const uint32_t at = smem_u32(smem) + rel * a.page * D;
                const uint32_t dk = at + sk * SM::kTile, dv = at + SM::kVRing + sv * SM::kTile;
                const int z = static_cast<int>(static_cast<long long>(cur.pg) * a.Hkv + kvh);
                if (once) {
                  tma_load_3d_hint(dk, &tmK, &bk->k_full[sk], 0, 0, z, policy);
                  tma_load_3d_hint(dv, &tmV, &bk->v_full[sv], 0, 0, z, policy);
                } else {
                  tma_load_3d(dk, &tmK, &bk->k_full[sk], 0, 0, z);
                  tma_load_3d(dv, &tmV, &bk->v_full[sv], 0, 0, z);
                }
              }
              __syncwarp();
              issued = j + 1;
              tile += kProducers;
            } while (cold && tile < b_end);
            if (!ok) break;
            if (!finished) finish(cur);
            cold = false;
            finished = true;
            for (; done < tile; done += kProducers) {
              const int s = (j0 + done) % kV, sk = (j0 + done) % kK;
              if (!SPARSE || done * 128 + 128 <= (q.n_pages << a.page_shift)) {
                // whole pages: each lane its own, and each softmax thread looks up its key's
                const int rel = bbase + lane - (done << tp);
                if (rel >= 0 && rel < ppt)
                  bk->page[s][rel] = make_float4(cur.ks, cur.f, __int_as_float(cur.lo), __int_as_float(cur.hi));
                if (rel == 0) {
                  bk->vmax[s] = cur.vm / prob_top<FMT>();
                  bk->info[s] = (cur.part >> lane) & ((1u << ppt) - 1u) ? kMasked : 0;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bk->k_full[sk]);
                if (!resolved && b_end < last) {
                  resolve(nxt);
                  resolved = true;
                }
                continue;
              }
              if constexpr (SPARSE) {
              // keys 4 lane .. 4 lane + 3 lie in one page slot, or among the sinks
              const int k0 = done * 128 + 4 * lane;
              const int slot = k0 >> a.page_shift, from = (slot - bbase) & 31, r = k0 & (a.page - 1);
              const int lo = __shfl_sync(0xffffffffu, cur.lo, from), hi = __shfl_sync(0xffffffffu, cur.hi, from);
              const float k = __shfl_sync(0xffffffffu, cur.ks, from), v = __shfl_sync(0xffffffffu, cur.vs, from);
              float ks[4], vs[4];
              bool on[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                on[e] = slot < q.n_pages && r + e >= lo && r + e < hi;
                ks[e] = k;
                vs[e] = on[e] ? v : 0.f;
              }
              {
                if (n_snk < 0) find_sinks();
                // position, page, scales and rows of the four keys, step by step for all of them:
                // each step is a round trip to memory
                int pos[4], pg[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int i = k0 + e - q.n_pages * a.page;
                  pos[e] = i >= 0 && i < n_snk ? snk_s[i] : -1;
                  pg[e] = -1;
                  if (pos[e] >= 0 && (pos[e] >> a.page_shift) < a.table_cols) pg[e] = trow[pos[e] >> a.page_shift];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (pos[e] < 0) continue;
                  if (pg[e] < 0 || pg[e] >= a.n_pages) {
                    record_dev_error(a.dev_err, DEV_ERR_BAD_INDEX);
                    pos[e] = -1;
                    continue;
                  }
                  const long long ph = static_cast<long long>(pg[e]) * a.Hkv + kvh;
                  on[e] = true;
                  ks[e] = __ldg(a.scale[0] + ph);
                  vs[e] = __ldg(a.scale[1] + ph);
                }
                const uint32_t dk = smem_u32(smem) + sk * SM::kTile, dv = smem_u32(smem) + SM::kVRing + s * SM::kTile;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (pos[e] < 0) continue;
                  const long long ph = static_cast<long long>(pg[e]) * a.Hkv + kvh;
                  const long long off = (ph * a.page + (pos[e] & (a.page - 1))) * D;
#pragma unroll
                  for (int c = 0; c < D / 16; ++c) {
                    cp_async16(dk + row_chunk<D>(4 * lane + e, c), a.code[0] + off + c * 16, 16);
                    cp_async16(dv + row_chunk<D>(4 * lane + e, c), a.code[1] + off + c * 16, 16);
                  }
                }
                cp_async_wait_all();
                fence_proxy_async_smem();
              }
              float vm = fmaxf(fmaxf(fabsf(vs[0]), fabsf(vs[1])), fmaxf(fabsf(vs[2]), fabsf(vs[3])));
              if (vs[0] != vs[0] || vs[1] != vs[1] || vs[2] != vs[2] || vs[3] != vs[3]) vm = NAN;
              vm = warp_max_nan(vm);
              // values relative to the tile's largest (four of a page are the same)
              float f[4];
              f[0] = vm == 0.f ? 0.f : vs[0] / vm * prob_top<FMT>();
#pragma unroll
              for (int e = 1; e < 4; ++e)
                f[e] = vs[e] == vs[0] ? f[0] : vm == 0.f ? 0.f : vs[e] / vm * prob_top<FMT>();
              float4* key = reinterpret_cast<float4*>(&bk->key[s][4 * lane]);
              key[0] = make_float4(ks[0], f[0], ks[1], f[1]);
              key[1] = make_float4(ks[2], f[2], ks[3], f[3]);
              *reinterpret_cast<uchar4*>(&bk->valid[s][4 * lane]) = make_uchar4(on[0], on[1], on[2], on[3]);
              if (lane == 0) {
                bk->vmax[s] = vm / prob_top<FMT>();
                bk->info[s] = kMasked | kByKey;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&bk->k_full[sk]);
              if (!resolved && b_end < last) {
                resolve(nxt);
                resolved = true;
              }
              }
            }
          }
          if (!resolved && b_end < last) resolve(nxt);
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
      auto land = [&](uint64_t* bar, int parity) {
        const unsigned long long w0 = globaltimer();
        while (!__all_sync(0xffffffffu, mbar_test(bar, parity & 1)) &&
               !__any_sync(0xffffffffu, globaltimer() - w0 > 500000000ull)) {
        }
      };
      for (int j = issued - 1; j >= 0 && j >= issued - kV; j -= kProducers) {
        land(&bk->v_full[j % kV], j / kV);
        if (j < issued - kK) continue;
        if (lane == 0) mbar_arrive(&bk->k_full[j % kK]);
        land(&bk->k_full[j % kK], j / kK);
      }
    }
    __syncwarp();
  } else if (warp == kMmaS || warp == kMmaO) {
    // ------------------------------------------------------------ MMA issuers
    // A warp for each product, so that neither a late tile holds up a finished P nor the other
    // way. The whole warp takes every step and one elected thread issues: the descriptors then
    // stay in uniform registers. (Inside a branch on lane == 0 an MMA cost 110 cycles to issue,
    // with the elected thread about 60.)
    const uint32_t elected = elect_one();
    const bool qk = warp == kMmaS;
    const uint32_t id = idesc8<FMT>(2 * NQ, !qk);
    const uint64_t k0 = tile_desc<D>(smem_u32(smem)), v0 = tile_desc<D>(smem_u32(smem) + SM::kVRing);
    const uint64_t q0 = tile_desc<D>(smem_u32(smem) + SM::kQ);
    const uint64_t p0 = tile_desc<SM::kPRow>(smem_u32(smem) + SM::kP);
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      return ok = wait_phase(bar, parity, abort_flag, a.dev_err, DEV_ERR_TIMEOUT_MMA);
    };
    auto test = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0; };
    const int lc = lane & (NQ - 1);              // the column whose reference this lane sets
    int j = 0;
    for (int di = 0; ok; ++di) {
      const int ds = di % kDescs, qb = di & 1;
      if (!wait(&bk->d_full[ds], (di / kDescs) & 1)) break;
      const int n = bk->desc[ds].n, je = j + n;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bk->d_empty[ds]);
      if (n == 0) break;
      if (!qk) {
        for (; j < je; ++j) {
          const int s = j % kV, buf = j & 1, ob = j % kO;
          if (j >= kO && !wait(&bk->o_free[ob], (j / kO - 1) & 1)) break;
          if (!wait(&bk->p_full[buf], (j >> 1) & 1)) break;
          if (!wait(&bk->v_full[s], (j / kV) & 1)) break;
          tc_fence_after();
          const uint64_t vd = v0 + static_cast<uint64_t>(s * SM::kTile / 16);
          const uint64_t pd = p0 + static_cast<uint64_t>(buf * SM::kPBuf / 16);
          if (elected) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma8<FMT>(tO + ob * SM::kAcc, vd + ks * (32 * D / 16), pd + ks * (32 * SM::kPRow / 16), id, ks > 0 ? 1u : 0u);
            mma_commit(&bk->o_full[ob]);
            mma_commit(&bk->v_empty[s]);
            mbar_arrive(&bk->o_full[ob]);
          }
          __syncwarp();
        }
        continue;
      }
      if (!wait(&bk->q_full[qb], (di >> 1) & 1)) break;
      // (a zero query or scale: with the smallest normal number instead, every finite score is
      // still 0, and a masked key's -infinity stays what it is)
      float qs = bk->q_scale[qb][lc], m_ref = -INFINITY;
      if (qs == 0.f) qs = 1.17549435e-38f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bk->q_empty[qb]);
      // whichever can go on next: the product of tile j, or the references of tile jr
      unsigned long long idle = 0;               // since when neither could
      for (int jr = j; jr < je;) {
        bool did = false;
        const int rb = jr % kS;
        if (jr < j && test(&bk->t_full[rb], (jr / kS) & 1)) {
          // A tile's probabilities are relative to a reference of its own, the next whole number
          // above its largest score in units of log2. (Against a running maximum instead, all that
          // lies 2^-18 below one large key, an attention sink, would be rounded away, and with
          // thousands of such keys a part of the result.) Sums over tiles are relative to m_ref, the
          // reference of the run's first tile with keys, which moves up only when another is above
          // it by 30: fp32 has the range, no sum is rescaled tile by tile, and the factor between
          // the two, a power of two, is exact in 16 bits: handing it to all threads costs
          // shared-memory bandwidth, of which the tensor cores take half. (The reference itself
          // takes all 32: rounded up to bf16 too, it lay 2^5 above scores of some thousands.)
          const float* tp = &bk->top[rb][0][lc];
          const float mt = max3_nan(max_nan(tp[0], tp[NQ]), tp[2 * NQ], tp[3 * NQ]);
          float ref = 0.f;                       // (a tile without keys adds nothing)
          uint32_t be16 = 0;                     // bf16 of the factor
          if (mt != -INFINITY) {
            ref = ceilf(__fmul_rn(mt, qs));
            if (ref > m_ref + 30.f || m_ref == -INFINITY) m_ref = ref;
            const float e = ref - m_ref;         // a whole number
            be16 = e != e ? 0x7fc0u : e < -126.f ? 0u : static_cast<uint32_t>(127 + static_cast<int>(e)) << 7;
          }
          const int e = jr % kE;
          bk->ref[e][lc] = -ref;
          bk->be[e][lc] = static_cast<uint16_t>(be16);
          bk->run[e][lc] = m_ref;
          if (lane == 0) bk->o_vmax[e] = bk->vmax[jr % kV];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bk->m_full[rb]);
          ++jr;
          did = true;
        }
        const int s = j % kK, sb = j % kS;
        if (j < je && j - jr < kS && test(&bk->k_full[s], (j / kK) & 1) &&
            (j < kS || test(&bk->s_free[sb], (j / kS - 1) & 1))) {
          tc_fence_after();
          const uint64_t kd = k0 + static_cast<uint64_t>(s * SM::kTile / 16);
          const uint64_t qd = q0 + static_cast<uint64_t>(qb * SM::kQBuf / 16);
          if (elected) {
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
              mma8<FMT>(tS + sb * SM::kAcc, kd + ks * 2, qd + ks * 2, id, ks > 0 ? 1u : 0u);
            mma_commit(&bk->s_full[sb]);
            mma_commit(&bk->k_empty[s]);
            if (j == je - 1) mma_commit(&bk->q_empty[qb]);
            mbar_arrive(&bk->s_full[sb]);
          }
          __syncwarp();
          ++j;
          did = true;
        }
        if (did) {
          idle = 0;
          continue;
        }
        const unsigned long long now = globaltimer();
        if (idle == 0) idle = now;
        bool stop = *abort_flag != 0;
        if (now - idle > kWaitLimitNs) {
          *abort_flag = 1;
          if (lane == 0) record_dev_error(a.dev_err, DEV_ERR_TIMEOUT_MMA);
          stop = true;
        }
        if (__any_sync(0xffffffffu, stop)) {
          ok = false;
          break;
        }
      }
    }
    // (after a wait that ran out, products may still be under way)
    if (elected) mma_commit(&bk->drain[qk ? 0 : 1]);
    __syncwarp();
    const unsigned long long w0 = globaltimer();
    while (!__all_sync(0xffffffffu, mbar_test(&bk->drain[qk ? 0 : 1], 0)) &&
           !__any_sync(0xffffffffu, globaltimer() - w0 > 500000000ull)) {
    }
  } else {
    // ------------------------------------------------------------ softmax stages
    const int wq = warp & 3;
    const int t = threadIdx.x & 127;             // key of the tile == TMEM lane == dim of O^T
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      return ok = wait_phase(bar, parity, abort_flag, a.dev_err, DEV_ERR_TIMEOUT_SOFTMAX);
    };
    // the next run; false at the end
    Desc d;
    auto next_run = [&](int di) {
      const int ds = di % kDescs;
      if (!wait(&bk->d_full[ds], (di / kDescs) & 1)) return false;
      d = bk->desc[ds];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bk->d_empty[ds]);
      if (d.n == 0) return false;
      if (di == 0) {                             // the first run's query rows: nothing else to do yet
        split_queries<FMT, D, NQ>(a, d, smem + SM::kQ, bk->q_scale[0], warp, kQParts);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bk->q_full[0]);
      }
      return true;
    };
    // what the scales of tile stage s say about this thread's key: (scale, factor of its value);
    // off: it is masked
    auto key_of = [&](int s, bool& off) {
      const int info = bk->info[s];
      const float4 pg = bk->page[s][t >> a.page_shift];
      float2 key = make_float2(pg.x, pg.y);
      off = false;
      if (info != 0) {
        asm volatile("" ::: "memory");           // (a branch: few tiles come here)
        if (info & kByKey) {
          key = bk->key[s][t];
          off = bk->valid[s][t] == 0;
        } else {
          const int r = t & (a.page - 1);
          off = r < __float_as_int(pg.z) || r >= __float_as_int(pg.w);
        }
      }
      return key;
    };
    if (warp < kExpWarp) {
      // ---------------------------------------------------------- largest scores
      auto queries = [&](const Desc& x, int qb) {
        split_queries<FMT, D, NQ>(a, x, smem + SM::kQ + qb * SM::kQBuf, bk->q_scale[qb], warp, 4);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_n(&bk->q_full[qb], kQParts / 4);
      };
      auto test = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0; };
      bool ready = false;                        // the next run's query rows are there
      for (int di = 0; next_run(di); ++di) {
        // the run's query rows, if there was no time during the run before
        if (di > 0 && !ready) {
          if (di >= 2 && !wait(&bk->q_empty[di & 1], ((di >> 1) - 1) & 1)) break;
          queries(d, di & 1);
        }
        ready = false;
        for (int j = d.j0; j < d.j0 + d.n; ++j) {
          const int s = j % kV, sb = j % kS;
          if (!wait(&bk->s_full[sb], (j / kS) & 1)) break;   // (and with it the tile's scales and bytes)
          tc_fence_after();
          bool off;
          const float ks = key_of(s, off).x;
#pragma unroll 1
          for (int h = 0; h < NQ; h += 16) {
            uint32_t r[16], r2[16];
            tmem_ld16(tS + sb * SM::kAcc + lane_addr + h, r);
            tmem_ld16(tS + sb * SM::kAcc + NQ + lane_addr + h, r2);
            tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < 16; n += 4) {
              const float2 x0 = key_score<FMT>(both2<FMT>(r + n, r2 + n), ks, off);
              const float2 x1 = key_score<FMT>(both2<FMT>(r + n + 2, r2 + n + 2), ks, off);
              float4 m;
              m.x = warp_max_nan(x0.x);
              m.y = warp_max_nan(x0.y);
              m.z = warp_max_nan(x1.x);
              m.w = warp_max_nan(x1.y);
              if (lane == 0) *reinterpret_cast<float4*>(&bk->top[sb][wq][h + n]) = m;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bk->t_full[sb]);
          // The next run's 16 query rows, as soon as that run is known and the rows of the one before
          // this are used up: its scores then follow this run's without a gap (sixteen ragged
          // sequences: 57 -> 50 us). 32 rows take twice as long, and in mid-run that costs the chain
          // as much as it saves (four sequences' kept blocks: 36 -> 39 us).
          if constexpr (NQ == 16) {
            const int dn = di + 1, ds = dn % kDescs;
            if (!ready && test(&bk->d_full[ds], (dn / kDescs) & 1) &&
                (dn < 2 || test(&bk->q_empty[dn & 1], ((dn >> 1) - 1) & 1))) {
              if (bk->desc[ds].n > 0) queries(bk->desc[ds], dn & 1);
              ready = true;
            }
          }
        }
        if (!ok) break;
      }
    } else if (warp < kSumWarp) {
      // ---------------------------------------------------------- probabilities
      const int we = warp - kExpWarp, grp = we >> 2;   // the group takes the tiles j with j % 2 == grp
      const int lc = lane & (NQ - 1);
      for (int di = 0; next_run(di); ++di) {
        const int qb = di & 1;
        if (!wait(&bk->q_full[qb], (di >> 1) & 1)) break;
        {
          const float qs = bk->q_scale[qb][lc];
          bk->qs[we][lc] = qs == 0.f ? 1.17549435e-38f : qs;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bk->q_empty[qb]);
        float m_ref = -INFINITY;                 // of the lane's column, what the row sums are relative to
        const uint32_t tl = tSum + grp * NQ + lane_addr;
        scale_columns<NQ>(tl, 0.f, true);
        const int je = d.j0 + d.n;
        for (int j = d.j0 + ((d.j0 ^ grp) & 1); j < je; j += 2) {
          const int s = j % kV, sb = j % kS, e = j % kE;
          if (!wait(&bk->m_full[sb], (j / kS) & 1)) break;
          if (!wait(&bk->s_full[sb], (j / kS) & 1)) break;
          tc_fence_after();
          bool off;
          const float2 key = key_of(s, off);
          const float m_new = bk->run[e][lc];
          if (__any_sync(0xffffffffu, m_new != m_ref)) {               // (the run's first tile, seldom another)
            scale_columns<NQ>(tl, m_new == m_ref ? 1.f : exp2_approx(m_ref - m_new), false);
            m_ref = m_new;
          }
          // the buffer of P is free once the product that used it is done
          if (j >= 2 && !wait(&bk->o_full[(j - 2) % kO], ((j - 2) / kO) & 1)) break;
          // P is written as it is held, a key to a row, hi then lo: an MN-major operand. (Stored
          // query-major, a byte at a time, the stores alone took 1500 cycles of a tile.)
          uint8_t* pbuf = smem + SM::kP + (j & 1) * SM::kPBuf;
          const uint32_t ts = tS + sb * SM::kAcc + lane_addr;
#pragma unroll 1
          for (int h = 0; h < NQ; h += 16) {
            uint32_t r[16], r2[16], rl[16];
            tmem_ld16(ts + h, r);
            tmem_ld16(ts + NQ + h, r2);
            tmem_ld16(tl + h, rl);
            tmem_ld_wait();
            if (h == NQ - 16) {                  // the scores have been read
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bk->s_free[sb]);
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x0 = key_score<FMT>(both2<FMT>(r + 4 * i, r2 + 4 * i), key.x, off);
              const float2 x1 = key_score<FMT>(both2<FMT>(r + 4 * i + 2, r2 + 4 * i + 2), key.x, off);
              const float4 rv = *reinterpret_cast<const float4*>(&bk->ref[e][h + 4 * i]);
              const uint2 bv = *reinterpret_cast<const uint2*>(&bk->be[e][h + 4 * i]);
              const float4 qv = *reinterpret_cast<const float4*>(&bk->qs[we][h + 4 * i]);
              // (The product is rounded before the reference is taken off, as that which gave the
              // reference was, so p <= 1 however large the scores. By one multiply-add, whose product
              // is exact, p came out above 1 where the reference's had been rounded down, and left the
              // 8 bits of a part.)
              float2 p0 = add2(round2(x0, make_float2(qv.x, qv.y)), make_float2(rv.x, rv.y));
              float2 p1 = add2(round2(x1, make_float2(qv.z, qv.w)), make_float2(rv.z, rv.w));
              p0 = make_float2(exp2_approx(p0.x), exp2_approx(p0.y));
              p1 = make_float2(exp2_approx(p1.x), exp2_approx(p1.y));
              const float2 l0 = fma2(p0, bf16_pair(bv.x), make_float2(__uint_as_float(rl[4 * i]), __uint_as_float(rl[4 * i + 1])));
              const float2 l1 = fma2(p1, bf16_pair(bv.y), make_float2(__uint_as_float(rl[4 * i + 2]), __uint_as_float(rl[4 * i + 3])));
              rl[4 * i] = __float_as_uint(l0.x);
              rl[4 * i + 1] = __float_as_uint(l0.y);
              rl[4 * i + 2] = __float_as_uint(l1.x);
              rl[4 * i + 3] = __float_as_uint(l1.y);
              split4<FMT>(mul2(p0, make_float2(key.y, key.y)), mul2(p1, make_float2(key.y, key.y)), hi[i], lo[i]);
            }
            tmem_st16(tl + h, rl);
            *reinterpret_cast<uint4*>(pbuf + row_chunk<SM::kPRow>(t, h / 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(pbuf + row_chunk<SM::kPRow>(t, (NQ + h) / 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          tmem_st_wait();
          // A masked key's values may be anything, NaN codes included, and 0 * NaN is NaN
          if (FMT == FOCUS_CACHE_E4M3 && __any_sync(0xffffffffu, off)) {
            if (!wait(&bk->v_full[s], (j / kV) & 1)) break;
            uint8_t* v = smem + SM::kVRing + s * SM::kTile;
            if (off) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c)
                *reinterpret_cast<uint4*>(v + row_chunk<D>(t, c)) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bk->p_full[j & 1]);
        }
        if (!ok) break;
        // row sums over the warp's keys, for the sum warps, which have the run before last behind them
        if (di >= 2 && !wait(&bk->x_done[qb], ((di >> 1) - 1) & 1)) break;
#pragma unroll 1
        for (int h = 0; h < NQ; h += 16) {
          uint32_t rl[16];
          tmem_ld16(tl + h, rl);
          tmem_ld_wait();
          float ls[16];
#pragma unroll
          for (int n = 0; n < 16; ++n) ls[n] = __uint_as_float(rl[n]);
          warp_sum_scatter16(ls);                // column h + n in lanes 2 n and 2 n + 1
          bk->x_l[qb][we][h + (lane >> 1)] = ls[0];
        }
        if (wq == 0) bk->x_m[qb][grp][lc] = m_ref;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bk->x_full[qb]);
      }
    } else {
      // ---------------------------------------------------------- sums and output
      const int ws = warp - kSumWarp;
      const int lc = lane & (NQ - 1);            // the column that this lane follows
      for (int di = 0; next_run(di); ++di) {
        const int qb = di & 1;
        float m_ref = -INFINITY;
        const uint32_t ta = tAcc + lane_addr;
        scale_columns<NQ>(ta, 0.f, true);
        for (int j = d.j0; j < d.j0 + d.n; ++j) {
          const int ob = j % kO, e = j % kE;
          if (!wait(&bk->o_full[ob], (j / kO) & 1)) break;
          tc_fence_after();
          const float2 vmax = make_float2(bk->o_vmax[e], bk->o_vmax[e]);
          const float m_new = bk->run[e][lc];
          if (__any_sync(0xffffffffu, m_new != m_ref)) {
            scale_columns<NQ>(ta, m_new == m_ref ? 1.f : exp2_approx(m_ref - m_new), false);
            m_ref = m_new;
          }
#pragma unroll 1
          for (int h = 0; h < NQ; h += 16) {
            uint32_t r[16], r2[16], ra[16];
            tmem_ld16(tO + ob * SM::kAcc + lane_addr + h, r);
            tmem_ld16(tO + ob * SM::kAcc + NQ + lane_addr + h, r2);
            tmem_ld16(ta + h, ra);
            uint32_t w[8];
            *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(&bk->be[e][h]);
            *reinterpret_cast<uint4*>(w + 4) = *reinterpret_cast<const uint4*>(&bk->be[e][h + 8]);
            tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float2 v = fma2(mul2(bf16_pair(w[n]), vmax), both2<FMT>(r + 2 * n, r2 + 2 * n),
                                    make_float2(__uint_as_float(ra[2 * n]), __uint_as_float(ra[2 * n + 1])));
              ra[2 * n] = __float_as_uint(v.x);
              ra[2 * n + 1] = __float_as_uint(v.y);
            }
            tmem_st16(ta + h, ra);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bk->o_free[ob]);
        }
        if (!ok) break;
        // join: the exp groups' row sums, each relative to its own reference, and O
        if (!wait(&bk->x_full[qb], (di >> 1) & 1)) break;
        const float m0 = bk->x_m[qb][0][lc], m1 = bk->x_m[qb][1][lc];
        const float M = max3_nan(m_ref, m0, m1);
        const float* xl = &bk->x_l[qb][0][lc];
        const float l0 = (xl[0] + xl[NQ]) + (xl[2 * NQ] + xl[3 * NQ]), l1 = (xl[4 * NQ] + xl[5 * NQ]) + (xl[6 * NQ] + xl[7 * NQ]);
        const float l = (l0 == 0.f ? 0.f : l0 * exp2_approx(m0 - M)) + (l1 == 0.f ? 0.f : l1 * exp2_approx(m1 - M));
        float fo = m_ref == -INFINITY ? 0.f : exp2_approx(m_ref - M);
        if (d.slot < 0) fo *= l == 0.f ? 0.f : 1.f / l;
        if (d.slot >= 0 && ws == 0 && lane < NQ && lane < d.rows)
          a.part_ml[static_cast<size_t>(d.slot) * NQ + lane] = make_float2(M, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bk->x_done[qb]);
        // output: every thread its dim of every row, row after row in memory
        const unsigned none = __ballot_sync(0xffffffffu, d.nq < a.qcap && (d.row0 + lc) % a.qcap >= d.nq);
        float* part = a.part_o + static_cast<size_t>(max(d.slot, 0)) * NQ * D + t;
        __nv_bfloat16* out = a.O + ((static_cast<size_t>(d.b) * a.Hq + d.kvh * a.g) * a.qcap + d.row0) * D + t;
#pragma unroll 1
        for (int h = 0; h < d.rows; h += 8) {
          uint32_t ra[8];
          tmem_ld8(ta + h, ra);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int n = h + i;
            const float v = __uint_as_float(ra[i]) * __shfl_sync(0xffffffffu, fo, n);
            if (n < d.rows && t < D) {
              if (d.slot >= 0) part[n * D] = v;
              else out[n * D] = __float2bfloat16_rn((none >> n) & 1u ? 0.f : v);
            }
          }
        }
      }
    }
    if (!ok) bk->abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaS) tmem_dealloc(tmem, SM::kTmem);
}

// Joins the parts of the units that several CTAs worked on (a warp per query row, a lane holds
// D / 32 dims): weights 2^(m - M) over the parts' (m, l), eight parts at a time. Units without
// keys get zeros; units of one CTA are done already. Which parts there are follows from the
// inputs alone, so it is worked out before the attention is done: two warps of 64 registers find
// room beside an attention CTA. (These inputs are read in front of the wait, which is right only
// because the attention kernel signals behind its own wait, when all before it has been written. All
// wait for the attention, those without work too: what follows in the stream waits for this kernel
// only.)
constexpr int kJoinWarps = 2;
template <int D, bool SPARSE>
__global__ void __launch_bounds__(kJoinWarps * 32, 16) cache_combine_kernel(const CacheAttnArgs a, int NQ) {
  constexpr int E = D / 32;
  griddep_launch_dependents();
  const int lane = lane_id();
  const unsigned rows = static_cast<unsigned>(a.g * a.qcap);   // of a KV head
  const unsigned w = blockIdx.x * kJoinWarps + warp_id();
  const unsigned bh = w / rows, r = w - bh * rows;
  const int b = static_cast<int>(bh) / a.Hkv, kvh = static_cast<int>(bh) - b * a.Hkv;
  if (b >= a.B) {
    griddep_wait();
    return;
  }
  const int slice = static_cast<int>(r) / a.slice_rows, n = static_cast<int>(r) - slice * a.slice_rows;
  const int tiles = sequence_of<SPARSE, true>(a, b).tiles;
  const int qi = static_cast<int>(r) % a.qcap;
  const bool real = !a.n_q || qi < __ldcg(a.n_q + b);
  int s0 = 0, s1 = -1;
  if (tiles > 0) {
    const int heads = a.Hkv * a.n_slices;
    const int T = length_of_all<SPARSE, true>(a) * heads;
    const int shares = min(a.grid, T);
    const int x0 = length_before<SPARSE, true>(a, b) * heads + (kvh * a.n_slices + slice) * unit_length(tiles) + kLead;
    s0 = share_of(x0, T, shares), s1 = share_of(x0 + tiles - 1, T, shares);
  }
  griddep_wait();
  if (s0 == s1) return;
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  float l = 0.f, M = -INFINITY;
  // slot of share c's part: a share's last run is its part of a unit that goes on, its first of one
  // that came before
  auto slot = [&](int c) { return static_cast<size_t>(2 * c + (c == s0 ? 1 : 0)) * NQ + n; };
  constexpr int kAhead = 8;              // parts of O on their way together
  for (int c0 = s0; c0 <= s1; c0 += kAhead) {
    const int cn = min(kAhead, s1 - c0 + 1);
    float v[kAhead][E];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float* src = a.part_o + slot(c0 + (i < cn ? i : 0)) * D + lane * E;
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[i][0] = x.x, v[i][1] = x.y;
      }
    }
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < cn) ml = a.part_ml[slot(c0 + lane)];
    const float mn = max_nan(M, warp_max_nan(ml.x));
    const float back = l == 0.f ? 0.f : exp2_approx(M - mn);
    const float f = ml.y == 0.f ? 0.f : exp2_approx(ml.x - mn);
    float lw = f * ml.y;
#pragma unroll
    for (int off = kAhead / 2; off; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
    l = l * back + __shfl_sync(0xffffffffu, lw, 0);
    M = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= back;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      if (i < cn)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += fi * v[i][e];
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* O = a.O + (static_cast<size_t>(bh) * rows + r) * D + lane * E;
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

// Query rows a CTA works on: 16 for single tokens of grouped heads, 32 for a step's active rows;
// where a KV head has more, every slice of 32 reads the codes again, from L2. (Slices of 64 need
// 64 sums a thread beside 96 registers, and the exp warps take as long for 64 rows as for twice 32.)
int rows_per_cta(int rows) { return rows <= 16 ? 16 : 32; }

template <int FMT, int D, int NQ, bool SPARSE>
int launch_attention(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnArgs& a, cudaStream_t stream) {
  auto kern = cache_attn_kernel<FMT, D, NQ, SPARSE>;
  constexpr int bytes = static_cast<int>(Lay<FMT, D, NQ>::kBytes);
  if (const int st = configure_dynamic_smem(reinterpret_cast<const void*>(kern), bytes, "cache attention")) return st;
  cudaError_t e = launch_k(kern, dim3(a.grid), dim3(kThreads), bytes, stream, mk, mv, a);
  note_launch();
  if (e == cudaSuccess) {
    const long long rows = static_cast<long long>(a.B) * a.Hkv * a.g * a.qcap;
    e = launch_k(cache_combine_kernel<D, SPARSE>, dim3(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps)),
                 dim3(kJoinWarps * 32), 0, stream, a, NQ);
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
  return rows_per_cta(a.g * a.qcap) == 16 ? launch_attention<FMT, D, 16, SPARSE>(mk, mv, a, stream)
                                          : launch_attention<FMT, D, 32, SPARSE>(mk, mv, a, stream);
}

template <bool SPARSE>
int run_cache_attention(CacheAttnArgs a, const focus_cache* c, void* ws, cudaStream_t stream) {
  if (a.B == 0) return FOCUS_OK;
  const int rows = a.g * a.qcap, nq = rows_per_cta(rows);
  a.n_slices = (rows + nq - 1) / nq;
  a.slice_rows = (rows + a.n_slices - 1) / a.n_slices;
  // tiles at most, for the grid and for the 32-bit tile numbers
  const long long top = static_cast<long long>(a.table_cols) * a.page;      // (of G, what the table can hold)
  const long long gen = (std::min<long long>(a.G, top) + a.page - 2) / a.page + 1;
  const long long per_unit = SPARSE ? ((gen + a.C) * a.page + a.S + 127) / 128 : (top + 127) / 128;
  const long long most = static_cast<long long>(a.B) * a.Hkv * a.n_slices * (per_unit + kLead);
  if (most >= (1LL << 31) || static_cast<long long>(a.B) * a.Hkv * rows >= (1LL << 31)) {
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
  // (room for the current block's edge, the kept blocks' slots, the sinks and the last tile behind them)
  FOCUS_CHECK_ARG(static_cast<long long>(table_cols) * cache->page <= (1LL << 31) - (1LL << 18),
                  "table of more than 2^31 - 2^18 positions");
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
  a.page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
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
