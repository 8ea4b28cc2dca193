// The 8-bit paged key/value cache: device view, code conversions and argument checks shared
// by the calls that write it (cache_rows.cu), read it (cache_attention.cu) and copy its pages
// (pages.cu).
#pragma once

#include <cuda_fp8.h>

#include "cache_index.cuh"
#include "focus_common.cuh"

namespace focus {

// Checks a cache and its table; n_mat_one: the call takes a single layer.
int check_cache(const focus_cache* c, const int32_t* table, int table_cols, bool n_mat_one);

#if defined(__CUDACC__)

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
  return unpair(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
  return unpair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
  return unpair(r);
}
// a b rounded to fp32, whatever is added to it: ptxas 12.9 makes one multiply-add of a packed
// product and a sum (mul2 and add2, each with its .rn), which rounds once, at the end.
__device__ __forceinline__ float2 round2(float2 a, float2 b) { return fma2(a, b, make_float2(0.f, 0.f)); }

template <int FMT>
struct CodeTop {
  static constexpr float value = FMT == FOCUS_CACHE_E4M3 ? 448.f : 127.f;
};

// Two codes of y0, y1 (the quotients x / s): e4m3 by the hardware conversion (nearest, ties to
// even, saturating), int8 by rounding to the nearest integer. |y| <= top * (1 + 2^-24), so
// saturation only ever takes back that last rounding of the quotient.
template <int FMT>
__device__ __forceinline__ uint32_t code2(float y0, float y1) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) {
    return __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
  } else {
    const int a = max(-127, min(127, __float2int_rn(y0))), b = max(-127, min(127, __float2int_rn(y1)));
    return static_cast<uint32_t>(a & 0xff) | (static_cast<uint32_t>(b & 0xff) << 8);
  }
}

// The values of the four codes of a word (exact in fp32).
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = static_cast<float>(static_cast<int8_t>(w >> (8 * j)));
  }
}

// The page of a table entry, or -1 (flagged) when it names none.
__device__ __forceinline__ int checked_page(const int32_t* table, int table_cols, int b, int col, int n_pages,
                                            int* dev_err) {
  int p = -1;
  if (col >= 0 && col < table_cols) p = table[static_cast<size_t>(b) * table_cols + col];
  if (p < 0 || p >= n_pages) {
    record_dev_error(dev_err, DEV_ERR_BAD_INDEX);
    return -1;
  }
  return p;
}

#endif  // __CUDACC__

}  // namespace focus
