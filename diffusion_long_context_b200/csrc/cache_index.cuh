// Index arithmetic of the 8-bit cache that has to hold at the ends of its ranges: plain C++, so that
// a host compiler can check it.
#pragma once

#if defined(__CUDACC__)
#define FOCUS_HD __host__ __device__ __forceinline__
#else
#define FOCUS_HD inline
#endif

namespace focus {

// Vectors (2^vec_shift to a row) of a sequence's page j that hold one of its first len >= 0 positions.
// (Clamped before the shift: a page 2^27 rows behind len shifted to a number above zero.)
FOCUS_HD int stored_vectors(int len, int j, int page_shift, int vec_shift) {
  const int left = len - (j << page_shift), page = 1 << page_shift;
  return (left < 0 ? 0 : left < page ? left : page) << vec_shift;
}

}  // namespace focus
