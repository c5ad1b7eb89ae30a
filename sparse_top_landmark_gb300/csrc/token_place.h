// Where a new token stands in its sequence.  Plain C++ (no CUDA header), so that a host compiler takes
// it too: the extremes that a caller's arrays can hold are tested there.
#pragma once

#ifdef __CUDACC__
#define MITA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MITA_HOST_DEVICE inline
#endif

namespace mita {

// The position of row t, one of the new tokens begin <= t < end of a sequence that then has `len`
// tokens in all; -1 where the new tokens do not all have a place in [0, len).  In 64 bits: the
// arrays that begin, end and len come from may hold any 32-bit number, and their differences
// have 33 bits (in 32, begin = -2^31 + 10, end = 2^31 - 1 and len = -4 would give a position near
// 2^31, and a page number read from far behind the table).
MITA_HOST_DEVICE int token_position(int len, int begin, int end, int t) {
  const long long n = (long long)end - begin;
  const long long pos = len - ((long long)end - t);
  return len > 0 && n <= len && pos >= 0 && pos < len ? (int)pos : -1;
}

// Whether a sequence of `len` > 0 tokens fits a row of `width` pages of 1 << page_log2 tokens.
MITA_HOST_DEVICE bool fits_table(int len, int width, int page_log2) {
  return (len - 1) >> page_log2 < width;
}

}  // namespace mita
