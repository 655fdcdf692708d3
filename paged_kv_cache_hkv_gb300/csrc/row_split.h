// Word w of a stream of rows: its token and its place in the token's words, with the
// division by a product (quant.cu). Plain C++ but for the device's operator.
#pragma once

#include <cstdint>

namespace pkv {

// Below 2^31 words by a product with the divisor's reciprocal to 32 bits above its
// size, which is exact there (with the plain division and 64-bit slots the write
// issued in 83% of its cycles and took 23.8 us for the 16001 rows).
struct RowSplit {
  uint32_t mul, shift;
  int row_pair, vec_per_row;
#ifdef __CUDACC__
  template <typename Index>
  __device__ __forceinline__ int operator()(Index w, Index* tok) const {
    if constexpr (sizeof(Index) == 4)
      *tok = static_cast<Index>((__umulhi(mul, static_cast<uint32_t>(w)) + static_cast<uint32_t>(w)) >> shift);
    else
      *tok = w / row_pair;
    return static_cast<int>(w - *tok * row_pair);
  }
#endif
};

// w / d = (umulhi(mul, w) + w) >> shift for w < 2^31, with 2^(shift - 1) < d <= 2^shift
// and mul = floor(2^32 (2^shift - d) / d) + 1: (2^32 + mul) d exceeds 2^(32 + shift)
// by at most d <= 2^shift.
inline RowSplit row_split(int vec_per_row) {
  RowSplit s;
  s.vec_per_row = vec_per_row;
  s.row_pair = 2 * vec_per_row;
  s.shift = 0;
  while ((1ll << s.shift) < s.row_pair) ++s.shift;
  s.mul = static_cast<uint32_t>(((((1ull << s.shift) - s.row_pair) << 32) / s.row_pair) + 1);
  return s;
}

}  // namespace pkv
