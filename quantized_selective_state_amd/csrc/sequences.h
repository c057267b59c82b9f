// Rows of dense or packed sequences, as the kernels over (tokens, channels) tensors walk them.
#pragma once

#include <algorithm>

#include "block_internal.h"

namespace ssdq {

struct Span { int32_t begin, end; };

// offsets null: dense, every sequence `length` rows.  Offsets are clamped into the tensor, so that wrong ones cannot
// lead outside it; an end before its begin is a sequence without rows.
struct Sequences {
  const int32_t* offsets;
  int32_t sequences, tokens;
  FastDiv length;   // tokens / sequences, at least 1; not used with offsets

  __device__ __forceinline__ Span span(int64_t s) const {
    if (offsets == nullptr) {
      if (tokens == 0) return Span{0, 0};
      return Span{int32_t(s) * int32_t(length.d), (int32_t(s) + 1) * int32_t(length.d)};
    }
    const int32_t begin = min(max(offsets[s], 0), tokens), end = min(max(offsets[s + 1], 0), tokens);
    return Span{begin, max(begin, end)};
  }
  // the last sequence that begins at or before `row` (0 if none does): rows from `row` on are in it or in later ones
  __device__ __forceinline__ int32_t at(int32_t row) const {
    if (offsets == nullptr) return int32_t(fdiv(uint32_t(row), length));
    int32_t low = 0, high = sequences;   // offsets[low] <= row, or low == 0; offsets[high] > row, or high == sequences
    while (high - low > 1) {
      const int32_t middle = low + (high - low) / 2;
      if (offsets[middle] <= row) low = middle;
      else high = middle;
    }
    return low;
  }
  // From sequence s, whose span ends at or before `row`, on to the first that ends behind it (`sequences` if none does).
  // The next one is tried; the end of a run of empty ones is searched for.  With offsets in order the last sequence that
  // begins at or before `row` is the wanted one, or no row from `row` on is in any.
  __device__ __forceinline__ void advance(int32_t row, int32_t& s, Span& now) const {
    if (++s >= sequences) return;
    now = span(s);
    if (now.end > row) return;
    s = at(row);
    now = span(s);
    if (now.end <= row) s = sequences;
  }
};

inline Sequences make_sequences(const int32_t* offsets, int32_t sequences, int64_t tokens) {
  return Sequences{offsets, sequences, int32_t(tokens),
                   make_fastdiv(uint32_t(std::max<int64_t>(1, tokens / sequences)))};
}

}  // namespace ssdq
