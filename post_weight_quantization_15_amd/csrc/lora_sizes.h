// How the adapter product divides its rows and the k of its hidden values:
// plain arithmetic, asked by the workspace queries and by the launches.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace gptq {

// Rows of activations handled at once (bounds the reordered copy).
constexpr int64_t kRowChunk = 16384;
// Rows of a workgroup that forms hidden values.
constexpr int kShrinkRows = 32;

// Shares of k per row tile that a launch over n rows wants: enough workgroups
// for the chip where rows are few, of at least 8 steps of 32 each.
inline int shrink_shares(int64_t n, int64_t len) {
  const int64_t tiles = (n + kShrinkRows - 1) / kShrinkRows;
  return tiles >= 128 ? 1 : int(std::max<int64_t>(1, std::min<int64_t>(512 / tiles, (len + 511) / 512)));
}

// ... and gets, where `have` floats are kept for the shares' sums.
inline int shrink_shares(int64_t n, int64_t len, int rank, size_t have) {
  return int(std::max<int64_t>(1, std::min<int64_t>(shrink_shares(n, len), int64_t(have) / (n * rank))));
}

// Floats to keep for the shares' sums of a launch over n rows.
inline size_t shrink_floats(int64_t n, int64_t len, int rank) {
  const int shares = shrink_shares(n, len);
  return shares > 1 ? size_t(shares) * n * rank : 0;
}

// The same for n rows taken a chunk at a time: the last chunk is the shorter
// one and may want shares where a whole one wants none.
inline size_t shrink_floats_chunked(int64_t n, int64_t len, int rank) {
  const size_t whole = shrink_floats(std::min(n, kRowChunk), len, rank);
  const int64_t last = n % kRowChunk;
  return last ? std::max(whole, shrink_floats(last, len, rank)) : whole;
}

}  // namespace gptq
