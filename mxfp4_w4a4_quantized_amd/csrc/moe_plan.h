// Layout of an expert plan (int32 words), shared by the kernel that writes it
// (moe_route.hip), the products that read it and the C-ABI layer.
//
//   offsets [experts + 1]   first row of each expert, then the number of rows
//   order   [pairs]         pair (token * topk + choice) of each row; -1 behind the last
//   slot    [pairs]         row of each pair; -1 where its expert is not one of these
//   token   [pairs]         token of each row (order / topk); 0 behind the last
//   ntiles  [kHeights]      row tiles of each height
//   tiles   [kHeights][..]  their entries, 4 words: expert, first and end row of the
//                           expert, number of its first tile of this height
//   counts  [chunks][experts]   pairs of each chunk of the input by expert
//
// A product with row tiles of height h finds the expert and the rows of a
// workgroup with one 16-byte load, whatever the experts' sizes are.
#pragma once
#include <cstdint>

namespace mxfp4 {
namespace moe {

constexpr int kHeights = 4;                                  // rows of a tile: 16, 32, 128, 256
constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxPairs = int64_t(1) << 28;
constexpr int shift_of(int i) { return i < 2 ? 4 + i : 5 + i; }   // height i is 2^this
constexpr int height_index(int rows) { return rows == 16 ? 0 : rows == 32 ? 1 : rows == 128 ? 2 : 3; }
constexpr int64_t height(int i) { return int64_t(1) << shift_of(i); }

// Tiles of `rows` rows at most: a partial one per expert that has rows.
inline int64_t max_tiles(int64_t pairs, int64_t experts, int64_t rows) {
  return pairs / rows + (experts < pairs ? experts : pairs);
}

// Pairs per workgroup of the sort: one workgroup up to kOneChunk of them, then
// 1024 each on up to 128 workgroups (each of them adds up the others' counts).
constexpr int64_t kOneChunk = 4096;
inline int64_t chunk_pairs(int64_t pairs) {
  if (pairs <= kOneChunk) return kOneChunk;
  const int64_t c = (pairs + 127) / 128;
  return c <= 1024 ? 1024 : (c + 1023) / 1024 * 1024;
}
inline int64_t chunks(int64_t pairs) {
  const int64_t c = chunk_pairs(pairs);
  return pairs == 0 ? 1 : (pairs + c - 1) / c;
}

struct PlanLayout {   // word offsets
  int64_t order, slot, token, ntiles, tiles[kHeights], counts, words;
};

inline PlanLayout plan_layout(int64_t pairs, int64_t experts) {
  PlanLayout l;
  l.order = experts + 1;
  l.slot = l.order + pairs;
  l.token = l.slot + pairs;
  l.ntiles = (l.token + pairs + 3) / 4 * 4;
  int64_t at = l.ntiles + 8;
  for (int i = 0; i < kHeights; ++i) {
    l.tiles[i] = at;
    at += 4 * max_tiles(pairs, experts, height(i));
  }
  l.counts = at;
  l.words = at + (chunks(pairs) > 1 ? chunks(pairs) * experts : 0);
  return l;
}

}  // namespace moe
}  // namespace mxfp4
