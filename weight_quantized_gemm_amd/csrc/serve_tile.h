// Tile geometry that the serving operators' planners share with their kernels (host and
// device code; no HIP types).
#pragma once
#include <cstdint>

namespace wq {

// ---- adapters
// Up to here a window is 16 token rows, beyond 64: short windows need no list and no tokens side by
// side with one adapter, long ones read an adapter less often.  16 and 64 rows, bf16, rank 64, k = n = 4096: 27.4 us
// and 36.8 us for 1100 tokens of 4 requests, 87 us and 52 us for 3000 of 20, 145 us and 82 us for
// 4096 of 100; k = n = 8192, 2048 tokens of 200 requests: 126 us and 136 us.
constexpr int64_t kLoraSmallM = 2048;
constexpr int kLoraRankTiles = 4;      // most 16-rank tiles of one workgroup of the first product
constexpr int kLoraCols = 128;         // columns of one round of the second product's workgroups
constexpr int kLoraSplits = 8;         // most k splits of the first product
constexpr int kLoraItemBytes = 32;      // a work item in the lists of the 64-row windows, and the number of lists
constexpr int kLoraLists = 64;

// ---- tree attention
constexpr int tree_key_waves(int d) { return d == 256 ? 2 : 4; }   // waves that split the keys, 32 to a tile
constexpr int kTreeCutBytes = 32;      // what is noted of a tile for the join
constexpr int tree_row_keys(int waves) { return waves == 2 ? 32 : 64; }  // keys of a tile whose rows the waves split

}  // namespace wq
