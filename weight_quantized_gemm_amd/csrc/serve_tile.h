// Tile geometry that the serving operators' planners share with their kernels (host and
// device code; no HIP types).
#pragma once
#include <cstdint>

namespace wq {

// ---- adapters
constexpr int64_t kLoraSmallM = 1024;  // up to here a window is 16 token rows, beyond 64
constexpr int kLoraRankTiles = 4;      // 16-rank tiles that one workgroup of the first product computes

// ---- tree attention
constexpr int kTreeKeys = 32;                                      // keys of a wave's tile
constexpr int tree_waves(int d) { return d == 256 ? 2 : 4; }       // waves of a workgroup, by head dim
constexpr int tree_unit(int d) { return kTreeKeys * tree_waves(d); }  // keys of a workgroup's round
// Workgroups that share the work: what the LDS lets reside on 256 compute units at once.
constexpr int tree_max_blocks(int d) { return d == 64 ? 512 : 256; }

}  // namespace wq
