// Planning of the serving operators: tile rows, splits and workspace sizes.  Host-only C++.
// The plans are for an MI355X's 256 compute units and depend on shapes alone, so that a size
// query answers without a device and a captured call keeps its workspace.
#include <algorithm>

#include "serve_problem.h"
#include "serve_tile.h"

namespace wq {
namespace {

constexpr int kCUs = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

LoraPlan plan_lora(const LoraProblem& p) {
  LoraPlan pl;
  if (p.m == 0) return pl;
  pl.window = p.m <= kLoraSmallM ? 16 : 64;
  pl.windows = ceil_div(p.m, pl.window);
  // Side-by-side work items of a 16-row window, whose rows may each have an adapter of their own:
  // all of them where there are few windows, otherwise 4, since most workgroups of more would find
  // nothing.  16 against 4 of them: 13.3 us and 20.1 us for 64 tokens of 64 adapters (rank 16, k = n =
  // 4096), 26.8 us and 23.2 us for 128 tokens of 64, 46 us and 37 us for 777 tokens of 100 requests.
  // Only where most rows of many windows differ does that rule lose (1500 tokens of 1500 requests
  // and 32 adapters: 87 us and 94 us), which the shapes do not tell.
  const int64_t distinct = std::min<int64_t>({p.L + 1, p.m, pl.window});
  if (pl.window == 16) pl.slots = (int)std::min<int64_t>(distinct, p.m <= 64 ? 16 : 4);
  pl.rank_tiles = p.r <= 16 ? 1 : p.r <= 32 ? 2 : kLoraRankTiles;
  pl.rank_blocks = (int)ceil_div(p.r, 16 * pl.rank_tiles);
  if (pl.window == 64) {  // as many workgroups as reside at once, both multiples of 8, share the steps
    pl.shrink_blocks = kCUs;
    pl.expand_blocks = 2 * kCUs;
    pl.list_bytes = align256(4 * kLoraLists + (p.m + 2 * pl.windows) * kLoraItemBytes);
    // parts of an item: its share is at least windows / kCUs items long, and never less than the least
    // that keeps the parts within kLoraSplits
    pl.splits = (int)std::min<int64_t>(kLoraSplits, kCUs / (pl.windows * pl.rank_blocks) + 2);
    pl.workspace = align256(pl.list_bytes + (int64_t)pl.splits * p.m * p.r * 4);
    return pl;
  }
  // k splits, a power of two, while workgroups are few: 2 adapters are counted for a window, so that up to 64
  // tokens have all 8.  (8 for more tokens instead of what is counted: 38.9 us for 37.3 us at 777 of 100 requests.)
  const int64_t most = ceil_div(p.k, 256);
  const int64_t items = pl.windows * 2 * pl.rank_blocks;
  while (2 * pl.splits <= std::min<int64_t>(kLoraSplits, most) && 2 * items * pl.splits <= 2 * kCUs) pl.splits *= 2;
  pl.kchunk = (int)(ceil_div(ceil_div(p.k, pl.splits), 64) * 64);
  pl.splits = (int)ceil_div(p.k, pl.kchunk);
  // second product: workgroups of whole rounds of columns, as many as reside at once if a larger
  // window has about two adapters
  const int64_t rounds = ceil_div(p.n, kLoraCols);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(rounds, 4 * kCUs / (pl.windows * (p.m <= 64 ? pl.slots : 2))));
  pl.cols = (int)(ceil_div(rounds, blocks) * kLoraCols);
  pl.col_blocks = (int)ceil_div(p.n, pl.cols);
  pl.shrink_blocks = ceil_div(pl.windows * pl.slots * pl.rank_blocks * pl.splits, 8) * 8;
  pl.expand_blocks = ceil_div(pl.windows * pl.slots * pl.col_blocks, 8) * 8;
  pl.workspace = align256((int64_t)pl.splits * p.m * p.r * 4);
  return pl;
}

TreePlan plan_tree(const TreeProblem& p) {
  TreePlan pl;
  if (p.N == 0 || p.B == 0) return pl;
  // Rows (tokens x heads that share a cached head) of the average sequence: a tile of too many rows
  // only pads, one of too few reads the keys again.  bf16, d = 128, 8 cached heads, 8192 keys:
  //   16 rows, 32 sequences: tiles of 16 rows 203 us, of 32 208 us
  //   20 rows, 32 sequences: tiles of 16 rows 383 us, of 32 204 us
  //   32 rows, 32 sequences: waves that split the keys 209 us, that split the rows (64) 221 us
  //   48 rows, 16 sequences: waves that split the keys 132 us, that split the rows (64) 126 us
  //   64 rows, 16 sequences: 2 waves 128 us, 4 141 us;  48 rows of 4 cached heads: 74 us, 79 us
  //   112 rows, 16 sequences: 2 waves 155 us, 4 143 us, 8 221 us
  //   256 rows, 16 sequences: 4 waves 240 us, 8 228 us;  512 rows, 8 sequences: 229 us, 218 us
  // At d = 256 the outputs of a wave of more than 16 rows, or of the other kernel as it stands, whose waves have
  // 32, would not fit its registers; that kernel with 16 rows a wave was not built.
  const int64_t rows = ceil_div(p.N, std::min(p.N, p.B)) * p.group;
  int per_cu = 1;  // workgroups that a compute unit holds: by LDS, and 8 waves of 256 registers
  if (rows <= 32 || p.d == 256) {
    pl.waves = tree_key_waves(p.d);
    pl.rows = rows <= 16 || p.d == 256 ? 16 : 32;
    pl.unit = 32 * pl.waves;
    per_cu = p.d == 64 ? 2 : 1;
  } else {
    pl.split_rows = true;
    pl.waves = rows <= 64 ? 2 : rows <= 128 ? 4 : 8;
    pl.rows = 32 * pl.waves;
    pl.unit = tree_row_keys(pl.waves);
    per_cu = 8 / pl.waves;
  }
  // tiles: each sequence with tokens has ceil(T_b * group / rows) for each cached head
  pl.tiles = (p.N * p.group / pl.rows + std::min(p.N, p.B)) * p.hkv;
  const int64_t units = std::max<int64_t>(1, ceil_div((int64_t)p.width * p.page, pl.unit));
  pl.blocks = std::min<int64_t>(kCUs * per_cu, pl.tiles * units);
  pl.notes_bytes = align256((pl.tiles + 1) * kTreeCutBytes);
  // two partial tiles for each workgroup: outputs, then (base, sum) of each row
  pl.workspace = align256(pl.notes_bytes + pl.blocks * 2 * pl.rows * (int64_t)(p.d + 2) * 4);
  return pl;
}

}  // namespace wq
