// Planning of the serving operators around a step's attention: splits and workspaces.  Host-only C++; like
// serve_plan.cpp the plans depend on shapes alone.
#include <algorithm>

#include "serve_step.h"
#include "serve_tile.h"

namespace wq {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

PrefixPlan plan_prefix(const PrefixProblem& p) {
  PrefixPlan pl;
  if (p.own.N == 0 || p.own.B == 0) return pl;
  pl.own = plan_tree(p.own);
  pl.shared = plan_tree(p.shared);  // without prefixes: nothing
  // Where the waves split the keys, heads of 128 take two waves to a workgroup and two workgroups to a compute unit, so
  // that one loads while the other finds its next piece (own keys of 64 sequences of 250 to 1000: 57 -> 50 us).  Prefix and
  // own keys then share one launch, and its rows.
  auto by_keys = [&](const TreePlan& t) { return t.tiles > 0 && !t.split_rows; };
  const int rows = by_keys(pl.own) && by_keys(pl.shared) ? std::max(pl.own.rows, pl.shared.rows) : 0;
  auto fit = [&](TreePlan& t, const TreeProblem& q) {
    if (!by_keys(t)) return;
    if (rows) t.rows = rows;
    t.waves = part_key_waves(q.d);
    t.unit = 32 * t.waves;
    t.tiles = (q.N * q.group / t.rows + std::min(q.N, q.B)) * q.hkv;
    const int64_t units = std::max<int64_t>(1, ceil_div((int64_t)q.width * q.page, t.unit));
    t.blocks = std::min<int64_t>(256 * (q.d == 256 ? 1 : 2), t.tiles * units);
  };
  fit(pl.own, p.own);
  fit(pl.shared, p.shared);
  // Where a tile of either kind has four parts or more (serve_tree.hip's join has figures of both sides).
  auto many = [](const TreePlan& t) { return t.tiles > 0 && t.blocks >= 4 * t.tiles; };
  pl.split_join = many(pl.own) || many(pl.shared);
  int64_t at = 0;
  auto take = [&](int64_t bytes) { const int64_t here = at; at += align256(bytes); return here; };
  auto parts = [&](const TreePlan& t) { return (2 * t.blocks + t.tiles) * t.rows * (int64_t)(p.own.d + 2) * 4; };
  pl.shared_notes = take(pl.shared.notes_bytes);
  pl.own_notes = take(pl.own.notes_bytes);
  pl.groups = take(p.shared.B * kPrefixGroupBytes);
  pl.shared_parts = take(parts(pl.shared));
  pl.own_parts = take(parts(pl.own));
  pl.workspace = at;
  return pl;
}

VerifyPlan plan_verify(const VerifyProblem& p) {
  VerifyPlan pl;
  if (p.B == 0) return pl;
  pl.unit = ceil_div(p.V, (int64_t)kVerifyUnits * kVerifyStep) * kVerifyStep;
  pl.units = ceil_div(p.V, pl.unit);
  // Workgroups of four waves: as many as give each of 256 compute units about eight, and a wave at least one unit.
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(ceil_div(pl.units, 4), ceil_div(8 * 256, p.B)));
  pl.chunk = ceil_div(ceil_div(pl.units, want), 4) * 4;
  pl.chunks = ceil_div(pl.units, pl.chunk);
  pl.sums = align256(p.B * kVerifyStateBytes);
  pl.refused = pl.sums + align256(p.B * pl.units * 8);
  pl.workspace = pl.refused + (p.draft ? 0 : align256(p.N * 4));
  return pl;
}

}  // namespace wq
