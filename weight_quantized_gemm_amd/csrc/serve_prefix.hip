// Attention of a batch whose sequences share long prefixes: the softmax of a token runs over the keys of
// its group's prefix and over its sequence's own keys.
//
// Both parts are the work of serve_tree.hip's kernels.  A prefix is a tile row of its own: all tokens of the
// group's sequences, times the query heads of a cached head, are the rows that share its keys, so that a prefix is read
// once for a tile of them instead of once for each sequence.  A tile has up to 256 rows, by those of the mean group
// (plan_tree), so that one large group beside many small ones reads its prefix more often (48 sequences behind 8000 keys,
// 4 query heads for a cached one of 128: 56 us; with 16 prefixes of one sequence beside them 90); with heads of
// 256 it has 16 (32 sequences of 16 tokens behind prefixes of 12001 and 16001, 32 heads for 4: 1870 us, 113 TFLOP/s).  Neither part knows the other: each leaves
// (output, base, sum) of its rows, and the join adds up a row's parts of both,
//
//   out = sum_i 2^(base_i - base) output_i / sum_i 2^(base_i - base) sum_i.
//
// The rows of a tile of own keys lie in one or two tiles of the prefix, at places that follow from
// where the group's tiles begin, which the kernel of the prefix notes for each group.
//
// Long prefixes of many rows are bound by the matrix cores and the vector units (serve_tree.hip says how), the own keys
// by memory, few rows by the launches and the workgroups' starts.  Measured (kernel trace, after 200 calls, heads of 128): 32
// trees of 16 tokens behind two shared prompts of up to 16001, prefix 316 us, own keys 40, join 19 (212 GFLOP in 375 us:
// 565 TFLOP/s, 850 with the weights' second terms); 64 single tokens behind 32768, prefix 66 (520 TFLOP/s), own keys 43 (164 MB
// at 3.8 TB/s), join 11; 8 behind 2000, both parts by one launch 16.6, join 5.9.  A card that comes from idle takes some 50
// calls to its full clock: the first 30 of the trees' prefix take 376.
#include "serve_tree.h"
#include "serve_step_kernels.h"

namespace wq {
namespace {

struct JoinArgs {
  PartArgs own, shared;
  const int32_t* group_starts;
  int32_t group_count;
};

// The group that holds sequence b, or -1; group_starts ascend.  A wave looks at 64 places at a time.
__device__ __forceinline__ int find_group(const JoinArgs& a, int b, int lane) {
  int lo = 0, count = a.group_count;  // among [lo, lo + count)
  while (count > 0) {
    const int step = (count + 63) / 64, at = lo + lane * step;
    // starts ascend: the last place whose start is at most b
    const uint64_t upto = __ballot(lane * step < count && a.group_starts[at] <= b);
    if (!upto) return -1;
    const int last = 63 - __builtin_clzll(upto);
    lo += last * step;
    count = min(step, count - last * step);
    if (step == 1) break;
  }
  return count > 0 && b < a.group_starts[lo + 1] ? lo : -1;
}

// Grid and lanes as in tree_join_kernel (serve_tree.hip), over the tiles of own keys.
template <int HD, bool SPLIT>
constexpr int prefix_join_rows() { return (SPLIT ? 64 : 256) / (HD / 8); }

template <int HD, bool BF16, bool SPLIT>
__global__ __launch_bounds__(256) void prefix_join_kernel(const JoinArgs a) {
  constexpr int TPR = HD / 8, U = SPLIT ? 8 : 4;  // U: parts in flight
  __shared__ __align__(16) float sums[SPLIT ? 4 : 1][64][12];  // of each lane: 8 columns, the base, the sum
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.y * prefix_join_rows<HD, SPLIT>() + (SPLIT ? lane : (int)threadIdx.x) / TPR, c = lane % TPR;
  const int tiles = *a.own.tiles, step = SPLIT ? 4 : 1;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Cut cut = a.own.cuts[tile];
    const bool live = row < a.own.R && cut.row0 + row < cut.rows;
    // own parts: a whole tile's one, or as in tree_join_kernel
    const int own_parts = cut.parts < 0 ? 1 : cut.parts;
    const int64_t whole = 2 * (int64_t)a.own.blocks + tile;
    // the same row among those of the group, and its tile's parts there
    int parts = 0, first = 0, shared_row = 0;
    int64_t shared_whole = -1;
    const int g = find_group(a, cut.b, lane);
    if (g >= 0) {
      const Group gr = a.shared.groups[g];
      const int64_t at = (int64_t)(cut.q0 - gr.q0) * a.own.group + cut.row0 + row;
      if (live && at >= 0 && at < (int64_t)gr.tokens * a.own.group && gr.tile0 >= 0 && gr.tiles > 0) {
        const int64_t there = (int64_t)gr.tile0 + (int64_t)cut.kvh * gr.tiles + at / a.shared.R;
        if (there < *a.shared.tiles) {
          const Cut sc = a.shared.cuts[there];
          shared_row = (int)(at % a.shared.R);
          if (sc.q0 == gr.q0 && sc.kvh == cut.kvh && sc.row0 + shared_row == at) {
            parts = sc.parts < 0 ? 1 : sc.parts;
            first = sc.first;
            shared_whole = sc.parts < 0 ? 2 * (int64_t)a.shared.blocks + there : -1;
          }
        }
      }
    }
    const int all = own_parts + parts;
    auto place = [&](int i, const float*& out, const float*& ml) {
      const bool mine = i < own_parts;
      const PartArgs& s = mine ? a.own : a.shared;
      const int j = mine ? i : i - own_parts;
      const int64_t w = mine ? (cut.parts < 0 ? whole : -1) : shared_whole;
      const int64_t part = w >= 0 ? w : (int64_t)2 * ((mine ? cut.first : first) + j) + (j == 0 ? 1 : 0);
      const int64_t at = part * s.R + (mine ? row : shared_row);
      out = s.part + at * HD + 8 * c;
      ml = s.part_ml + 2 * at;
    };
    float base = kNone, sum = 0.f;
    f32x4_t y0 = f32x4_t{0.f, 0.f, 0.f, 0.f}, y1 = y0;
    for (int i0 = SPLIT ? wave : 0; live && i0 < all; i0 += U * step) {
      float ml[U][2], top = base;
      f32x4_t t0[U], t1[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {  // past the last part: it again, with no weight
        const float *out, *stat;
        place(min(i0 + step * i, all - 1), out, stat);
        ml[i][0] = stat[0];
        ml[i][1] = stat[1];
        t0[i] = *(const f32x4_t*)out;
        t1[i] = *(const f32x4_t*)(out + 4);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) top = fmaxf(top, ml[i][0]);
      const float off = top == kNone ? 0.f : top, keep = __builtin_amdgcn_exp2f(base - off);
      base = top;
      sum *= keep;
      y0 *= keep;
      y1 *= keep;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (i0 + step * i < all) {
          const float f = __builtin_amdgcn_exp2f(ml[i][0] - off);
          sum += f * ml[i][1];
          y0 += f * t0[i];
          y1 += f * t1[i];
        }
    }
    if constexpr (SPLIT) {
      float* mine = sums[wave][lane];
      *(f32x4_t*)mine = y0;
      *(f32x4_t*)(mine + 4) = y1;
      mine[8] = base;
      mine[9] = sum;
      __syncthreads();
      float top = kNone;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, sums[w][lane][8]);
      const float off = top == kNone ? 0.f : top;
      sum = 0.f;
      y0 = y1 = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(sums[w][lane][8] - off);
        sum += f * sums[w][lane][9];
        y0 += f * *(const f32x4_t*)sums[w][lane];
        y1 += f * *(const f32x4_t*)(sums[w][lane] + 4);
      }
      __syncthreads();  // read before the next tile's
    }
    if (live && (!SPLIT || wave == 0)) {
      const float inv = inverse(sum);
      const int tok = (int)divide((uint32_t)(cut.row0 + row), a.own.by_group);
      const int head = cut.kvh * a.own.group + cut.row0 + row - tok * a.own.group;
      *(u32x4_t*)(a.own.out + (int64_t)(cut.q0 + tok) * a.own.o_t + (int64_t)head * a.own.o_h + 8 * c) =
          u32x4_t{pack2<BF16>(y0[0] * inv, y0[1] * inv), pack2<BF16>(y0[2] * inv, y0[3] * inv),
                  pack2<BF16>(y1[0] * inv, y1[1] * inv), pack2<BF16>(y1[2] * inv, y1[3] * inv)};
    }
  }
}

// Prefix and own keys by one launch, where both take the kernel whose waves split the keys (tiles of 16 RT rows): neither
// waits for the other.
template <int HD, bool BF16, int RT>
hipError_t launch_keys(const JoinArgs& a, hipStream_t stream) {
  using L = KeysLds<HD, RT, true>;
  const auto kern = tree_keys_kernel<HD, BF16, RT, BothArgs>;
  const hipError_t e = raise_lds_limit((const void*)kern, L::Total);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.shared.blocks + a.own.blocks)), dim3(64 * L::NW), L::Total, stream,
                     BothArgs{{a.shared, a.own}});
  return hipGetLastError();
}

template <int HD, bool BF16>
hipError_t launch_both(const JoinArgs& a, const PrefixPlan& pl, hipStream_t stream) {
  if (a.group_count > 0 && !pl.shared.split_rows && !pl.own.split_rows) {
    if (pl.shared.rows != pl.own.rows) return hipErrorInvalidValue;
    if constexpr (HD != 256)
      if (pl.own.rows == 32) return launch_keys<HD, BF16, 2>(a, stream);
    return launch_keys<HD, BF16, 1>(a, stream);
  }
  hipError_t e = hipSuccess;
  if (a.group_count > 0) e = launch_parts<HD, BF16>(a.shared, pl.shared, stream);
  return e == hipSuccess ? launch_parts<HD, BF16>(a.own, pl.own, stream) : e;
}

template <int HD, bool BF16>
hipError_t launch(const JoinArgs& a, const PrefixPlan& pl, hipStream_t stream) {
  const hipError_t e = launch_both<HD, BF16>(a, pl, stream);
  if (e != hipSuccess) return e;
  const bool split = pl.split_join;
  const int rows = split ? prefix_join_rows<HD, true>() : prefix_join_rows<HD, false>();
  const dim3 grid((unsigned)std::min<int64_t>(pl.own.tiles, 1 << 20), (unsigned)((pl.own.rows + rows - 1) / rows));
  if (split) hipLaunchKernelGGL((prefix_join_kernel<HD, BF16, true>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((prefix_join_kernel<HD, BF16, false>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prefix(const PrefixProblem& p, const PrefixPlan& pl, float scale, void* workspace, hipStream_t stream) {
  static_assert(sizeof(Group) == kPrefixGroupBytes, "the plan's size of a group's note");
  char* ws = (char*)workspace;
  JoinArgs a{};
  a.group_starts = p.group_starts;
  a.group_count = (int32_t)p.shared.B;
  fill_args(a.shared, p.shared, pl.shared, scale, ws + pl.shared_notes, ws + pl.shared_parts,
            2 * pl.shared.blocks + pl.shared.tiles);
  fill_args(a.own, p.own, pl.own, scale, ws + pl.own_notes, ws + pl.own_parts, 2 * pl.own.blocks + pl.own.tiles);
  a.shared.group_starts = p.group_starts;
  a.shared.groups = (Group*)(ws + pl.groups);
  a.shared.seqs = (int32_t)p.own.B;
  const bool bf16 = p.own.act == WQ_BF16;
  switch (p.own.d) {
    case 64: return bf16 ? launch<64, true>(a, pl, stream) : launch<64, false>(a, pl, stream);
    case 128: return bf16 ? launch<128, true>(a, pl, stream) : launch<128, false>(a, pl, stream);
    default: return bf16 ? launch<256, true>(a, pl, stream) : launch<256, false>(a, pl, stream);
  }
}

}  // namespace wq
