// Attention of each sequence's newest tokens (one token, a chain, a tree of drafts) over its
// pages of a key / value cache: out[i] = sum_j softmax_j(scale q_i . k_j) v_j over the keys that
// token i sees.
//
// Work.  The tokens of a sequence and the G query heads of one cached head share that head's
// keys, so they are the rows of one tile: row = token * G + query head, R rows.  A tile's keys
// are cut into units, and all units of all tiles stand in one row (sequence, cached head,
// tile, key).  Each workgroup takes an equal share of that row, wherever it begins and ends:
// ragged lengths, few long sequences and many short ones load the chip alike, without knowing a
// length on the host.  A tile that one workgroup holds whole is written by it; one that is cut
// leaves partial results (output, base, sum) that a second kernel joins in key order.  A
// workgroup has at most two such parts, its first and its last; the one that holds a tile's first
// keys notes what is to be joined.
//
// Two kernels, by the rows of the average sequence (plan_tree):
//   keys: up to 32 rows, bound by memory.  The waves of a workgroup split the keys; each streams
//     its own 32-key tiles through its own LDS and waits for nobody until they join at the end.
//   rows: more rows, bound by the matrix cores and the exponentials.  The waves split the rows,
//     32 each, and share every tile of K and V, so that a key is read from memory and into
//     LDS once for up to 256 rows.
// In both, K and V go straight from memory to LDS (16 bytes a lane, two stages); the rows of
// pages are found through slot numbers that the workgroup writes to LDS ahead.
//
// S^T = K Q^T (keys as MFMA rows, query rows as columns): element i of lane l is key 4 (l / 16) +
// i of row l % 16, so a row's maximum is two cross-lane steps away, its statistics stand in the
// lanes that need them, and the lane's own 8 weights of 32 keys are, in this order, the B
// operand of O^T += V^T P^T, if V^T takes the keys in the same order: two transpose reads of 4
// keys each.  The weights never leave the registers.
//
// Scores, sums and outputs are fp32 (base 2: scale * log2(e) is folded into the scores).  The base
// that is taken off a row's scores is the maximum of the tile that last set it, less kLow.  Weights may reach
// 2^(kLow + kSlack), which fp32 and both 16-bit types hold; a tile whose weights pass that is taken again,
// with its maximum found, the base raised and the outputs rescaled.  Most tiles thus find no
// maximum at all, which costs as many vector instructions as the weights themselves.  A weight
// enters the second product as two 16-bit terms, itself rounded and what the rounding left, for an error of at most
// 2^-16 (bf16) or 2^-22 (fp16) of it, and in fp16 2^-32 of the largest, less than the sums' own
// rounding.  One term would be off by as much as the result's last rounding is; the second costs nothing where
// memory bounds the kernel, and up to 28 % where the matrix cores do (512 rows: 238 us without it, 300 us).  The sums
// are taken of the same two terms, by the matrix cores (against ones), so that the weights add up to 1 exactly.
//
// Measured (MI355X, both kernels of a call):
//   64 single tokens over 2144 to 8192 keys, 8 cached heads of 128, fp16: 249 us for 1.36 GB, 5.4 TB/s; reads
//     of 256-byte pieces 2 KB apart, which a cache of 8 heads is made of, reach 6.1 TB/s with no
//     arithmetic at all;
//   one token over 1001 keys (4.1 MB): 13.1 us: two launches and the chain length -> page -> key ->
//     score -> join, in about 64 workgroups of 128 keys;
//   8 sequences of 60 to 64 drafted tokens over 5632 to 16384 keys, 64 query heads for 8 cached ones of 128,
//     bf16: 300 us, 600 TFLOP/s of the formula's products and 900 with those of the second terms, of the 1215
//     that a large product reaches.  The matrix cores are busy for 48 % of the cycles, the vector units for
//     47 % (exponentials, packing, addresses), LDS for 16 % without bank conflicts: what is lost
//     is that the two waves of a SIMD, held together by the shared tiles, do the same thing at the same time.
#include "serve_tree.h"

namespace wq {
namespace {

// ------------------------------------------------------------------------------ the join
// Grid x: tiles (the kernels note how many there are; past the grid, in turn), y: blocks of rows.  HD / 8
// lanes to a row, 8 columns each.  SPLIT: the four waves take every fourth part of the same rows
// and meet in LDS; otherwise each has rows of its own.  Where a workgroup's share is a small part
// of a tile there are many parts and few tiles (64 parts for 131072 keys of one sequence: 9 us
// split, 35 us one wave a row); where shares and tiles are alike, two parts and many rows (512 rows
// of 64 tiles: 20 us and 31 us split).
template <int HD, bool SPLIT>
constexpr int join_rows() { return (SPLIT ? 64 : 256) / (HD / 8); }

template <int HD, bool BF16, bool SPLIT>
__global__ __launch_bounds__(256) void tree_join_kernel(const TreeArgs a) {
  constexpr int TPR = HD / 8, U = SPLIT ? 8 : 4;  // U: parts in flight
  __shared__ __align__(16) float sums[SPLIT ? 4 : 1][64][12];  // of each lane: 8 columns, the base, the sum
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.y * join_rows<HD, SPLIT>() + (SPLIT ? lane : (int)threadIdx.x) / TPR, c = lane % TPR;
  const int tiles = *a.tiles, step = SPLIT ? 4 : 1;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Cut cut = a.cuts[tile];
    if (cut.parts == 0) continue;
    // part 0 is the first workgroup's second, part i the first of the workgroup i places on
    auto place = [&](int i) { return ((int64_t)2 * (cut.first + i) + (i == 0 ? 1 : 0)) * a.R + row; };
    const bool live = row < a.R && cut.row0 + row < cut.rows;  // (at d = 64 a block may be two tiles' rows high)
    float base = kNone, sum = 0.f;
    f32x4_t y0 = f32x4_t{0.f, 0.f, 0.f, 0.f}, y1 = y0;
    for (int i0 = SPLIT ? wave : 0; live && i0 < cut.parts; i0 += U * step) {
      float ml[U][2], top = base;
      f32x4_t t0[U], t1[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {  // past the last part: it again, with no weight
        const int64_t at = place(min(i0 + step * i, cut.parts - 1));
        ml[i][0] = a.part_ml[2 * at];
        ml[i][1] = a.part_ml[2 * at + 1];
        t0[i] = *(const f32x4_t*)(a.part + at * HD + 8 * c);
        t1[i] = *(const f32x4_t*)(a.part + at * HD + 8 * c + 4);
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
        if (i0 + step * i < cut.parts) {
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
      const int tok = (int)divide((uint32_t)(cut.row0 + row), a.by_group);
      const int head = cut.kvh * a.group + cut.row0 + row - tok * a.group;
      *(u32x4_t*)(a.out + (int64_t)(cut.q0 + tok) * a.o_t + (int64_t)head * a.o_h + 8 * c) =
          u32x4_t{pack2<BF16>(y0[0] * inv, y0[1] * inv), pack2<BF16>(y0[2] * inv, y0[3] * inv),
                  pack2<BF16>(y1[0] * inv, y1[1] * inv), pack2<BF16>(y1[2] * inv, y1[3] * inv)};
    }
  }
}

template <int HD, bool BF16>
hipError_t launch(const TreeArgs& a, const TreePlan& pl, hipStream_t stream) {
  const hipError_t e = launch_parts<HD, BF16>(a, pl, stream);
  if (e != hipSuccess) return e;
  const bool split = pl.blocks >= 4 * pl.tiles;  // four workgroups or more to a tile
  const int join = split ? join_rows<HD, true>() : join_rows<HD, false>();
  const dim3 grid((unsigned)std::min<int64_t>(pl.tiles, 1 << 20), (unsigned)((a.R + join - 1) / join));
  if (split) hipLaunchKernelGGL((tree_join_kernel<HD, BF16, true>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((tree_join_kernel<HD, BF16, false>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_tree(const TreeProblem& p, const TreePlan& pl, float scale, void* workspace, hipStream_t stream) {
  TreeArgs a{};
  fill_args(a, p, pl, scale, workspace, (char*)workspace + pl.notes_bytes, pl.blocks * 2);
  const bool bf16 = p.act == WQ_BF16;
  switch (p.d) {
    case 64: return bf16 ? launch<64, true>(a, pl, stream) : launch<64, false>(a, pl, stream);
    case 128: return bf16 ? launch<128, true>(a, pl, stream) : launch<128, false>(a, pl, stream);
    default: return bf16 ? launch<256, true>(a, pl, stream) : launch<256, false>(a, pl, stream);
  }
}

}  // namespace wq
