// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = x3[t] + scale[i] * ((x1[t] @ A_i^T) @ B_i^T),   i = indices[t]
//
// Two kernels, h = x1 @ A_i^T (fp32, k split over workgroups) and out = x3 + h @ B_i^T.
//
// Tokens of one adapter need not stand together, and nothing is sorted: the token rows are
// cut into windows of 16 or 64, and a work item is one (window, distinct adapter of it)
// pair.  The item's product is taken for whole 16-row blocks of the window and only the rows
// of its adapter are stored, so a row never depends on its neighbours.  Up to kLoraSmallM
// tokens, windows are 16 rows and every workgroup finds its window's distinct adapters by
// itself, with one load of 16 indices and ballots: a launch less.  Beyond, windows are 64 rows
// and a first kernel lists the items; all steps of all items (64 k of the first product, 128 columns
// of the second) then stand in one row, of which each workgroup takes an equal share.  An item
// whose k are cut leaves a part of h from each of its workgroups, which the second product adds in
// order.
//
// Both products move far more memory than they multiply; what bounds them is how the reads
// meet the caches and channels:
//  * workgroups side by side on the chip take different columns of the same rows (second
//    product) or start at different k (first product).  Rows are a power of two apart in most
//    models; walked down in step, all of a chip's reads would meet on a few channels.
//  * each XCD takes a run of neighbouring items, so that its L2 holds the adapters of those only;
//  * operands go to LDS first (direct loads, each wave into its own), in rows of adjacent lanes, and
//    from there into the matrix cores' layout.  Loaded from memory in that layout, where lanes
//    that follow each other hold different rows, every lane is an access of its own: 389 us
//    instead of 125 us without the loads of B, for 16384 tokens x 8192 columns at rank 64.
//
// Measured (bf16, MI355X, a call with both products; kernels: medians under a tracer, which makes each a
// little longer):
//   1 token, rank 16, k = n = 4096: 8.9 us; kernels 3.8 and 5.3 us: two launches and the chain index ->
//     rank -> operands -> sum in each;
//   64 tokens of 32 adapters, rank 32, k = n = 8192 (fp16): 18.9 us for 26.8 MB; kernels 8.1 and
//     11.4 us: a workgroup lives for four rounds of loads, one stage ahead, and its launch and
//     start take as long as those;
//   16384 tokens of 8 adapters, rank 64, k = 4096, n = 8192: 205 us for 669 MB (3.3 TB/s; a copy runs at
//     5.2); 5 us the list, 49 us the first product (2.7 TB/s of x1), 156 us the second (3.4 TB/s: x3
//     and out through LDS, between loads of B that stand in the same queue).
#include <algorithm>

#include "serve_device.h"
#include "serve_kernels.h"
#include "serve_tile.h"
#include "wq_pipeline.h"

namespace wq {
namespace {

// A window (its first token), an adapter (-1: rows without one), its rank and scale, and the rows
// that have it.
struct Item {
  int64_t w0;
  uint64_t rows;
  int32_t key, rank;
  float scale;
};

struct LoraArgs {
  const uint16_t* x1;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* indices;
  const float* scale;
  const int32_t* ranks;
  const uint16_t* x3;
  uint16_t* out;
  float* h;               // [splits or parts][m][r]
  Item* items;            // 64-row windows: the lists, and the lengths
  int32_t* count;
  int64_t m, n, sx, s3, so, windows;
  int32_t k, r, L, splits, kchunk, slots, cols, col_blocks, rank_blocks;
  int32_t steps, shrink_blocks;  // 64-row windows: 64-k steps of an item, workgroups of the first product
};

// The adapter of this lane's row of the window at w0 (rows past m and lanes past the window:
// -2, no row; a row without adapter: -1).
template <int W>
__device__ __forceinline__ int lane_key(const LoraArgs& p, int64_t w0, int lane) {
  if (lane >= W || w0 + lane >= p.m) return -2;
  const int i = p.indices[w0 + lane];
  return (uint32_t)i < (uint32_t)p.L ? i : -1;
}

__device__ __forceinline__ Item make_item(const LoraArgs& p, int64_t w0, int key, uint64_t rows) {
  Item it{w0, rows, key, 0, 1.f};
  if (key >= 0) {
    it.rank = p.ranks ? min(max(p.ranks[key], 0), p.r) : p.r;
    if (p.scale) it.scale = p.scale[key];
  }
  return it;
}

// The items of 64-row windows.  The first item of window w is items[w]; the others of the windows of
// workgroup i of this kernel stand from items[windows + its first row] on, count[i] of them, in the order
// of the windows.  The order is part of the result: the shares cut an item's sum where it stands.
__global__ __launch_bounds__(256) void lora_items_kernel(const LoraArgs p) {
  __shared__ int32_t found[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t share = (p.windows + kLoraLists - 1) / kLoraLists, lo = blockIdx.x * share;
  const int64_t hi = min(p.windows, lo + share);
  int total = 0;
  for (int64_t w4 = lo; w4 < hi; w4 += 4) {  // a window for each wave
    const int64_t w = w4 + wave;
    const int mine = w < hi ? lane_key<64>(p, w * 64, lane) : -2;
    int keys = 0, nth = -1;  // of the window; the key whose first row is this lane's, or -1
    uint64_t its_rows = 0;
    for (uint64_t left = __ballot(mine >= -1); left; ++keys) {
      const int first = __builtin_ctzll(left);
      const uint64_t rows = __ballot(mine == __builtin_amdgcn_readlane(mine, first));
      left &= ~rows;
      if (lane == first) nth = keys, its_rows = rows;
    }
    if (lane == 0) found[wave] = max(keys - 1, 0);
    __syncthreads();
    int64_t at = p.windows + lo * 64 + total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < wave) at += found[i];
      total += found[i];
    }
    if (nth >= 0) p.items[nth == 0 ? w : at + nth - 1] = make_item(p, w * 64, mine, its_rows);
    __syncthreads();
  }
  if (threadIdx.x == 0) p.count[blockIdx.x] = total;
}

// 16-row windows: calls body(item, part) for this workgroup's items, `parts` workgroups to an item, parts
// fastest; each XCD has an eighth of the units.  One unit to a workgroup, windows x slots x parts of
// them, and a workgroup takes every slots-th distinct adapter of its window.
template <typename Body>
__device__ __forceinline__ void for_window(const LoraArgs& p, int parts, const Body& body) {
  const int lane = threadIdx.x & 63;
  const uint32_t u = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const int part = u % parts, slot = u / parts % p.slots;
  const int64_t w0 = (int64_t)(u / parts / p.slots) * 16;
  const int mine = lane_key<16>(p, w0, lane);  // windows past the last have no rows
  uint64_t left = __ballot(mine >= -1);
  for (int s = 0; left; ++s) {
    const int key = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t rows = __ballot(mine == key);
    left &= ~rows;
    if (s % p.slots == slot) body(make_item(p, w0, key, rows), part);
  }
}

// 64-row windows: where item i stands.
struct Lists {
  int own, upto;  // this lane's list: its items, and those up to and with it
  int64_t items, share;

  __device__ __forceinline__ explicit Lists(const LoraArgs& p) {
    static_assert(kLoraLists == 64, "a lane for each list");
    const int lane = threadIdx.x & 63;
    own = upto = p.count[lane];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(upto, o, 64);
      if (lane >= o) upto += t;
    }
    items = p.windows + uniform(__shfl(upto, 63, 64));
    share = (p.windows + kLoraLists - 1) / kLoraLists;
  }
  __device__ __forceinline__ int64_t at(const LoraArgs& p, int64_t i) const {
    if (i < p.windows) return i;
    const int e = (int)(i - p.windows), l = __builtin_ctzll(__ballot(upto > e));
    return p.windows + l * share * 64 + e - uniform(__shfl(upto - own, l, 64));
  }
};

// Shares of the first product's steps: so many that an item is cut into at most kLoraSplits parts.
struct Shares {
  int64_t total, n;
  __device__ __forceinline__ Shares(const LoraArgs& p, int64_t items) {
    total = items * p.rank_blocks * p.steps;
    const int64_t least = (p.steps + kLoraSplits - 3) / (kLoraSplits - 2);  // steps of a share
    n = max((int64_t)1, min((int64_t)p.shrink_blocks, total / least));
  }
  __device__ __forceinline__ int64_t begin(int64_t i) const { return total * i / n; }
  // the share that holds step s: the largest i with begin(i) <= s
  __device__ __forceinline__ int64_t of(int64_t s) const { return ((s + 1) * n - 1) / total; }
};

// ------------------------------------------------------------------------------- h = x1 A^T
// A wave's stage is a step of 64 k: 16 MT rows of x1, then 16 NT rows of A_i, 128 bytes each, with
// the chunks of a row in row_slot's places.
template <int MT, int NT>
struct ShrinkStage {
  static constexpr int X = MT * 2048, Bytes = (MT + NT) * 2048, Loads = 2 * (MT + NT);
};

// One item's h for NT 16-rank tiles from rank r0 and k kb .. ke - 1.  MT 16-row blocks
// from row w0 + 16 * m0.  The NW waves take 64-k steps in turn, two 16x16x32 MFMAs each (rows of
// x1 against rows of A_i), the next step on its way meanwhile, and their sums meet in LDS, in
// wave order.
template <bool BF16, int W, int MT, int NT, int NW>
__device__ __forceinline__ void shrink_item(const LoraArgs& p, uint8_t* lds, int64_t w0, int m0, int key, uint64_t rows,
                                            int r0, int kb, int ke, float* h) {
  using S = ShrinkStage<MT, NT>;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  f32x4_t acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // one load takes 8 rows; rows past m or r read the last one, and their sums are not stored
  const uint16_t* src[S::Loads];
#pragma unroll
  for (int i = 0; i < S::Loads; ++i) {
    const int row = 8 * i + (lane >> 3);  // of the stage
    const int c = 8 * row_slot<128>(row, lane & 7);
    if (i < 2 * MT) src[i] = p.x1 + min(w0 + 16 * m0 + row, p.m - 1) * p.sx + c;
    else src[i] = p.a + ((int64_t)key * p.r + min(r0 + row - 16 * MT, p.r - 1)) * p.k + c;
  }
  uint8_t* mine = lds + wave * 2 * S::Bytes;
  const uint32_t to = lds_address(lds) + wave * 2 * S::Bytes;
  const int full = (ke - kb) / 64;  // whole steps; the waves take them in turn from step `turn` on
  const int turn = W == 16 ? (int)(w0 / W % 1024) * NW : 0;  // (equal shares begin at different k by themselves)
  auto load = [&](int i, uint32_t stage) {
    const int k0 = kb + 64 * (int)((uint32_t)(i + turn) % (uint32_t)full);
#pragma unroll
    for (int l = 0; l < S::Loads; ++l) dma16_global(src[l] + k0, stage + 1024 * l);
  };
  auto multiply = [&](const uint8_t* stage) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4_t xf[MT];
      const int slot = 16 * row_slot<128>(l16, 4 * s + g);
#pragma unroll
      for (int t = 0; t < MT; ++t) xf[t] = *(const u32x4_t*)(stage + (16 * t + l16) * 128 + slot);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const u32x4_t af = *(const u32x4_t*)(stage + S::X + (16 * j + l16) * 128 + slot);
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t][j] = mfma16x16x32<BF16>(xf[t], af, acc[t][j]);
      }
    }
  };
  __syncthreads();  // the LDS has been read
  wave_wait<0>();
  int st = 0;
  if (wave < full) load(wave, to);
  for (int i = wave; i < full; i += NW, st ^= 1) {
    if (i + NW < full) {
      load(i + NW, to + (st ^ 1) * S::Bytes);
      wave_wait<S::Loads>();
    } else {
      wave_wait<0>();
    }
    multiply(mine + st * S::Bytes);
    // every read of this stage has returned before the next load into it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  const int k0 = kb + 64 * full;
  if (k0 < ke && wave == full % NW) {  // the k tail: 8-k pieces past ke are zeros on both sides
#pragma unroll
    for (int l = 0; l < S::Loads; ++l) {
      const int row = 8 * l + (lane >> 3);
      u32x4_t v = u32x4_t{0, 0, 0, 0};
      if (k0 + 8 * row_slot<128>(row, lane & 7) < ke) v = *(const u32x4_t*)(src[l] + k0);
      *(u32x4_t*)(mine + 1024 * l + 16 * lane) = v;
    }
    __builtin_amdgcn_wave_barrier();
    multiply(mine);
  }
  // block t of row blocks: element i of a lane is row 4 g + i, rank l16
  float* red = (float*)lds;
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(wave * 16 * MT + 16 * t + 4 * g + i) * (16 * NT) + 16 * j + l16] = acc[t][j][i];
  __syncthreads();
  for (int e = tid; e < 256 * MT * NT; e += 64 * NW) {
    const int row = e / (16 * NT), c = e % (16 * NT), wr = 16 * m0 + row;
    if (r0 + c >= p.r || !((rows >> wr) & 1)) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w * (256 * MT * NT) + e];
    h[(w0 + wr) * p.r + r0 + c] = v;
  }
}

constexpr int kShrinkWaves = 4;
template <int W, int NT>
constexpr int shrink_lds() {
  return kShrinkWaves * std::max(2 * ShrinkStage<W / 16, NT>::Bytes, 1024 * (W / 16) * NT);
}

template <bool BF16, int W, int NT>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(const LoraArgs p) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int NW = kShrinkWaves;
  if constexpr (W == 16) {
    // parts of an item: blocks of NT rank tiles x k splits, splits fastest
    for_window(p, p.splits * p.rank_blocks, [&](const Item& it, int part) {
      const int split = part % p.splits, r0 = part / p.splits * (16 * NT);
      // rows without an adapter; ranks past the adapter's (the first block does not wait for the rank)
      if (uniform(it.key) < 0 || (r0 > 0 && r0 >= uniform(it.rank))) return;
      const int kb = split * p.kchunk, ke = min(p.k, kb + p.kchunk);
      shrink_item<BF16, W, 1, NT, NW>(p, lds, uniform(it.w0), 0, uniform(it.key),
                                      (uint64_t)uniform((int64_t)it.rows), r0, kb, ke, p.h + (int64_t)split * p.m * p.r);
    });
  } else {
    const Lists lists(p);
    const Shares shares(p, lists.items);
    int64_t me = blockIdx.x;
    if (me >= shares.n) return;
    if ((shares.n & 7) == 0) me = (me & 7) * (shares.n >> 3) + (me >> 3);
    const int64_t end = shares.begin(me + 1);
    for (int64_t s = shares.begin(me); s < end;) {
      const int64_t ir = s / p.steps;  // item x block of NT rank tiles
      const int s0 = (int)(s - ir * p.steps), s1 = (int)min((int64_t)p.steps, s0 + (end - s));
      s += s1 - s0;
      const int64_t i = ir / p.rank_blocks;
      const int r0 = (int)(ir - i * p.rank_blocks) * (16 * NT);
      const Item it = p.items[lists.at(p, i)];
      if (r0 >= uniform(it.rank)) continue;
      float* h = p.h + (me - shares.of(ir * p.steps)) * p.m * p.r;  // this part's place
      const int key = uniform(it.key), kb = 64 * s0, ke = min(p.k, 64 * s1);
      const uint64_t rows = (uint64_t)uniform((int64_t)it.rows);
      const int64_t w0 = uniform(it.w0);
      // rows inside one 16-row block (single tokens, the ends of prompts) read that block only
      const int lo = __builtin_ctzll(rows) >> 4, hi = (63 - __builtin_clzll(rows)) >> 4;
      if (lo == hi) shrink_item<BF16, W, 1, NT, NW>(p, lds, w0, lo, key, rows, r0, kb, ke, h);
      else shrink_item<BF16, W, 4, NT, NW>(p, lds, w0, 0, key, rows, r0, kb, ke, h);
    }
  }
}

// ------------------------------------------------------------------------- out = x3 + h B^T
// Both factors of this product are 16-bit in the matrix cores, but h is fp32: it is taken as
// the sum of two 16-bit numbers, hi + lo, which are off by at most 2^-16 (bf16) or 2^-22 (fp16) of it.  A
// row is first scaled by a power of two to a largest magnitude in [1, 2) in bf16 and [2^14, 2^15) in fp16, whose
// last place of 2^-24 then is 2^-38 of that (an error of 2^-39 where it is more than 2^-22 of the number); the
// power comes back in fp32 at the end.  The contraction of one 16x16x32 MFMA
// covers 16 ranks twice, against hi (lanes 0..31) and lo (lanes 32..63).  This product is
// bound by x3 and out, so the doubled matrix work is free.
//
// The product is taken transposed (columns n as MFMA rows, tokens as MFMA columns), and of
// each pair of MFMAs lane group g computes columns 8 g .. 8 g + 7: a lane's results are then
// 16 contiguous bytes of one token's row.
template <bool BF16>
__device__ __forceinline__ uint32_t split_hi_lo(float v) {  // hi in bits 0-15, lo in bits 16-31
  const uint16_t hi = f32_to_act<BF16>(v);
  const float f = act_to_f32<BF16>(hi);
  // an infinite or NaN hi is the whole value: inf - inf must not make a NaN of it
  const uint16_t lo = __builtin_isfinite(f) ? f32_to_act<BF16>(v - f) : (uint16_t)0;
  return (uint32_t)hi | ((uint32_t)lo << 16);
}

// B in LDS: 32 columns of CH 16-byte chunks (8 ranks each), chunk c of column n in slot
// c ^ column_turn(n): the 16 columns that one read takes (4 neighbours of every 8) then stand in 16
// different places of the 256 bytes that a bank cycle covers.
constexpr int kSumRow = 36;  // floats of a row of 32 sums: rows 16 bytes apart in the banks
__device__ __forceinline__ int column_turn(int n) { return ((n >> 1) & 1) | (((n >> 3) & 3) << 1); }

// 16-row windows: parts of an item are blocks of p.cols columns.  A wave takes the window's rows (MT 16-row blocks) x 32
// columns at a time, and the ranks in blocks of up to 8 CH.  Its sums go through LDS, 16 rows at a time,
// so that four adjacent lanes read x3 and write the output in 64 bytes of a row.  Dynamic LDS: for
// each wave two stages of B and 16 rows of sums, then W rows of hp = (r rounded up to 16) + 4
// packed values, then W row factors.
template <bool BF16, int W, int CH>
__global__ __launch_bounds__(256, W == 64 ? 2 : CH == 8 ? 3 : 4) void lora_expand_kernel(const LoraArgs p) {
  extern __shared__ __align__(16) uint8_t stages[];
  constexpr int MT = W / 16, Stage = 32 * CH * 16, Loads = Stage / 1024, RB = 8 * CH;  // RB: ranks of a stage
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int r16 = (p.r + 15) & ~15, hp = r16 + 4;
  float* sums = (float*)(stages + 8 * Stage) + wave * (16 * kSumRow);
  uint32_t* lds = (uint32_t*)(stages + 8 * Stage + 4 * 16 * kSumRow * 4);
  float* factor = (float*)(lds + W * hp);
  uint8_t* mine = stages + wave * 2 * Stage;
  const uint32_t to = lds_address(stages) + wave * 2 * Stage;
  // columns n_lo .. n1 - 1 of an item, whose h has parts_of(block of ranks) parts
  auto expand_item = [&](const Item& it, int64_t n_lo, int64_t n1, const auto& parts_of) {
    const int key = uniform(it.key);
    const uint64_t rows = (uint64_t)uniform((int64_t)it.rows);
    const int64_t w0 = uniform(it.w0);
    int64_t nc = n_lo + wave * 32;
    if (key < 0 && p.x3 == p.out) return;  // nothing to add in place

    // Loads take any row or column of the tensors where theirs are past the end (what comes of it is not
    // stored, or is cleared below): without a condition they all go out at once.
    const uint16_t* bk = p.b + (int64_t)max(key, 0) * p.n * p.r;
    const int row4 = lane >> 2, col4 = 8 * (lane & 3);  // of each 16 rows x 32 columns of x3 and output
    u32x4_t x[MT];
    auto load_x = [&](int64_t nc) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        x[t] = u32x4_t{0, 0, 0, 0};
        if (p.x3 && ((rows >> (16 * t)) & 0xffff))
          x[t] = *(const u32x4_t*)(p.x3 + min(w0 + 16 * t + row4, p.m - 1) * p.s3 + min(nc + col4, p.n - 8));
      }
    };
    auto load_b = [&](int64_t nc, int r0, uint32_t stage) {  // ranks r0 .. + RB - 1
#pragma unroll
      for (int i = 0; i < Loads; ++i) {
        const int e = 64 * i + lane, n = e / CH, c = (e % CH) ^ (column_turn(n) & (CH - 1));
        dma16_global(bk + min(nc + n, p.n - 1) * p.r + min(r0 + 8 * c, p.r - 8), stage + 1024 * i);
      }
    };
    const bool busy = nc < n1;
    if (busy) {  // on their way while h is made ready
      load_x(nc);
      if (key >= 0) load_b(nc, 0, to);
    }

    const int rank = uniform(it.rank), nk = (rank + 15) / 16, steps = (rank + RB - 1) / RB;
    if (rank) {  // h of the adapter's rows: splits added in order, scaled, split into hi + lo
      __syncthreads();
      constexpr int TPR = 256 / W;  // threads of a row, four ranks each at a time
      const int row = tid / TPR, first = 4 * (tid % TPR);
      const bool have = (rows >> row) & 1;
      const float sc = it.scale;
      const float* hr = p.h + (w0 + row) * p.r;
      const int64_t step = p.m * p.r;
      float big = 0.f;
      auto keep = [&](f32x4_t v, int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = have && c + i < rank ? v[i] * sc : 0.f;
          if (__builtin_isfinite(v[i])) big = fmaxf(big, fabsf(v[i]));  // infinities and NaN stay what they are
        }
        *(f32x4_t*)(lds + row * hp + c) = v;
      };
      for (int r0 = 0; r0 < (CH == 8 ? 16 * nk : 1); r0 += RB) {  // blocks of ranks of the first product
        const int parts = parts_of(r0 / RB), r1 = min(16 * nk, r0 + RB);
        if (parts == 1) {
          for (int c = r0 + first; c < r1; c += 16 * TPR) {  // four loads in flight
            f32x4_t t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (have && c + 4 * TPR * i < rank) t[i] = *(const f32x4_t*)(hr + c + 4 * TPR * i);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + 4 * TPR * i < r1) keep(t[i], c + 4 * TPR * i);
          }
        } else {
          for (int c = r0 + first; c < r1; c += 4 * TPR) {
            f32x4_t t[kLoraSplits], v = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (have && c < rank) {  // all parts in flight
#pragma unroll
              for (int z = 0; z < kLoraSplits; ++z) t[z] = *(const f32x4_t*)(hr + min(z, parts - 1) * step + c);
#pragma unroll
              for (int z = 0; z < kLoraSplits; ++z)
                if (z < parts) v += t[z];
            }
            keep(v, c);
          }
        }
      }
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) big = fmaxf(big, __shfl_xor(big, o, 64));
      // 2^-e: exponent of the largest magnitude, kept where 2^-e and 2^e are normal numbers
      int e = big > 0.f ? (int)(__float_as_uint(big) >> 23) - 127 : 0;
      e = min(max(e - (BF16 ? 0 : 14), -126), 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      if (first == 0) factor[row] = __uint_as_float((uint32_t)(127 + e) << 23);
      for (int c = first; c < 16 * nk; c += 4 * TPR) {
        const f32x4_t v = *(const f32x4_t*)(lds + row * hp + c);
        *(u32x4_t*)(lds + row * hp + c) = u32x4_t{split_hi_lo<BF16>(v[0] * down), split_hi_lo<BF16>(v[1] * down),
                                                  split_hi_lo<BF16>(v[2] * down), split_hi_lo<BF16>(v[3] * down)};
      }
      __syncthreads();
    }
    if (!busy) return;

    // Of 8 columns of a row, those whose sums are not finite, summed anew in fp32 from h itself: against an infinity in B,
    // terms of unlike signs or a zero one make a NaN, and a row's factor may bring back what passed fp32.  The
    // row's factor f is in all of them then, and 1 afterwards.
    auto sum_apart = [&](float (&y)[8], float& f, int64_t row, int64_t n) {
      float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int r = 0; r < rank; ++r) {
        const int parts = parts_of(r / RB);
        float h = 0.f;
#pragma unroll 1
        for (int z = 0; z < parts; ++z) h += p.h[(z * p.m + row) * p.r + r];
        h *= it.scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = fmaf(h, act_to_f32<BF16>(bk[(n + i) * p.r + r]), s[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_isfinite(y[i]) ? f * y[i] : s[i];
      f = 1.f;
    };

    f32x4_t acc[2][MT];
    int st = 0;
#pragma unroll 1
    for (; nc < n1; nc += kLoraCols) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[e][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int s = 0; s < steps; ++s, st ^= 1) {
        const bool last = s + 1 == steps;
        if (!last || nc + kLoraCols < n1) {
          load_b(last ? nc + kLoraCols : nc, last ? 0 : RB * (s + 1), to + (st ^ 1) * Stage);
          wave_wait<Loads>();
        } else {
          wave_wait<0>();
        }
        const uint8_t* stage = mine + st * Stage;
#pragma unroll
        for (int j = 0; j < CH / 2; ++j) {
          const int c = RB * s + 16 * j + 8 * (g & 1);  // this lane's 8 ranks
          if (RB * s + 16 * j >= rank) break;
          u32x4_t hf[MT], bf[2];
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const u32x4_t* src = (const u32x4_t*)(lds + (16 * t + l16) * hp + c);
            const u32x4_t u = src[0], v = src[1];
            const uint32_t sel = g < 2 ? 0x05040100u : 0x07060302u;  // the hi or the lo halves
            hf[t] = u32x4_t{__builtin_amdgcn_perm(u[1], u[0], sel), __builtin_amdgcn_perm(u[3], u[2], sel),
                            __builtin_amdgcn_perm(v[1], v[0], sel), __builtin_amdgcn_perm(v[3], v[2], sel)};
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int n = 8 * (l16 >> 2) + 4 * e + (l16 & 3);
            bf[e] = *(const u32x4_t*)(stage + 16 * (n * CH + ((2 * j + (g & 1)) ^ (column_turn(n) & (CH - 1)))));
          }
          if (RB * s + 16 * j + 16 > rank) {  // columns past the rank hold anything
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const uint32_t keep = (c + 2 * d < rank ? 0x0000ffffu : 0u) | (c + 2 * d + 1 < rank ? 0xffff0000u : 0u);
              bf[0][d] &= keep;
              bf[1][d] &= keep;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[e][t] = mfma16x16x32<BF16>(bf[e], hf[t], acc[e][t]);
        }
        // every read of this stage has returned before the next load into it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      u32x4_t o[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        o[t] = x[t];
        if (rank) {
          // lane l16's row, columns 8 g .. + 7
          *(f32x4_t*)(sums + l16 * kSumRow + 8 * g) = acc[0][t];
          *(f32x4_t*)(sums + l16 * kSumRow + 8 * g + 4) = acc[1][t];
          __builtin_amdgcn_wave_barrier();
          const f32x4_t y0 = *(const f32x4_t*)(sums + row4 * kSumRow + col4);
          const f32x4_t y1 = *(const f32x4_t*)(sums + row4 * kSumRow + col4 + 4);
          float f = factor[16 * t + row4], z = 0.f;
          float y[8] = {y0[0], y0[1], y0[2], y0[3], y1[0], y1[1], y1[2], y1[3]};
#pragma unroll
          for (int i = 0; i < 8; ++i) z = fmaf(y[i], 0.f, z);
          const int wr = 16 * t + row4;
          if (z != 0.f && ((rows >> wr) & 1) && nc + col4 < n1) sum_apart(y, f, w0 + wr, nc + col4);
#pragma unroll
          for (int d = 0; d < 4; ++d)
            o[t][d] = pack2<BF16>(act_to_f32<BF16>((uint16_t)o[t][d]) + f * y[2 * d],
                                  act_to_f32<BF16>((uint16_t)(o[t][d] >> 16)) + f * y[2 * d + 1]);
          __builtin_amdgcn_wave_barrier();
        }
      }
      if (nc + kLoraCols < n1) load_x(nc + kLoraCols);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int wr = 16 * t + row4;
        if (((rows >> wr) & 1) && nc + col4 < n1) *(u32x4_t*)(p.out + (w0 + wr) * p.so + nc + col4) = o[t];
      }
    }
    if (rank == 0) wave_wait<0>();  // B was asked for; no load into the LDS is left
  };
  if constexpr (W == 16) {
    for_window(p, p.col_blocks, [&](const Item& it, int part) {
      expand_item(it, (int64_t)part * p.cols, min(p.n, ((int64_t)part + 1) * p.cols), [&](int) { return p.splits; });
    });
  } else {
    const Lists lists(p);
    const Shares shares(p, lists.items);
    const int64_t rounds = (p.n + kLoraCols - 1) / kLoraCols, total = lists.items * rounds;
    const int64_t me = (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3), end = total * (me + 1) / gridDim.x;
    for (int64_t u = total * me / gridDim.x; u < end;) {
      const int64_t i = u / rounds, c0 = u - i * rounds, c1 = min(rounds, c0 + (end - u));
      u += c1 - c0;
      expand_item(p.items[lists.at(p, i)], c0 * kLoraCols, min(p.n, c1 * kLoraCols), [&](int rb) {
        const int64_t s = (i * p.rank_blocks + rb) * p.steps;
        return (int)(shares.of(s + p.steps - 1) - shares.of(s)) + 1;
      });
    }
  }
}

// NT: 16-rank tiles of the first product's workgroups, and half the 16-byte chunks of a column of
// the second's stages.
template <bool BF16, int W, int NT>
hipError_t launch(const LoraArgs& a, const LoraPlan& pl, hipStream_t stream) {
  hipError_t e;
  if constexpr (W == 64) {
    hipLaunchKernelGGL(lora_items_kernel, dim3(kLoraLists), dim3(256), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  auto shrink = lora_shrink_kernel<BF16, W, NT>;
  if ((e = raise_lds_limit((const void*)shrink, shrink_lds<W, NT>())) != hipSuccess) return e;
  hipLaunchKernelGGL(shrink, dim3((unsigned)pl.shrink_blocks), dim3(64 * kShrinkWaves), (shrink_lds<W, NT>()), stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const size_t lds = 8 * (32 * 2 * NT * 16) + 4 * 16 * kSumRow * 4 + (size_t)W * (((a.r + 15) & ~15) + 4 + 1) * 4;
  auto expand = lora_expand_kernel<BF16, W, 2 * NT>;
  if ((e = raise_lds_limit((const void*)expand, (int)lds)) != hipSuccess) return e;
  hipLaunchKernelGGL(expand, dim3((unsigned)pl.expand_blocks), dim3(256), lds, stream, a);
  return hipGetLastError();
}

template <bool BF16, int W>
hipError_t launch_ranks(const LoraArgs& a, const LoraPlan& pl, hipStream_t stream) {
  if (pl.rank_tiles == 1) return launch<BF16, W, 1>(a, pl, stream);
  if (pl.rank_tiles == 2) return launch<BF16, W, 2>(a, pl, stream);
  return launch<BF16, W, 4>(a, pl, stream);
}

}  // namespace

hipError_t launch_lora(const LoraProblem& p, const LoraPlan& pl, void* workspace, hipStream_t stream) {
  LoraArgs a{};
  a.x1 = (const uint16_t*)p.x1; a.a = (const uint16_t*)p.a; a.b = (const uint16_t*)p.b;
  a.indices = p.indices; a.scale = p.scale; a.ranks = p.ranks;
  a.x3 = (const uint16_t*)p.x3; a.out = (uint16_t*)p.out; a.h = (float*)((char*)workspace + pl.list_bytes);
  a.count = (int32_t*)workspace;
  a.items = (Item*)((char*)workspace + 4 * kLoraLists);
  a.m = p.m; a.n = p.n; a.sx = p.sx; a.s3 = p.s3; a.so = p.so;
  a.k = p.k; a.r = p.r; a.L = (int32_t)p.L; a.splits = pl.splits; a.kchunk = pl.kchunk; a.slots = pl.slots; a.cols = pl.cols;
  a.windows = pl.windows; a.col_blocks = pl.col_blocks; a.rank_blocks = pl.rank_blocks;
  a.steps = (p.k + 63) / 64; a.shrink_blocks = (int32_t)pl.shrink_blocks;
  static_assert(sizeof(Item) == kLoraItemBytes, "the plan's size of the list");
  const bool bf16 = p.act == WQ_BF16;
  if (pl.window == 16) return bf16 ? launch_ranks<true, 16>(a, pl, stream) : launch_ranks<false, 16>(a, pl, stream);
  return bf16 ? launch_ranks<true, 64>(a, pl, stream) : launch_ranks<false, 64>(a, pl, stream);
}

}  // namespace wq
