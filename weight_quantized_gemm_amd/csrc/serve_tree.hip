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
#include <algorithm>
#include <cmath>

#include "serve_device.h"
#include "serve_kernels.h"
#include "serve_tile.h"
#include "wq_pipeline.h"

namespace wq {
namespace {

// What the join needs of a tile: its parts are the second part of workgroup `first` and the first
// parts of the next parts - 1.  parts 0: the tile was not cut.
struct Cut {
  int32_t parts, first, q0, kvh, row0, rows, pad[2];
};

struct TreeArgs {
  const uint16_t *q, *k, *v;
  const int32_t *table, *context, *starts;
  const uint32_t* mask;
  uint16_t* out;
  float* part;        // partial outputs [2 * blocks][R][d]
  float* part_ml;     // their (base, sum) [2 * blocks][R][2]
  Cut* cuts;          // of each tile, in the row's order
  int32_t* tiles;     // how many there are
  int64_t q_t, q_h, k_h, v_h, o_t, o_h;
  uint32_t k_row, v_row;  // bytes from one slot to the next
  int64_t pages, room;    // room: for this many cuts
  int32_t N, B, hkv, group, width, words, has_mask;
  int32_t blocks;     // workgroups of the launch
  int32_t R, unit;    // rows of a tile, keys of a unit
  FastDiv by_page, by_group;
  // The scores' factor, |scale| * log2(e), is positive, so that it neither turns the order of the
  // scores nor moves -inf; a negative scale flips the queries' signs, a zero one clears them.
  float scale;
  uint32_t q_and, q_xor;
};

// A base stands kLow below the maximum that sets it, and a weight may pass that maximum's by 2^kSlack.  bf16 has the
// range of fp32; of fp16's, all of the upper end is used: a weight's last place is 2^-24, so that one loses at
// most 2^-32 of the largest there (2^-25 with a base at the maximum, which summed up over a long context).
constexpr int kSlack = 8;
template <bool BF16> constexpr int kLow = BF16 ? 0 : 7;
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
constexpr float kNone = -__builtin_inff();

// ------------------------------------------------------------------------------ the schedule
struct Seq {
  int q0 = 0, tokens = 0, ctx = 0, len = 0;  // first query row, tokens, context, visible cache length
  int tiles = 0, units = 0;                  // row tiles of a cached head, units of a tile
};

__device__ __forceinline__ Seq sequence(const TreeArgs& a, int b) {
  Seq s;
  s.q0 = min(max(a.starts[b], 0), a.N);
  s.tokens = min(max(a.starts[b + 1], s.q0), a.N) - s.q0;
  s.ctx = max(a.context[b], 0);
  const int64_t len = (int64_t)s.ctx + s.tokens, most = a.pages ? (int64_t)a.width * a.by_page.d : 0;
  s.len = (int)min(len, most);
  s.tiles = (int)(((int64_t)s.tokens * a.group + a.R - 1) / a.R);
  s.units = max(1, (s.len + a.unit - 1) / a.unit);  // a tile without keys still writes zeros
  return s;
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ int64_t wave_upto(int64_t v, int lane) {  // of lanes 0 .. lane
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t t = __shfl_up(v, o, 64);
    if (lane >= o) v += t;
  }
  return v;
}
__device__ __forceinline__ int64_t units_of(const TreeArgs& a, const Seq& s) { return (int64_t)s.tiles * s.units * a.hkv; }

// 64 sequences as a wave sees them: lane l has sequence b0 + l, and the units and tiles up to and with
// it among the 64.
struct Sight {
  Seq mine;
  int64_t units = 0, tiles = 0;
};

__device__ __forceinline__ Sight see(const TreeArgs& a, int lane, int b0) {
  Sight c;
  if (b0 + lane < a.B) c.mine = sequence(a, b0 + lane);
  c.units = wave_upto(units_of(a, c.mine), lane);
  c.tiles = wave_upto((int64_t)c.mine.tiles * a.hkv, lane);
  return c;
}

__device__ __forceinline__ int64_t total_units(const TreeArgs& a, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < a.B; b += 64) sum += units_of(a, sequence(a, b));
  return wave_sum(sum);
}

// The sequence that holds unit u (u < total), and the units and tiles before it.
__device__ __forceinline__ int find_sequence(const TreeArgs& a, int lane, int64_t u, Seq& s, int64_t& before,
                                             int64_t& tiles_before) {
  int64_t base = 0, tiles = 0;
  for (int b0 = 0;; b0 += 64) {
    const Sight c = see(a, lane, b0);
    const uint64_t past = __ballot(base + c.units > u);
    if (past) {
      const int at = __builtin_ctzll(past);
      before = uniform(base + __shfl(c.units - units_of(a, c.mine), at, 64));
      tiles_before = uniform(tiles + __shfl(c.tiles - (int64_t)c.mine.tiles * a.hkv, at, 64));
      s.q0 = __builtin_amdgcn_readlane(c.mine.q0, at);
      s.tokens = __builtin_amdgcn_readlane(c.mine.tokens, at);
      s.ctx = __builtin_amdgcn_readlane(c.mine.ctx, at);
      s.len = __builtin_amdgcn_readlane(c.mine.len, at);
      s.tiles = __builtin_amdgcn_readlane(c.mine.tiles, at);
      s.units = __builtin_amdgcn_readlane(c.mine.units, at);
      return b0 + at;
    }
    base += __shfl(c.units, 63, 64);
    tiles += __shfl(c.tiles, 63, 64);
  }
}

// Workgroups that share `total` units, and the first unit of share i.
__device__ __forceinline__ int64_t shares(const TreeArgs& a, int64_t total) { return min((int64_t)a.blocks, total); }
__device__ __forceinline__ int64_t share_begin(int64_t total, int64_t n, int64_t i) { return total * i / n; }
// The share that holds unit u: the largest i with total * i / n <= u.
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t n, int64_t u) { return ((u + 1) * n - 1) / total; }

// ------------------------------------------------------------------------------ a tile of keys
template <int HD, int KT>
struct Cfg {
  static constexpr int CH = HD / 8, RB = HD * 2;              // 16-byte chunks and bytes of a row
  static constexpr int Half = KT * RB, Stage = 2 * Half;      // K, then V
  static constexpr int Loads = Half / 1024;                   // per tensor and tile, 1 KB each
};

// 16-byte chunk c of K row r stands in slot row_slot (16-byte reads of 16 rows at one chunk hit all
// banks); the 32-byte pair p of V row r in pair_slot (a transpose read takes 32 bytes of 8 rows).
// Rows of 512 bytes start in the same bank as rows of 256, so they take the latter's pattern.
template <int HD> __device__ __forceinline__ uint32_t k_chunk(uint32_t r, uint32_t c) {
  if constexpr (HD == 64) return c ^ ((r / 2) % 8);  // row_slot<128>
  else return c ^ (r % 16);
}
template <int HD> __device__ __forceinline__ uint32_t v_chunk(uint32_t r, uint32_t c) {
  if constexpr (HD == 64) return c ^ (2 * ((r / 2) % 4));  // pair_slot<128>
  else return c ^ (2 * (r % 8));
}

// Load part `w` of `parts` of a tile, to LDS address `stage`: keys first + 0 .. KT - 1 of the slots in LDS.
template <int HD, int KT, int PARTS>
__device__ __forceinline__ void load_tile(const TreeArgs& a, const uint16_t* kh, const uint16_t* vh, const int* slots,
                                          int first, uint32_t stage, int w, int lane) {
  using C = Cfg<HD, KT>;
  static_assert(C::Loads % PARTS == 0, "whole loads for each wave");
  asm volatile("" : "+v"(lane));  // addresses are made anew for each tile: kept, they would take 100 registers
  stage += 1024 * (C::Loads / PARTS) * w;
  const uint32_t e0 = (uint32_t)(64 * (C::Loads / PARTS) * w + lane);
#pragma unroll
  for (int i = 0; i < C::Loads / PARTS; ++i) {
    const uint32_t row = (e0 + 64 * i) / C::CH, c = (e0 + 64 * i) % C::CH;
    const uint32_t slot = (uint32_t)max(slots[first + row], 0);  // no such key: any row of the cache
    dma16_global((const uint8_t*)kh + (uint64_t)slot * a.k_row + 16 * k_chunk<HD>(row, c), stage + 1024 * i);
    dma16_global((const uint8_t*)vh + (uint64_t)slot * a.v_row + 16 * v_chunk<HD>(row, c), stage + C::Half + 1024 * i);
  }
}

template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t half) {
  const uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  return (half & e) == e;
}

// Edge tiles hold keys that some row does not see: past the end, on no page, or drafted tokens.
// The scores of unseen keys become -inf there, and V loses, for the matrix product, its rows
// without a key and its infinities and NaN (0 * inf would reach rows that do not see them); what
// those contribute to rows that do see them is added afterwards, with fp32 weights.  In a tile that is no
// edge they are met by the product, whose 16-bit terms make a NaN of an infinity where they have
// unlike signs or are 0: a piece of work whose outputs show any (finite) is taken again, with all its tiles as edges.

// Bit r: whether key r of the tile exists.
template <int KT>
__device__ __forceinline__ uint64_t tile_keys(const int* slots, int first, int lane) {
  return __ballot(lane < KT && slots[first + (lane & (KT - 1))] >= 0);
}

// Part `w` of `parts` of V without what the product must not meet; returns the rows (bits) of this
// part that held an infinity or NaN.
template <int HD, bool BF16, int KT, int PARTS>
__device__ __forceinline__ uint64_t clean_values(uint8_t* stage, uint64_t keys, int w, int lane) {
  using C = Cfg<HD, KT>;
  uint64_t odd = 0;
#pragma unroll 1
  for (int e = w * (KT * C::CH / PARTS) + lane; e < (w + 1) * (KT * C::CH / PARTS); e += 64) {
    const int row = e / C::CH;
    u32x4_t* at = (u32x4_t*)(stage + C::Half + 16 * e);
    u32x4_t x = *at;
    bool change = !((keys >> row) & 1);
    if (change) x = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const bool lo = not_finite<BF16>(x[d]), hi = not_finite<BF16>(x[d] >> 16);
      if (lo || hi) {
        odd |= 1ull << row;
        change = true;
        x[d] &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
      }
    }
    if (change) *at = x;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) odd |= (uint64_t)__shfl_xor((long long)odd, o, 64);
  return odd;
}

// Which of the 32 keys from drafted token draft0 on (negative: the context's end) a token sees,
// as far as the mask goes: 32 bits of its row of the mask, which two words hold.
__device__ __forceinline__ uint32_t tile_bits(const TreeArgs& a, const Seq& s, int token, int draft0) {
  if (draft0 <= -32) return ~0u;
  if (!a.has_mask) {  // drafted tokens 0 .. token
    const int last = token - draft0;
    return last < 0 ? 0u : last >= 31 ? ~0u : (2u << last) - 1u;
  }
  const uint32_t* row = a.mask + (int64_t)(s.q0 + token) * a.words;
  const int w = draft0 >> 5, shift = draft0 & 31;  // w may be -1: the context, which is seen
  const uint64_t lo = w < 0 ? ~0u : w < a.words ? row[w] : 0u;
  const uint64_t hi = w + 1 < a.words ? row[w + 1] : 0u;
  return (uint32_t)(((hi << 32) | lo) >> shift);
}

// The maximum of a value over the four lanes l % 16 + 16 * {0, 1, 2, 3}, in all of them.
__device__ __forceinline__ float across_max(float v) {
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
  const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// What a wave keeps of its RT 16-row blocks: queries (MFMA B operands), tokens, outputs
// (transposed: element i of o[t][d] is column 16 d + 4 (l / 16) + i of row l % 16), bases and sums
// (the four elements of l alike).
template <int HD, int RT>
struct Rows {
  u32x4_t q[RT][HD / 32];
  int token[RT];
  f32x4_t o[RT][HD / 16];
  f32x4_t l[RT];
  float m[RT];
};

template <int HD, bool BF16, int RT>
__device__ __forceinline__ void start_rows(const TreeArgs& a, const Seq& s, int kvh, int row0, int rows, int lane,
                                           Rows<HD, RT>& w) {
  const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = min(row0 + 16 * t + l16, rows - 1);
    w.token[t] = (int)divide((uint32_t)row, a.by_group);
    const int head = kvh * a.group + row - w.token[t] * a.group;
    const uint16_t* qr = a.q + (int64_t)(s.q0 + w.token[t]) * a.q_t + (int64_t)head * a.q_h + 8 * g;
#pragma unroll
    for (int j = 0; j < HD / 32; ++j) w.q[t][j] = (*(const u32x4_t*)(qr + 32 * j) & a.q_and) ^ a.q_xor;
    w.m[t] = kNone;
    w.l[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) w.o[t][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
}

// A tile of KT keys for NT of a wave's row blocks, from block t0 on.
//
// SLOW: finds the rows' maxima, raises their bases and rescales what has been summed; and of an edge
// tile it takes `keys` that exist, drafted tokens from draft0 on (the tile's first key; at most -KT: none),
// and the rows `odd` of V that clean_values took infinities or NaN from.  Otherwise all keys are seen and
// the bases stay; returns false, with nothing summed, where a row has no base yet or a weight
// passes 2^(kLow + kSlack).
template <int HD, bool BF16, int RT, int NT, int KT, bool SLOW>
__device__ __forceinline__ bool compute_rows(const TreeArgs& a, const Seq& s, const int* slots, int first, int draft0,
                                             uint64_t keys, uint64_t odd, const uint8_t* stage, const uint16_t* vh,
                                             int lane, const int t0, Rows<HD, RT>& w) {
  using C = Cfg<HD, KT>;
  constexpr int KB = KT / 16;
  if constexpr (!SLOW) {
    bool unset = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) unset |= w.m[t0 + t] == kNone;
    if (__ballot(unset)) return false;
  }
  asm volatile("" : "+v"(lane));  // as in load_tile
  const int l16 = lane & 15, g = lane >> 4;
  f32x4_t sc[NT][KB];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int h = 0; h < KB; ++h) sc[t][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // row 16 h + l16's chunk 4 j + g: the places of rows 16 apart are alike, and those of chunks 4 apart
  // differ by an exclusive or
  const uint32_t k0 = l16 * C::RB + 16 * k_chunk<HD>(l16, g);
#pragma unroll
  for (int j = 0; j < HD / 32; ++j)
#pragma unroll
    for (int h = 0; h < KB; ++h) {
      const u32x4_t kf = *(const u32x4_t*)(stage + (k0 ^ (64 * j)) + 16 * h * C::RB);
#pragma unroll
      for (int t = 0; t < NT; ++t) sc[t][h] = mfma16x16x32<BF16>(kf, w.q[t0 + t][j], sc[t][h]);
    }

  // vector instructions first: the other wave of the SIMD is then sooner at its matrix products
  // (512 rows, before the weights' second terms: 243 -> 238 us)
  if constexpr (!SLOW) __builtin_amdgcn_s_setprio(1);
  uint32_t seen[NT][KT / 32];  // SLOW: bit r of word b, whether this lane's row sees key 32 b + r
  if constexpr (SLOW) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int b = 0; b < KT / 32; ++b) {
        seen[t][b] = (uint32_t)(keys >> (32 * b)) & tile_bits(a, s, w.token[t0 + t], draft0 + 32 * b);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen[t][b] >> (16 * h + 4 * g + i)) & 1)) sc[t][2 * b + h][i] = kNone;
      }
      float top = sc[t][0][0];
#pragma unroll
      for (int h = 0; h < KB; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[t][h][i]);
      const float now = fmaxf(w.m[t0 + t], across_max(top) * a.scale - kLow<BF16>);
      const float keep = __builtin_amdgcn_exp2f(w.m[t0 + t] - (now == kNone ? 0.f : now));
      w.m[t0 + t] = now;
      w.l[t0 + t] *= keep;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) w.o[t0 + t][d] *= keep;
    }
  }

  u32x4_t pf[NT][KT / 32], pl[NT][KT / 32];  // pl: what the rounding of pf left
  u16x2_t most = {0, 0};  // of the weights' bits, which order like the weights (a NaN is above all)
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float base = SLOW && w.m[t0 + t] == kNone ? 0.f : w.m[t0 + t];  // no key seen so far: every weight is 0
#pragma unroll
    for (int h = 0; h < KB; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[t][h][i] = __builtin_amdgcn_exp2f(fmaf(sc[t][h][i], a.scale, -base));
#pragma unroll
    for (int b = 0; b < KT / 32; ++b) {
      pf[t][b] = u32x4_t{pack2<BF16>(sc[t][2 * b][0], sc[t][2 * b][1]), pack2<BF16>(sc[t][2 * b][2], sc[t][2 * b][3]),
                         pack2<BF16>(sc[t][2 * b + 1][0], sc[t][2 * b + 1][1]),
                         pack2<BF16>(sc[t][2 * b + 1][2], sc[t][2 * b + 1][3])};
      asm volatile("" : "+v"(pf[t][b]));  // rounded once: it is not made again for the product
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = pf[t][b][e];
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2_t, two));
      }
    }
  }
  if constexpr (!SLOW) {
    constexpr uint16_t kMost = BF16 ? (127 + kSlack) << 7 : (15 + kLow<BF16> + kSlack) << 10;
    if (__ballot(most[0] > kMost || most[1] > kMost)) {
      __builtin_amdgcn_s_setprio(0);
      return false;
    }
  }

  if constexpr (!SLOW) __builtin_amdgcn_s_setprio(0);
  constexpr uint32_t kOne2 = BF16 ? 0x3f803f80u : 0x3c003c00u;

  // V^T: column 16 d + l16, keys 4 g .. + 3 and 16 + 4 g .. + 3 of each 32; rows 16 apart and columns 16
  // apart as above
  const uint32_t vr = 4 * g + (l16 >> 2), v0 = vr * C::RB + 16 * v_chunk<HD>(vr, (l16 & 3) >> 1) + 8 * (l16 & 1);
  const uint8_t* vs = stage + C::Half;
#pragma unroll
  for (int b = 0; b < KT / 32; ++b) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w.l[t0 + t] = mfma16x16x32<BF16>(u32x4_t{kOne2, kOne2, kOne2, kOne2}, pf[t][b], w.l[t0 + t]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p0 = sc[t][2 * b + e / 2][2 * (e & 1)], p1 = sc[t][2 * b + e / 2][2 * (e & 1) + 1];
        pl[t][b][e] = pack2<BF16>(p0 - act_to_f32<BF16>((uint16_t)pf[t][b][e]),
                                  p1 - act_to_f32<BF16>((uint16_t)(pf[t][b][e] >> 16)));
      }
      w.l[t0 + t] = mfma16x16x32<BF16>(u32x4_t{kOne2, kOne2, kOne2, kOne2}, pl[t][b], w.l[t0 + t]);
    }
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
      const u32x2_t lo = lds_read_tr16(vs + (v0 ^ (32 * d)) + 32 * b * C::RB);
      const u32x2_t hi = lds_read_tr16(vs + (v0 ^ (32 * d)) + (32 * b + 16) * C::RB);
      const u32x4_t vf = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        w.o[t0 + t][d] = mfma16x16x32<BF16>(vf, pf[t][b], w.o[t0 + t][d]);
        w.o[t0 + t][d] = mfma16x16x32<BF16>(vf, pl[t][b], w.o[t0 + t][d]);
      }
    }
  }

  if constexpr (SLOW) {
    while (odd) {
      const int r = __builtin_ctzll(odd);
      odd &= odd - 1;
      const uint16_t* vr = (const uint16_t*)((const uint8_t*)vh + (uint64_t)(uint32_t)slots[first + r] * a.v_row) + 4 * g;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float p = 0.f;  // the row's weight of key r, from the lane that has it
        uint32_t sees = 0;
#pragma unroll
        for (int h = 0; h < KB; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((r >> 4) == h && (r & 3) == i) p = sc[t][h][i];
#pragma unroll
        for (int b = 0; b < KT / 32; ++b)
          if ((r >> 5) == b) sees = (seen[t][b] >> (r & 31)) & 1;
        p = __shfl(p, l16 + 16 * ((r >> 2) & 3), 64);
#pragma unroll
        for (int d = 0; d < HD / 16; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            asm volatile("" ::: "memory");  // one element at a time: this path is rare, registers are not plenty
            const uint16_t x = vr[16 * d + i];
            if (not_finite<BF16>(x) && sees) w.o[t0 + t][d][i] += p * act_to_f32<BF16>(x);
          }
      }
    }
  }
  return true;
}

// All of a wave's row blocks: at once, where that will do (false: nothing was done) ...
template <int HD, bool BF16, int RT, int KT>
__device__ __forceinline__ bool compute_fast(const TreeArgs& a, const uint8_t* stage, int lane, Rows<HD, RT>& w) {
  return compute_rows<HD, BF16, RT, RT, KT, false>(a, Seq{}, nullptr, 0, 0, 0, 0, stage, nullptr, lane, 0, w);
}
// ... or one by one, which takes fewer registers.  The loops over tiles below keep to the first form
// and leave for the second: in one loop with both, the outputs would change registers at every
// tile (40 moves).
template <int HD, bool BF16, int RT, int KT>
__device__ __forceinline__ void compute_slow(const TreeArgs& a, const Seq& s, const int* slots, int first, bool edge,
                                             int draft0, uint64_t keys, uint64_t odd, const uint8_t* stage,
                                             const uint16_t* vh, int lane, Rows<HD, RT>& w) {
  if (!edge) {
    keys = ~0ull;
    odd = 0;
    draft0 = -KT;
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
    compute_rows<HD, BF16, RT, 1, KT, true>(a, s, slots, first, draft0, keys, odd, stage, vh, lane, t, w);
}

// Whether a wave's outputs are all finite.
template <int HD, int RT>
__device__ __forceinline__ bool finite(const Rows<HD, RT>& w) {
  float z = 0.f;
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int d = 0; d < HD / 16; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) z = fmaf(w.o[t][d][i], 0.f, z);
  return z == 0.f;
}

// 1 / sum; no key seen: 0; NaN stays
__device__ __forceinline__ float inverse(float sum) { return sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f; }

// ------------------------------------------------------------------------------ a workgroup's share
// A piece of work: keys [key_lo, key_hi) of rows row0 .. of a tile.
struct Piece {
  Seq s;
  int b, kvh, row0, rows;      // rows: of the sequence and cached head
  int key_lo, key_hi;
  int whole, begins;           // whether all units of the tile, and its first
  int64_t tile_end, tile_id;   // the unit past the tile; its place among all tiles
};

// The piece at unit u of the share that ends at u_end; u moves past it.
__device__ __forceinline__ Piece next_piece(const TreeArgs& a, int lane, int64_t& u, int64_t u_end) {
  Piece p;
  int64_t before, tiles_before;
  p.b = find_sequence(a, lane, u, p.s, before, tiles_before);
  const int64_t in = u - before;
  const int tile = (int)(in / p.s.units), u0 = (int)(in - (int64_t)tile * p.s.units);
  const int u1 = (int)min((int64_t)p.s.units, u0 + (u_end - u));
  u = uniform(u + u1 - u0);
  p.kvh = uniform(tile / p.s.tiles);
  p.row0 = uniform((tile - p.kvh * p.s.tiles) * a.R);
  p.rows = p.s.tokens * a.group;
  p.key_lo = uniform(u0 * a.unit);
  int key_hi = (int)min((int64_t)p.s.len, (int64_t)u1 * a.unit);
  if (!a.has_mask) {  // a chain's rows see no key past their last token
    const int last = (int)divide((uint32_t)min(p.row0 + a.R, p.rows) - 1, a.by_group);
    key_hi = (int)min((int64_t)key_hi, (int64_t)p.s.ctx + last + 1);
  }
  p.key_hi = uniform(key_hi);
  p.tile_end = uniform(before + (int64_t)(tile + 1) * p.s.units);
  p.tile_id = uniform(tiles_before + tile);
  p.whole = uniform(u0 == 0 && u1 == p.s.units);
  p.begins = uniform(u0 == 0);
  return p;
}

// The slots of keys key0 .. + count - 1 of sequence b, -1 for one on no page and for those that fill the
// last tile; returns whether a key is on no page.
__device__ __forceinline__ int find_slots(const TreeArgs& a, int b, int key0, int count, int* slots, int tid, int threads) {
  int lost = 0;
  for (int i = tid; i < (count + 63) / 64 * 64; i += threads) {
    int slot = -1;
    if (i < count) {
      const uint32_t key = (uint32_t)(key0 + i), page = divide(key, a.by_page);
      const int e = a.table[(int64_t)b * a.width + page];
      if (e >= 0 && e < a.pages) slot = (int)((uint32_t)e * a.by_page.d + (key - page * a.by_page.d));
      else lost = 1;
    }
    slots[i] = slot;
  }
  return lost;
}

// This workgroup's share of all `total` units; false: none.  Shares in a row stand on one XCD
// (workgroups go round the 8 XCDs), so that tiles of the same keys meet in its L2.
__device__ __forceinline__ bool my_share(const TreeArgs& a, int lane, int64_t& total, int64_t& me, int64_t& u, int64_t& u_end) {
  total = uniform(total_units(a, lane));
  const int64_t n = shares(a, total);
  me = blockIdx.x;
  if (n == 0 && me == 0 && threadIdx.x == 0) *a.tiles = 0;
  if (me >= n) return false;
  if ((n & 7) == 0) me = (me & 7) * (n >> 3) + (me >> 3);
  u = share_begin(total, n, me);
  u_end = share_begin(total, n, me + 1);
  return true;
}

// Notes the tile of a piece with its first keys.  The last tile's place is the number of tiles, less 1.
// There is room for the tiles of ascending starts; of others, those past it are not joined.
__device__ __forceinline__ void note_tile(const TreeArgs& a, int64_t total, int64_t me, const Piece& p) {
  if (threadIdx.x != 0 || !p.begins) return;
  const int64_t last = share_of(total, shares(a, total), p.tile_end - 1);
  if (p.tile_id < a.room) a.cuts[p.tile_id] = Cut{p.whole ? 0 : (int)(last - me) + 1, (int)me, p.s.q0, p.kvh, p.row0, p.rows, {0, 0}};
  if (p.tile_end == total) *a.tiles = (int)min(p.tile_id + 1, a.room);
}

// ------------------------------------------------------------------------------ waves split the keys
template <int HD, int RT>
struct KeysLds {
  static constexpr int NW = tree_key_waves(HD), R = 16 * RT, Pad = HD + 4;  // Pad: floats of a joining row
  // the waves' stages, later their rows
  static constexpr int Area = std::max(NW * 2 * Cfg<HD, 32>::Stage, NW * R * Pad * 4);
  static constexpr int Slots = HD == 64 ? 2048 : 4096;          // keys whose slots stand in LDS at a time
  static constexpr int Total = Area + Slots * 4 + NW * R * 8;  // slots, (base, sum) of each wave's rows
};

template <int HD, bool BF16, int RT>
__global__ __launch_bounds__(64 * tree_key_waves(HD), HD == 256 ? 1 : 2) void tree_keys_kernel(const TreeArgs a) {
  using C = Cfg<HD, 32>;
  using L = KeysLds<HD, RT>;
  constexpr int R = L::R, NW = L::NW;
  extern __shared__ __align__(16) uint8_t lds[];
  int* slots = (int*)(lds + L::Area);
  float* stat = (float*)(lds + L::Area + L::Slots * 4);
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  int64_t total, me, u, u_end;
  if (!my_share(a, lane, total, me, u, u_end)) return;

  while (u < u_end) {
    const Piece p = next_piece(a, lane, u, u_end);
    note_tile(a, total, me, p);
    const uint16_t* kh = a.k + (int64_t)p.kvh * a.k_h;
    const uint16_t* vh = a.v + (int64_t)p.kvh * a.v_h;
    Rows<HD, RT> w;
    uint8_t* mine = lds + wave * 2 * C::Stage;
    const uint32_t to = lds_address(lds) + wave * 2 * C::Stage;
    for (int again = 0;; again = 1) {
      start_rows<HD, BF16, RT>(a, p.s, p.kvh, p.row0, p.rows, lane, w);
      for (int key0 = p.key_lo; key0 < p.key_hi; key0 += L::Slots) {
        const int count = min(L::Slots, p.key_hi - key0);
        __syncthreads();  // the slots (and the joining rows in the stages) have been read
        const int lost = again | uniform(__syncthreads_or(find_slots(a, p.b, key0, count, slots, tid, 64 * NW)));
        const int tiles = (count + 31) / 32;
        wave_wait<0>();  // from here on the loads in flight are the tiles'
        if (wave < tiles) load_tile<HD, 32, 1>(a, kh, vh, slots, 32 * wave, to, 0, lane);
        // Tiles j = wave, wave + NW, ...; stage of tile j: its turn's parity.
        int j = wave, st = 0;
        auto begin = [&]() {  // the next tile is on its way, this one is here; whether it is an edge tile
          const int first = 32 * j;
          if (j + NW < tiles) {
            load_tile<HD, 32, 1>(a, kh, vh, slots, first + 32 * NW, to + (st ^ 1) * C::Stage, 0, lane);
            wave_wait<2 * C::Loads>();
          } else {
            wave_wait<0>();
          }
          return lost || first + 32 > count || key0 + first - p.s.ctx + 32 > 0;
        };
        auto end = [&]() {
          // every read of this stage has returned before the next load into it
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          j += NW;
          st ^= 1;
        };
        while (j < tiles) {
          bool edge = false;
          for (; j < tiles; end()) {
            edge = begin();
            if (edge || !compute_fast<HD, BF16, RT, 32>(a, mine + st * C::Stage, lane, w)) break;
          }
          if (j >= tiles) break;
          uint8_t* stage = mine + st * C::Stage;
          uint64_t keys = 0, odd = 0;
          if (edge) {
            keys = tile_keys<32>(slots, 32 * j, lane);
            odd = clean_values<HD, BF16, 32, 1>(stage, keys, 0, lane);
            __builtin_amdgcn_wave_barrier();
          }
          compute_slow<HD, BF16, RT, 32>(a, p.s, slots, 32 * j, edge, key0 + 32 * j - p.s.ctx, keys, odd, stage, vh, lane, w);
          end();
        }
      }
      if (again || !__syncthreads_or(!finite(w))) break;
    }

    // the waves' results meet in LDS, in the place of the stages
    __syncthreads();
    float* rowsum = (float*)lds;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float l = w.l[t][0];
      const int row = wave * R + 16 * t + l16;
      if (g == 0) {
        stat[row * 2] = w.m[t];
        stat[row * 2 + 1] = l;
      }
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) *(f32x4_t*)(rowsum + row * L::Pad + 16 * d + 4 * g) = w.o[t][d];
    }
    __syncthreads();
    const int64_t part = 2 * me + (p.begins ? 1 : 0);
    for (int e = tid; e < R * (HD / 8); e += 64 * NW) {
      const int row = e / (HD / 8), c = e % (HD / 8);
      if (p.row0 + row >= p.rows) continue;
      float top = kNone;
#pragma unroll
      for (int i = 0; i < NW; ++i) top = fmaxf(top, stat[(i * R + row) * 2]);
      const float base = top == kNone ? 0.f : top;
      float sum = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const float f = __builtin_amdgcn_exp2f(stat[(i * R + row) * 2] - base);
        sum += f * stat[(i * R + row) * 2 + 1];
        const f32x4_t y0 = *(const f32x4_t*)(rowsum + (i * R + row) * L::Pad + 8 * c);
        const f32x4_t y1 = *(const f32x4_t*)(rowsum + (i * R + row) * L::Pad + 8 * c + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          y[q] += f * y0[q];
          y[4 + q] += f * y1[q];
        }
      }
      if (p.whole) {
        const float inv = inverse(sum);
        const int tk = (int)divide((uint32_t)(p.row0 + row), a.by_group);
        const int head = p.kvh * a.group + p.row0 + row - tk * a.group;
        *(u32x4_t*)(a.out + (int64_t)(p.s.q0 + tk) * a.o_t + (int64_t)head * a.o_h + 8 * c) =
            u32x4_t{pack2<BF16>(y[0] * inv, y[1] * inv), pack2<BF16>(y[2] * inv, y[3] * inv),
                    pack2<BF16>(y[4] * inv, y[5] * inv), pack2<BF16>(y[6] * inv, y[7] * inv)};
      } else {
        float* to = a.part + (part * R + row) * HD + 8 * c;
        *(f32x4_t*)to = f32x4_t{y[0], y[1], y[2], y[3]};
        *(f32x4_t*)(to + 4) = f32x4_t{y[4], y[5], y[6], y[7]};
        if (c == 0) {
          a.part_ml[(part * R + row) * 2] = top;
          a.part_ml[(part * R + row) * 2 + 1] = sum;
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------ waves split the rows
template <int HD, int NW>
struct RowsLds {
  static constexpr int KT = tree_row_keys(NW);
  static constexpr int Area = 2 * Cfg<HD, KT>::Stage;
  static constexpr int Slots = 512 * NW;                   // keys whose slots stand in LDS at a time
  static constexpr int Total = Area + Slots * 4 + NW * 8;  // slots, each wave's odd rows
};

template <int HD, bool BF16, int NW>
__global__ __launch_bounds__(64 * NW, 2) void tree_rows_kernel(const TreeArgs a) {
  constexpr int KT = RowsLds<HD, NW>::KT, RT = 2, R = 32 * NW;
  using C = Cfg<HD, KT>;
  extern __shared__ __align__(16) uint8_t lds[];
  int* slots = (int*)(lds + RowsLds<HD, NW>::Area);
  uint64_t* odd_of = (uint64_t*)(slots + RowsLds<HD, NW>::Slots);
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  int64_t total, me, u, u_end;
  if (!my_share(a, lane, total, me, u, u_end)) return;

  while (u < u_end) {
    const Piece p = next_piece(a, lane, u, u_end);
    note_tile(a, total, me, p);
    const uint16_t* kh = a.k + (int64_t)p.kvh * a.k_h;
    const uint16_t* vh = a.v + (int64_t)p.kvh * a.v_h;
    const int row0 = p.row0 + 16 * RT * wave;
    Rows<HD, RT> w;
    for (int again = 0;; again = 1) {
      start_rows<HD, BF16, RT>(a, p.s, p.kvh, row0, p.rows, lane, w);
      for (int key0 = p.key_lo; key0 < p.key_hi; key0 += RowsLds<HD, NW>::Slots) {
        const int count = min(RowsLds<HD, NW>::Slots, p.key_hi - key0);
        __syncthreads();  // the slots and stages have been read
        const int lost = again | uniform(__syncthreads_or(find_slots(a, p.b, key0, count, slots, tid, 64 * NW)));
        const int tiles = (count + KT - 1) / KT;
        wave_wait<0>();
        const uint32_t to = lds_address(lds);
        load_tile<HD, KT, NW>(a, kh, vh, slots, 0, to, wave, lane);
        int j = 0;
        // The workgroup's waves may leave the inner loop at different tiles: a wave in compute_slow takes
        // part in the barriers of its next tile when it gets there.  Only edge tiles, which are edges for
        // all, hold barriers of their own.
        while (j < tiles) {
          bool edge = false;
          for (; j < tiles; ++j) {
            // this tile has landed for every wave, and every wave has read the one before it
            stage_barrier<0>();
            if (j + 1 < tiles)
              load_tile<HD, KT, NW>(a, kh, vh, slots, KT * (j + 1), to + ((j + 1) & 1) * C::Stage, wave, lane);
            edge = lost || KT * (j + 1) > count || key0 + KT * (j + 1) - p.s.ctx > 0;
            if (edge || !compute_fast<HD, BF16, RT, KT>(a, lds + (j & 1) * C::Stage, lane, w)) break;
          }
          if (j >= tiles) break;
          uint8_t* stage = lds + (j & 1) * C::Stage;
          uint64_t keys = 0, odd = 0;
          if (edge) {
            keys = tile_keys<KT>(slots, KT * j, lane);
            const uint64_t mine = clean_values<HD, BF16, KT, NW>(stage, keys, wave, lane);
            if (lane == 0) odd_of[wave] = mine;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NW; ++i) odd |= odd_of[i];
          }
          compute_slow<HD, BF16, RT, KT>(a, p.s, slots, KT * j, edge, key0 + KT * j - p.s.ctx, keys, odd, stage, vh, lane, w);
          ++j;
        }
      }
      if (again || !__syncthreads_or(!finite(w))) break;
    }

    const int64_t part = 2 * me + (p.begins ? 1 : 0);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = row0 + 16 * t + l16;
      const float l = w.l[t][0];
      if (row >= p.rows) continue;
      if (p.whole) {
        const float inv = inverse(l);
        const int head = p.kvh * a.group + row - w.token[t] * a.group;
        uint16_t* to = a.out + (int64_t)(p.s.q0 + w.token[t]) * a.o_t + (int64_t)head * a.o_h + 4 * g;
#pragma unroll
        for (int d = 0; d < HD / 16; ++d)
          *(u32x2_t*)(to + 16 * d) = u32x2_t{pack2<BF16>(w.o[t][d][0] * inv, w.o[t][d][1] * inv),
                                             pack2<BF16>(w.o[t][d][2] * inv, w.o[t][d][3] * inv)};
      } else {
        const int64_t at = part * R + row - p.row0;
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) *(f32x4_t*)(a.part + at * HD + 16 * d + 4 * g) = w.o[t][d];
        if (g == 0) {
          a.part_ml[at * 2] = w.m[t];
          a.part_ml[at * 2 + 1] = l;
        }
      }
    }
  }
}

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
  const void* kern = nullptr;
  int threads = 64 * pl.waves, lds = 0;
  if (!pl.split_rows) {
    threads = 64 * tree_key_waves(HD);
    if (pl.rows == 16) kern = (const void*)tree_keys_kernel<HD, BF16, 1>, lds = KeysLds<HD, 1>::Total;
    if constexpr (HD != 256)
      if (pl.rows == 32) kern = (const void*)tree_keys_kernel<HD, BF16, 2>, lds = KeysLds<HD, 2>::Total;
  } else if constexpr (HD != 256) {
    if (pl.waves == 2) kern = (const void*)tree_rows_kernel<HD, BF16, 2>, lds = RowsLds<HD, 2>::Total;
    if (pl.waves == 4) kern = (const void*)tree_rows_kernel<HD, BF16, 4>, lds = RowsLds<HD, 4>::Total;
    if (pl.waves == 8) kern = (const void*)tree_rows_kernel<HD, BF16, 8>, lds = RowsLds<HD, 8>::Total;
  }
  if (!kern) return hipErrorInvalidValue;
  hipError_t e = raise_lds_limit(kern, lds);
  if (e != hipSuccess) return e;
  TreeArgs args = a;
  void* argv[1] = {&args};
  e = hipLaunchKernel(kern, dim3((unsigned)a.blocks), dim3((unsigned)threads), argv, (size_t)lds, stream);
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
  a.q = (const uint16_t*)p.q; a.k = (const uint16_t*)p.k; a.v = (const uint16_t*)p.v;
  a.table = p.table; a.context = p.context; a.starts = p.starts; a.mask = p.mask; a.out = (uint16_t*)p.out;
  static_assert(sizeof(Cut) == kTreeCutBytes, "the plan's size of the notes");
  a.tiles = (int32_t*)workspace;
  a.cuts = (Cut*)workspace + 1;
  a.part = (float*)((char*)workspace + pl.notes_bytes);
  a.part_ml = a.part + pl.blocks * 2 * pl.rows * p.d;
  a.R = pl.rows; a.unit = pl.unit;
  a.q_t = p.q_t; a.q_h = p.q_h; a.k_h = p.k_h; a.v_h = p.v_h;
  a.o_t = p.o_t; a.o_h = p.o_h;
  a.k_row = (uint32_t)(2 * p.k_t); a.v_row = (uint32_t)(2 * p.v_t);
  a.pages = p.pages; a.room = pl.tiles; a.N = (int32_t)p.N; a.B = (int32_t)p.B; a.hkv = p.hkv; a.group = p.group;
  a.width = p.width; a.words = p.words; a.has_mask = p.has_mask; a.blocks = (int32_t)pl.blocks;
  a.by_page = fast_div((uint32_t)p.page); a.by_group = fast_div((uint32_t)p.group);
  a.scale = scale == 0.f ? 1.f : std::fabs(scale) * 1.4426950408889634f;
  a.q_and = scale == 0.f ? 0u : ~0u;
  a.q_xor = scale < 0.f ? 0x80008000u : 0u;
  const bool bf16 = p.act == WQ_BF16;
  switch (p.d) {
    case 64: return bf16 ? launch<64, true>(a, pl, stream) : launch<64, false>(a, pl, stream);
    case 128: return bf16 ? launch<128, true>(a, pl, stream) : launch<128, false>(a, pl, stream);
    default: return bf16 ? launch<256, true>(a, pl, stream) : launch<256, false>(a, pl, stream);
  }
}

}  // namespace wq
