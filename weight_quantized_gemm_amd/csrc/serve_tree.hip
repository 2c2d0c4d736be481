// Attention of each sequence's newest tokens (one token, a chain, a tree of drafts) over its
// pages of a key / value cache: out[i] = sum_j softmax_j(scale q_i . k_j) v_j over the keys that
// token i sees.
//
// Work.  The tokens of a sequence and the G query heads of one cached head share that head's
// keys, so they are the rows of one tile: row = token * G + query head, R = 16 * RT rows.  A
// tile's keys are cut into units of 32 keys a wave, and all units of all tiles stand in one
// row (sequence, cached head, tile, key).  Each workgroup takes an equal share of that row,
// wherever it begins and ends: ragged lengths, few long sequences and many short ones load the
// chip alike, without knowing a length on the host.  A tile that one workgroup holds whole is
// written by it; one that is cut leaves partial results (output, maximum, sum) that a second
// kernel joins in key order.  A workgroup has at most two such parts: its first and its last.
//
// One wave's tile is 32 keys.  K and V go straight from memory to the wave's own LDS (16 bytes a
// lane, two stages), so waves wait for nobody and the next tile is always in flight; the rows
// of pages are found through slot numbers that the workgroup writes to LDS ahead, 2048 keys at a
// time.
//
// S^T = K Q^T (keys as MFMA rows, query rows as columns): element i of lane l is key 4 (l / 16) +
// i of row l % 16, so a row's maximum is two cross-lane steps away, its statistics stand in the
// lanes that need them, and the lane's own 8 weights of a 32-key tile are, in this order, the B
// operand of O^T += V^T P^T, if V^T takes the keys in the same order: two transpose reads of 4
// keys each.  The weights never leave the registers.
//
// Scores, maxima, sums and outputs are fp32 (base 2: scale * log2(e) is folded into the scores).
// The weights, at most 1, are rounded to 16 bits for the second product: an error of
// at most 2^-8 (bf16) or 2^-11 (fp16) of each, of the size of the result's own rounding.
#include <algorithm>
#include <cmath>

#include "serve_device.h"
#include "serve_kernels.h"
#include "serve_tile.h"
#include "wq_pipeline.h"

namespace wq {
namespace {

struct TreeArgs {
  const uint16_t *q, *k, *v;
  const int32_t *table, *context, *starts;
  const uint32_t* mask;
  uint16_t* out;
  float* part;        // partial outputs [2 * blocks][R][d]
  float* part_ml;     // their (maximum, sum) [2 * blocks][R][2]
  int64_t q_t, q_h, k_h, v_h, o_t, o_h;
  uint32_t k_row, v_row;  // bytes from one slot to the next
  int64_t pages;
  int32_t N, B, hq, hkv, group, width, words, has_mask;
  int32_t blocks;     // workgroups of the launch
  FastDiv by_page, by_group;
  // The scores' factor, |scale| * log2(e), is positive, so that it neither turns the order of the
  // scores nor moves -inf; a negative scale flips the queries' signs, a zero one clears them.
  float scale;
  uint32_t q_and, q_xor;
};

constexpr int kSlots = 2048;  // keys whose slots stand in LDS at a time
constexpr float kNone = -__builtin_inff();

// ------------------------------------------------------------------------------ the schedule
struct Seq {
  int q0 = 0, tokens = 0, ctx = 0, len = 0;  // first query row, tokens, context, visible cache length
  int tiles = 0, units = 0;                  // row tiles of a cached head, units of a tile
};

template <int R, int UNIT>
__device__ __forceinline__ Seq sequence(const TreeArgs& a, int b) {
  Seq s;
  s.q0 = min(max(a.starts[b], 0), a.N);
  s.tokens = min(max(a.starts[b + 1], s.q0), a.N) - s.q0;
  s.ctx = max(a.context[b], 0);
  const int64_t len = (int64_t)s.ctx + s.tokens, most = a.pages ? (int64_t)a.width * a.by_page.d : 0;
  s.len = (int)min(len, most);
  s.tiles = (int)(((int64_t)s.tokens * a.group + R - 1) / R);
  s.units = max(1, (s.len + UNIT - 1) / UNIT);  // a tile without keys still writes zeros
  return s;
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <int R, int UNIT>
__device__ __forceinline__ int64_t total_units(const TreeArgs& a, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < a.B; b += 64) {
    const Seq s = sequence<R, UNIT>(a, b);
    sum += (int64_t)s.tiles * s.units * a.hkv;
  }
  return wave_sum(sum);
}

// The sequence that holds unit u (u < total), and the number of units before it.
template <int R, int UNIT>
__device__ __forceinline__ int find_sequence(const TreeArgs& a, int lane, int64_t u, int64_t& before) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int64_t own = 0;
    if (b0 + lane < a.B) {
      const Seq s = sequence<R, UNIT>(a, b0 + lane);
      own = (int64_t)s.tiles * s.units * a.hkv;
    }
    int64_t upto = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t t = __shfl_up(upto, o, 64);
      if (lane >= o) upto += t;
    }
    const uint64_t past = __ballot(base + upto > u);
    if (past) {
      const int at = __builtin_ctzll(past);
      before = base + __shfl(upto - own, at, 64);
      return b0 + at;
    }
    base += __shfl(upto, 63, 64);
  }
  before = base;
  return -1;
}

// Workgroups that share `total` units, and the first unit of share i.
__device__ __forceinline__ int64_t shares(const TreeArgs& a, int64_t total) { return min((int64_t)a.blocks, total); }
__device__ __forceinline__ int64_t share_begin(int64_t total, int64_t n, int64_t i) { return total * i / n; }
// The share that holds unit u: the largest i with total * i / n <= u.
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t n, int64_t u) { return ((u + 1) * n - 1) / total; }

// ------------------------------------------------------------------------------ one wave's tile
template <int HD>
struct Cfg {
  static constexpr int NW = tree_waves(HD), UNIT = tree_unit(HD), CH = HD / 8, RB = HD * 2;
  static constexpr int Half = kTreeKeys * RB, Stage = 2 * Half;  // K, then V
  static constexpr int Loads = Half / 1024;                      // per tensor and tile, 1 KB each
  static constexpr int Pad = HD + 4;                             // floats of a merge row
};

// 16-byte chunk c of K row r stands in slot row_slot (16-byte reads of 16 rows at one chunk hit all
// banks); the 32-byte pair p of V row r in pair_slot (a transpose read takes 32 bytes of 8 rows).
// Rows of 512 bytes start in the same bank as rows of 256, so they take the latter's pattern.
template <int HD> __device__ __forceinline__ int k_chunk(int r, int c) {
  if constexpr (HD == 256) return c ^ (r & 15);
  else return row_slot<HD * 2>(r, c);
}
template <int HD> __device__ __forceinline__ int v_chunk(int r, int c) {
  if constexpr (HD == 256) return c ^ (2 * (r & 7));
  else return 2 * pair_slot<HD * 2>(r, c >> 1) + (c & 1);
}

template <int HD>
__device__ __forceinline__ void load_tile(const TreeArgs& a, const uint16_t* kh, const uint16_t* vh, const int* slots,
                                          int first, int count, uint8_t* stage, int lane) {
  using C = Cfg<HD>;
  asm volatile("" : "+v"(lane));  // addresses are made anew for each tile: kept, they would take 100 registers
#pragma unroll
  for (int i = 0; i < C::Loads; ++i) {
    const int e = i * 64 + lane, row = e / C::CH, c = e % C::CH;
    const uint32_t slot = (uint32_t)max(slots[min(first + row, count - 1)], 0);  // no such key: any row of the cache
    dma16_global((const uint8_t*)kh + (uint64_t)slot * a.k_row + 16 * k_chunk<HD>(row, c), stage + 1024 * i);
  }
#pragma unroll
  for (int i = 0; i < C::Loads; ++i) {
    const int e = i * 64 + lane, row = e / C::CH, c = e % C::CH;
    const uint32_t slot = (uint32_t)max(slots[min(first + row, count - 1)], 0);
    dma16_global((const uint8_t*)vh + (uint64_t)slot * a.v_row + 16 * v_chunk<HD>(row, c), stage + C::Half + 1024 * i);
  }
}

template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t half) {
  const uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  return (half & e) == e;
}

// Which of the 32 keys from drafted token draft0 on (negative: the context's end) a token sees,
// as far as the mask goes: 32 bits of its row of the mask, which two words hold.
__device__ __forceinline__ uint32_t tile_bits(const TreeArgs& a, const Seq& s, int token, int draft0) {
  if (draft0 <= -kTreeKeys) return ~0u;
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

// One 32-key tile (keys key0 + 0 .. 31, of which those at or past key_end do not belong to this
// piece of work) for RT 16-row blocks.  EDGE tiles hold keys that some row does not see: past the end, on no
// page, or drafted tokens.  There the scores of unseen keys become -inf, and V loses, for the
// matrix product, its rows without a key and its infinities and NaN (0 * inf would reach rows
// that do not see them); what those contribute to rows that do see them is added afterwards.
template <int HD, bool BF16, int RT, bool EDGE>
__device__ __forceinline__ void compute_tile(const TreeArgs& a, const Seq& s, const int* slots, int first, int key0,
                                             int key_end, uint8_t* stage, const uint16_t* vh, int lane,
                                             const u32x4_t (&qf)[RT][HD / 32], const int (&token)[RT],
                                             f32x4_t (&o)[RT][HD / 16], float (&m)[RT], float (&l)[RT]) {
  using C = Cfg<HD>;
  asm volatile("" : "+v"(lane));  // as in load_tile
  const int l16 = lane & 15, g = lane >> 4;
  f32x4_t sc[RT][2];
#pragma unroll
  for (int t = 0; t < RT; ++t) sc[t][0] = sc[t][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < HD / 32; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 16 * h + l16;
      const u32x4_t kf = *(const u32x4_t*)(stage + row * C::RB + 16 * k_chunk<HD>(row, 4 * j + g));
#pragma unroll
      for (int t = 0; t < RT; ++t) sc[t][h] = mfma16x16x32<BF16>(kf, qf[t][j], sc[t][h]);
    }

  uint32_t seen[RT];      // EDGE: bit r, whether this lane's row sees key r of the tile
  uint32_t odd_rows = 0;  // EDGE: keys whose V holds an infinity or NaN
  if constexpr (EDGE) {
    const bool is_key = lane < kTreeKeys && key0 + lane < key_end && slots[min(first + lane, kSlots - 1)] >= 0;
    const uint32_t keys = (uint32_t)__ballot(is_key);
    const int draft0 = key0 - s.ctx;  // the drafted token of the tile's first key, negative in the context
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      seen[t] = keys & tile_bits(a, s, token[t], draft0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((seen[t] >> (16 * h + 4 * g + i)) & 1)) sc[t][h][i] = kNone;
    }
#pragma unroll 1
    for (int e = lane; e < kTreeKeys * C::CH; e += 64) {
      const int row = e / C::CH;
      u32x4_t* at = (u32x4_t*)(stage + C::Half + 16 * e);
      u32x4_t x = *at;
      bool change = !((keys >> row) & 1);
      if (change) x = u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const bool lo = not_finite<BF16>(x[d]), hi = not_finite<BF16>(x[d] >> 16);
        if (lo || hi) {
          odd_rows |= 1u << row;
          change = true;
          x[d] &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
        }
      }
      if (change) *at = x;
    }
#pragma unroll
    for (int w = 1; w < 64; w <<= 1) odd_rows |= (uint32_t)__shfl_xor((int)odd_rows, w, 64);
    __builtin_amdgcn_wave_barrier();
  }

  u32x4_t pf[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    float top = fmaxf(fmaxf(fmaxf(sc[t][0][0], sc[t][0][1]), fmaxf(sc[t][0][2], sc[t][0][3])),
                      fmaxf(fmaxf(sc[t][1][0], sc[t][1][1]), fmaxf(sc[t][1][2], sc[t][1][3])));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float now = fmaxf(m[t], top * a.scale);
    const float base = now == kNone ? 0.f : now;  // no key seen so far: every weight is 0
    const float keep = __builtin_amdgcn_exp2f(m[t] - base);
    m[t] = now;
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f(fmaf(sc[t][h][i], a.scale, -base));
        sc[t][h][i] = p;
        sum += p;
      }
    l[t] = l[t] * keep + sum;
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) o[t][d] *= keep;
    pf[t] = u32x4_t{pack2<BF16>(sc[t][0][0], sc[t][0][1]), pack2<BF16>(sc[t][0][2], sc[t][0][3]),
                    pack2<BF16>(sc[t][1][0], sc[t][1][1]), pack2<BF16>(sc[t][1][2], sc[t][1][3])};
  }

  // V^T: column 16 d + l16, keys 4 g .. + 3 and 16 + 4 g .. + 3
  const uint8_t* vs = stage + C::Half;
  const int vrow = 4 * g + (l16 >> 2), vhalf = 8 * (l16 & 1);
#pragma unroll
  for (int d = 0; d < HD / 16; ++d) {
    const int c = 2 * d + ((l16 & 3) >> 1);
    const u32x2_t v0 = lds_read_tr16(vs + vrow * C::RB + 16 * v_chunk<HD>(vrow, c) + vhalf);
    const u32x2_t v1 = lds_read_tr16(vs + (vrow + 16) * C::RB + 16 * v_chunk<HD>(vrow + 16, c) + vhalf);
    const u32x4_t vf = u32x4_t{v0[0], v0[1], v1[0], v1[1]};
#pragma unroll
    for (int t = 0; t < RT; ++t) o[t][d] = mfma16x16x32<BF16>(vf, pf[t], o[t][d]);
  }

  if constexpr (EDGE) {
    while (odd_rows) {
      const int r = __builtin_ctz(odd_rows);
      odd_rows &= odd_rows - 1;
      const uint16_t* vr = (const uint16_t*)((const uint8_t*)vh + (uint64_t)(uint32_t)slots[first + r] * a.v_row) + 4 * g;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float p = 0.f;  // the row's weight of key r, from the lane that has it
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((r >> 4) == h && (r & 3) == i) p = sc[t][h][i];
        p = __shfl(p, l16 + 16 * ((r >> 2) & 3), 64);
        const bool sees = (seen[t] >> r) & 1;
#pragma unroll
        for (int d = 0; d < HD / 16; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            asm volatile("" ::: "memory");  // one element at a time: this path is rare, registers are not plenty
            const uint16_t x = vr[16 * d + i];
            if (not_finite<BF16>(x) && sees) o[t][d][i] += p * act_to_f32<BF16>(x);
          }
      }
    }
  }
}

// ------------------------------------------------------------------------------ the kernel
template <int HD, bool BF16, int RT>
__global__ __launch_bounds__(64 * tree_waves(HD), RT == 4 || HD == 256 ? 1 : 2) void tree_kernel(const TreeArgs a) {
  using C = Cfg<HD>;
  constexpr int R = 16 * RT, NW = C::NW, UNIT = C::UNIT;
  extern __shared__ __align__(16) uint8_t lds[];
  // stages of the waves (and after them the merge's rows), slots, row statistics of the waves
  constexpr int kArea = std::max(NW * 2 * C::Stage, NW * R * C::Pad * 4);
  int* slots = (int*)(lds + kArea);
  float* stat = (float*)(lds + kArea + kSlots * 4);  // [NW][R][2]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, g = lane >> 4;

  const int64_t total = total_units<R, UNIT>(a, lane);
  if (total == 0) return;
  const int64_t n = shares(a, total);
  // shares in a row on one XCD (workgroups go round the 8 XCDs): tiles of the same keys meet in its L2
  int64_t me = blockIdx.x;
  if (me >= n) return;
  if ((n & 7) == 0) me = (me & 7) * (n >> 3) + (me >> 3);
  int64_t u = share_begin(total, n, me);
  const int64_t u_end = share_begin(total, n, me + 1);

  while (u < u_end) {
    int64_t before;
    const int b = find_sequence<R, UNIT>(a, lane, u, before);
    const Seq s = sequence<R, UNIT>(a, b);
    const int64_t in = u - before;
    const int tile = (int)(in / s.units), u0 = (int)(in - (int64_t)tile * s.units);
    const int u1 = (int)min((int64_t)s.units, u0 + (u_end - u));
    u += u1 - u0;
    const int kvh = tile / s.tiles, row0 = (tile - kvh * s.tiles) * R, rows = s.tokens * a.group;

    // this lane's row of each 16-row block, its token, and its query
    int token[RT];
    u32x4_t qf[RT][HD / 32];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = min(row0 + 16 * t + l16, rows - 1);
      token[t] = (int)divide((uint32_t)row, a.by_group);
      const int head = kvh * a.group + row - token[t] * a.group;
      const uint16_t* qr = a.q + (int64_t)(s.q0 + token[t]) * a.q_t + (int64_t)head * a.q_h + 8 * g;
#pragma unroll
      for (int j = 0; j < HD / 32; ++j) qf[t][j] = (*(const u32x4_t*)(qr + 32 * j) & a.q_and) ^ a.q_xor;
    }
    const int key_lo = u0 * UNIT;
    int key_hi = min(s.len, u1 * UNIT);
    if (!a.has_mask) {  // a chain's rows see no key past their last token
      const int last = (int)divide((uint32_t)min(row0 + R, rows) - 1, a.by_group);
      key_hi = (int)min((int64_t)key_hi, (int64_t)s.ctx + last + 1);
    }
    const uint16_t* kh = a.k + (int64_t)kvh * a.k_h;
    const uint16_t* vh = a.v + (int64_t)kvh * a.v_h;

    f32x4_t o[RT][HD / 16];
    float m[RT], l[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = kNone;
      l[t] = 0.f;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) o[t][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    uint8_t* mine = lds + wave * 2 * C::Stage;
    for (int key0 = key_lo; key0 < key_hi; key0 += kSlots) {
      const int count = min(kSlots, key_hi - key0);
      int lost = 0;
      __syncthreads();  // the slots (and the merge rows in the stages) have been read
      for (int i = tid; i < count; i += 64 * NW) {
        const uint32_t key = (uint32_t)(key0 + i), page = divide(key, a.by_page);
        const int e = a.table[(int64_t)b * a.width + page];
        const bool ok = e >= 0 && e < a.pages;
        slots[i] = ok ? (int)((uint32_t)e * a.by_page.d + (key - page * a.by_page.d)) : -1;
        lost |= !ok;
      }
      lost = __syncthreads_or(lost);

      const int tiles = (count + kTreeKeys - 1) / kTreeKeys;
      // everything this wave's loads below are counted against is then theirs alone
      wave_wait<0>();
      if (wave < tiles) load_tile<HD>(a, kh, vh, slots, wave * kTreeKeys, count, mine, lane);
      int st = 0;
      for (int j = wave; j < tiles; j += NW, st ^= 1) {
        const int first = j * kTreeKeys;
        if (j + NW < tiles) {
          load_tile<HD>(a, kh, vh, slots, first + NW * kTreeKeys, count, mine + (st ^ 1) * C::Stage, lane);
          wave_wait<2 * C::Loads>();
        } else {
          wave_wait<0>();
        }
        uint8_t* stage = mine + st * C::Stage;
        if (lost || first + kTreeKeys > count || key0 + first + kTreeKeys > s.ctx)
          compute_tile<HD, BF16, RT, true>(a, s, slots, first, key0 + first, key0 + count, stage, vh, lane, qf, token, o,
                                           m, l);
        else
          compute_tile<HD, BF16, RT, false>(a, s, slots, first, key0 + first, key0 + count, stage, vh, lane, qf, token,
                                            o, m, l);
        // every read of this stage has returned before the next load into it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
    }

    // the waves' results meet in LDS, in the place of the stages
    __syncthreads();
    float* rowsum = (float*)lds;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      l[t] += __shfl_xor(l[t], 16, 64);
      l[t] += __shfl_xor(l[t], 32, 64);
      const int row = 16 * t + l16;
      if (g == 0) {
        stat[(wave * R + row) * 2] = m[t];
        stat[(wave * R + row) * 2 + 1] = l[t];
      }
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) *(f32x4_t*)(rowsum + (wave * R + row) * C::Pad + 16 * d + 4 * g) = o[t][d];
    }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == s.units;
    const int64_t part = 2 * me + (u0 == 0 ? 1 : 0);
    for (int e = tid; e < R * (HD / 8); e += 64 * NW) {
      const int row = e / (HD / 8), c = e % (HD / 8);
      if (row0 + row >= rows) continue;
      float top = kNone;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, stat[(w * R + row) * 2]);
      const float base = top == kNone ? 0.f : top;
      float sum = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = __builtin_amdgcn_exp2f(stat[(w * R + row) * 2] - base);
        sum += f * stat[(w * R + row) * 2 + 1];
        const f32x4_t y0 = *(const f32x4_t*)(rowsum + (w * R + row) * C::Pad + 8 * c);
        const f32x4_t y1 = *(const f32x4_t*)(rowsum + (w * R + row) * C::Pad + 8 * c + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] += f * y0[i];
          y[4 + i] += f * y1[i];
        }
      }
      if (whole) {
        const float inv = sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f;
        const int tk = (int)divide((uint32_t)(row0 + row), a.by_group);
        const int head = kvh * a.group + row0 + row - tk * a.group;
        *(u32x4_t*)(a.out + (int64_t)(s.q0 + tk) * a.o_t + (int64_t)head * a.o_h + 8 * c) =
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

// ------------------------------------------------------------------------------ the join
// One wave per query row and head: the parts of its tile, in key order.  HD / 64 elements a lane.
template <int HD, bool BF16, int R>
__global__ __launch_bounds__(256) void tree_join_kernel(const TreeArgs a) {
  constexpr int UNIT = tree_unit(HD), E = HD / 64;
  const int lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t total = total_units<R, UNIT>(a, lane);
  if (total == 0 || id >= (int64_t)a.N * a.hq) return;
  const int64_t n = shares(a, total);
  const int tok = (int)(id / a.hq), head = (int)(id - (int64_t)tok * a.hq);

  // the sequence of the token: the first whose query rows end past it, and the units before it
  int b = -1;
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int64_t own = 0;
    bool has = false;
    if (b0 + lane < a.B) {
      const Seq s = sequence<R, UNIT>(a, b0 + lane);
      own = (int64_t)s.tiles * s.units * a.hkv;
      has = tok >= s.q0 && tok < s.q0 + s.tokens;
    }
    const uint64_t at = __ballot(has);
    if (at) {
      b = b0 + __builtin_ctzll(at);
      before += wave_sum(b0 + lane < b ? own : 0);
      break;
    }
    before += wave_sum(own);
  }
  if (b < 0) return;
  const Seq s = sequence<R, UNIT>(a, b);
  const int kvh = head / a.group, row = (tok - s.q0) * a.group + head - kvh * a.group;
  const int64_t u0 = before + ((int64_t)kvh * s.tiles + row / R) * s.units;
  const int64_t i0 = share_of(total, n, u0), i1 = share_of(total, n, u0 + s.units - 1);
  if (i0 == i1) return;  // one workgroup held the tile and wrote it
  float top = kNone, sum = 0.f, y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  for (int64_t i = i0; i <= i1; ++i) {
    const int64_t at = (2 * i + (i == i0 ? 1 : 0)) * R + row % R;
    const float pm = a.part_ml[at * 2], pl = a.part_ml[at * 2 + 1];
    const float now = fmaxf(top, pm), base = now == kNone ? 0.f : now;
    const float f0 = __builtin_amdgcn_exp2f(top - base), f1 = __builtin_amdgcn_exp2f(pm - base);
    sum = sum * f0 + pl * f1;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = y[e] * f0 + a.part[at * HD + lane * E + e] * f1;
    top = now;
  }
  const float inv = sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f;
  uint16_t* to = a.out + (int64_t)tok * a.o_t + (int64_t)head * a.o_h + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) to[e] = f32_to_act<BF16>(y[e] * inv);
}

template <int HD, bool BF16, int RT>
hipError_t launch(const TreeArgs& a, hipStream_t stream) {
  using C = Cfg<HD>;
  constexpr int R = 16 * RT;
  constexpr int lds = std::max(C::NW * 2 * C::Stage, C::NW * R * C::Pad * 4) + kSlots * 4 + C::NW * R * 8;
  auto kern = tree_kernel<HD, BF16, RT>;
  hipError_t e = raise_lds_limit((const void*)kern, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)a.blocks), dim3(64 * C::NW), lds, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t waves = (int64_t)a.N * a.hq;
  hipLaunchKernelGGL((tree_join_kernel<HD, BF16, R>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <int HD, bool BF16>
hipError_t launch_rows(const TreeArgs& a, int row_blocks, hipStream_t stream) {
  if (row_blocks == 1) return launch<HD, BF16, 1>(a, stream);
  if constexpr (HD != 256) {
    if (row_blocks == 2) return launch<HD, BF16, 2>(a, stream);
    if (row_blocks == 4) return launch<HD, BF16, 4>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_tree(const TreeProblem& p, const TreePlan& pl, float scale, void* workspace, hipStream_t stream) {
  TreeArgs a{};
  a.q = (const uint16_t*)p.q; a.k = (const uint16_t*)p.k; a.v = (const uint16_t*)p.v;
  a.table = p.table; a.context = p.context; a.starts = p.starts; a.mask = p.mask; a.out = (uint16_t*)p.out;
  a.part = (float*)workspace;
  a.part_ml = a.part + pl.blocks * 2 * 16 * pl.row_blocks * p.d;
  a.q_t = p.q_t; a.q_h = p.q_h; a.k_h = p.k_h; a.v_h = p.v_h;
  a.o_t = p.o_t; a.o_h = p.o_h;
  a.k_row = (uint32_t)(2 * p.k_t); a.v_row = (uint32_t)(2 * p.v_t);
  a.pages = p.pages; a.N = (int32_t)p.N; a.B = (int32_t)p.B; a.hq = p.hq; a.hkv = p.hkv; a.group = p.group;
  a.width = p.width; a.words = p.words; a.has_mask = p.has_mask; a.blocks = (int32_t)pl.blocks;
  a.by_page = fast_div((uint32_t)p.page); a.by_group = fast_div((uint32_t)p.group);
  a.scale = scale == 0.f ? 1.f : std::fabs(scale) * 1.4426950408889634f;
  a.q_and = scale == 0.f ? 0u : ~0u;
  a.q_xor = scale < 0.f ? 0x80008000u : 0u;
  const bool bf16 = p.act == WQ_BF16;
  switch (p.d) {
    case 64: return bf16 ? launch_rows<64, true>(a, pl.row_blocks, stream) : launch_rows<64, false>(a, pl.row_blocks, stream);
    case 128: return bf16 ? launch_rows<128, true>(a, pl.row_blocks, stream) : launch_rows<128, false>(a, pl.row_blocks, stream);
    default: return bf16 ? launch_rows<256, true>(a, pl.row_blocks, stream) : launch_rows<256, false>(a, pl.row_blocks, stream);
  }
}

}  // namespace wq
