// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// The tests of a request's tokens need one probability of the target's and one of the draft's each, whatever
// the vocabulary's size; only the row of the last accepted token is read whole, for what is left of it
// after the refused children, r(x) = max(p(x) - q(x), 0) or p(x) without the refused tokens, and the first x
// whose running sum passes u times the whole.
//
//   sums: each workgroup has a chunk of a request's row.  It walks through the tests itself (the wave's lanes hold
//     the tokens, so that a step is a ballot), which takes less than a launch of its own, and its waves sum
//     r over units of 512 elements in a row (more where a row would have over 1024 units).
//   pick: a workgroup for each request finds the unit that the random share falls into, and a wave the
//     token in it.  Where nothing is left of r it sums the units of p first.
//
// Where drafts of a tree have probabilities, the second child of a token is tested against what the first left,
// divided by its sum: a row to be summed in the middle of the walk.  There a workgroup for each request walks
// first (walk), and the sums take up what it found.  What c refusals leave has a closed form: with
//
//   C_0 = 0, T_0 = 1,  C_(i+1) = C_i + T_i,  T_i = sum_x max(p(x) - C_i q(x), 0),
//
// r_c = max(p - C_c q, 0) / T_c, since max(max(p - C q, 0) / T - q, 0) = max(p - (C + T) q, 0) / T.  An element
// takes one multiply-add however many children were refused, and a refusal with a further child one pass over the
// two rows, by the one workgroup of its request; the child x is accepted if u q(x) T_c < max(p(x) - C_c q(x), 0).
// (1023 refusals over 65536 tokens: 6.6 ms, 6.5 us each; a request's row is not shared among workgroups.)
//
// Everything that is compared or summed is fp64, in an order that depends on sizes alone: equal calls give
// equal tokens.  With e = 2^-53 a running sum goes through at most unit / 64 + unit / 512 + 46 additions (in a lane, across
// lanes, units and waves, and again inside the unit that is found), its share of the whole through unit / 64 + 21, and the numbers that are
// summed are off by e each: a token differs from the exact one where the random number is within 2^-46 of a border of the
// running sums, as a share of the whole (V up to 2^19, unit = 512; 2^-43 at V = 2^24).  In fp32 one call in a hundred
// would be so near one of V borders.  After two or more refusals C is a sum too: T_i goes through V / 1024 + 23
// additions, an error of C moves the later T the other way by no more than itself, and so what c refusals leave is off by
// (V / 1024 + 24 + c) e C / T of itself, which is more where the refusals left little.
//
// Bound by two launches and the chain request -> tests -> row -> sums -> unit -> token.  Measured (kernel trace): a chain of
// 5 over 32000 tokens 3.7 + 4.0 us; 16 trees of 24 4.9 + 5.4; 64 chains of 9 with draft's probabilities, 67 MB read, 12.9
// (5.2 TB/s, within the 256 MB cache) + 7.2.  With running sums of single tokens by the whole workgroup in place of units of
// 512 the pick took 13 to 15 us.  Trees of 24 with draft's probabilities, by three launches: one request over 32000
// 5.5 + 3.1 + 3.7, 16 over 131072 28.5 (the walk, a workgroup each) + 4.8 + 6.8.
#include <algorithm>

#include "serve_device.h"
#include "serve_step_kernels.h"
#include "serve_tile.h"

namespace wq {
namespace {

constexpr int kThreads = 256;       // of the sums and the pick
constexpr int kWide = 1024;         // of the walk of its own
constexpr int kMaxTokens = kVerifyTokens;

struct State {
  int32_t row;      // of the last accepted token; -1: a request without tokens
  int32_t refused;  // children refused since
  double taken;     // with draft: how many times its row has been taken off, C above
};
static_assert(sizeof(State) == kVerifyStateBytes, "the plan's size of a state");

struct VerifyArgs {
  const void *target, *draft;
  const int32_t *tokens, *parents, *starts;
  const float *accept, *sample;
  int32_t *accepted, *counts, *next;
  State* state;
  double* sums;      // of each request's units
  int32_t* refused;  // without draft: the refused tokens of a request, from its first row on
  int64_t t_row, d_row;
  int32_t N, V, depth, unit, units, chunk;
};

enum Kind { kF32, kF16, kBf16 };

template <int KIND>
__device__ __forceinline__ float value(const void* base, int64_t i) {
  if constexpr (KIND == kF32) return ((const float*)base)[i];
  else return act_to_f32<KIND == kBf16>(((const uint16_t*)base)[i]);
}
// A probability: negative numbers and NaN are 0.
__device__ __forceinline__ double prob(float v) { return (double)fmaxf(v, 0.f); }

// What another lane of the wave has, by a data-parallel move (0 where there is none).
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  const i32x2_t x = __builtin_bit_cast(i32x2_t, v);
  return __builtin_bit_cast(double, i32x2_t{__builtin_amdgcn_update_dpp(0, x[0], CTRL, ROWS, 0xf, false),
                                            __builtin_amdgcn_update_dpp(0, x[1], CTRL, ROWS, 0xf, false)});
}
// The sum of lanes 0 .. this one: within rows of 16, then from row to row.
__device__ __forceinline__ double wave_upto(double v) {
  v += moved<0x111, 0xf>(v);
  v += moved<0x112, 0xf>(v);
  v += moved<0x114, 0xf>(v);
  v += moved<0x118, 0xf>(v);
  v += moved<0x142, 0xa>(v);         // lane 15 of rows 0 and 2 to rows 1 and 3
  return v + moved<0x143, 0xc>(v);   // lane 31 to rows 2 and 3
}
__device__ __forceinline__ double lane_before(double v) { return moved<0x138, 0xf>(v); }
__device__ __forceinline__ double lane_of(double v, int lane) {
  const i32x2_t x = __builtin_bit_cast(i32x2_t, v);
  return __builtin_bit_cast(double, i32x2_t{__builtin_amdgcn_readlane(x[0], lane), __builtin_amdgcn_readlane(x[1], lane)});
}
__device__ __forceinline__ double wave_total(double v) { return lane_of(wave_upto(v), 63); }

struct Rows {
  int q0 = 0, n = 0;  // first row, tokens looked at
};
__device__ __forceinline__ Rows request(const VerifyArgs& a, int b) {
  Rows r;
  r.q0 = min(max(a.starts[b], 0), a.N);
  r.n = min(min(max(a.starts[b + 1], r.q0), a.N) - r.q0, kMaxTokens);
  return r;
}

// What a walk leaves in LDS.
struct Walk {
  int row, refused, depth;
  int path[kMaxTokens];       // the accepted tokens
  int token[kMaxTokens];      // the refused ones (without draft)
  double taken;               // State's (with draft)
};

// What is left of a probability p at a token that the draft gives q, times T: r_c T_c above.
__device__ __forceinline__ double left_of(double p, double q, double taken) { return fmax(fma(-taken, q, p), 0.0); }

// The tests of a request's tokens by one wave: of a chain, or of a tree without draft.
template <int KIND>
__device__ void walk_tests(const VerifyArgs& a, const Rows& r, int lane, Walk& w) {
  int cur = 0, depth = 0, refused = 0;
  double lost = 0.0;
  for (int base = 0; base < r.n && depth < a.depth; base += 64) {
    // this lane's token: its parent and the two probabilities after that
    const int j = base + lane;
    int parent = -1, token = -1;
    float u = 0.f;
    double p = 0.0, q = 0.0;
    if (j > 0 && j < r.n) {
      parent = a.parents ? a.parents[r.q0 + j] : j - 1;
      token = a.tokens[r.q0 + j];
      u = a.accept[r.q0 + j];
      if (parent < 0 || parent >= j) parent = -1;
      if (parent >= 0 && token >= 0 && token < a.V) {
        p = prob(value<KIND>(a.target, (int64_t)(r.q0 + parent) * a.t_row + token));
        if (a.draft) q = prob(value<KIND>(a.draft, (int64_t)(r.q0 + parent) * a.d_row + token));
      }
    }
    int from = base;  // tokens before it have been tested or passed
    while (depth < a.depth) {
      const uint64_t next = __ballot(parent == cur && j >= from);
      if (!next) break;
      const int at = __builtin_ctzll(next);
      from = base + at + 1;
      const int x = __builtin_amdgcn_readlane(token, at);
      const double ux = (double)__int_as_float(__builtin_amdgcn_readlane(__float_as_int(u), at)), qx = lane_of(q, at);
      double px = lane_of(p, at);
      if (!a.draft) {  // a sibling of the same token that was refused has taken it all
        bool same = false;
        for (int i = lane; i < refused; i += 64) same |= w.token[i] == x;
        if (__ballot(same)) px = 0.0;
      }
      if (ux * (a.draft ? qx : 1.0 - lost) < px) {
        cur = base + at;
        if (lane == 0) w.path[depth] = cur;
        ++depth;
        refused = 0;
        lost = 0.0;
      } else {
        if (lane == 0) w.token[refused] = x;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
        ++refused;
        lost += px;
      }
    }
  }
  if (lane == 0) {
    w.row = r.n > 0 ? r.q0 + cur : -1;
    w.refused = refused;
    w.taken = refused > 0 ? 1.0 : 0.0;  // a token of a chain has one child
    w.depth = depth;
  }
}

// 16-byte loads from any element on: rows start wherever the vocabulary's size puts them.
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

// Eight probabilities from element v of a row on, 0 past its end.
template <int KIND>
__device__ __forceinline__ void load8(const void* base, int64_t row, int v, int end, float* f) {
  if (v + 8 <= end) {
    if constexpr (KIND == kF32) {
      const f32x4_any_t lo = *(const f32x4_any_t*)((const float*)base + row + v);
      const f32x4_any_t hi = *(const f32x4_any_t*)((const float*)base + row + v + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = lo[i], f[4 + i] = hi[i];
    } else {
      const u32x4_any_t x = *(const u32x4_any_t*)((const uint16_t*)base + row + v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = act_to_f32<KIND == kBf16>((uint16_t)x[i]);
        f[2 * i + 1] = act_to_f32<KIND == kBf16>((uint16_t)(x[i] >> 16));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = v + i < end ? value<KIND>(base, row + v + i) : 0.f;
}

// What is left of a row at the 8 elements from v on; list: the refused tokens (without draft) of this chunk.
struct Left {
  const int* list = nullptr;
  int refused = 0, listed = 0;
  double taken = 0.0;
};

// draft: whether refusals have taken the draft's row off, which qf holds.
__device__ __forceinline__ void left8(const float* pf, const float* qf, bool draft, const Left& l, int v, double* r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = prob(pf[i]);
  if (draft) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = left_of(r[i], prob(qf[i]), l.taken);
  } else {
    for (int k = 0; k < l.listed; ++k) {
      const uint32_t in = (uint32_t)(l.list[k] - v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in == (uint32_t)i) r[i] = 0.0;
    }
  }
}

// The sum of what is left over a unit, by a wave.
template <int KIND, bool DRAFT>
__device__ __forceinline__ double unit_sum(const VerifyArgs& a, int64_t at_t, int64_t at_d, const Left& l, int u, int lane) {
  const int lo = u * a.unit, hi = (int)min((int64_t)lo + a.unit, (int64_t)a.V);
  const bool draft = DRAFT && l.refused > 0;  // without a refusal p is all that is read
  double sum = 0.0;
  for (int v = lo + 8 * lane; v < hi; v += kVerifyStep) {
    float pf[8], qf[8];
    double x[8];
    load8<KIND>(a.target, at_t, v, hi, pf);
    if (draft) load8<KIND>(a.draft, at_d, v, hi, qf);
    left8(pf, qf, draft, l, v, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += x[i];
  }
  return wave_total(sum);
}

// The refused tokens of elements [lo, hi) among `count`, into LDS by all threads.
__device__ __forceinline__ void pick_listed(const int* tokens, int count, int lo, int hi, int* list, int* listed, int tid,
                                            int threads) {
  for (int i = tid; i < count; i += threads)
    if (tokens[i] >= lo && tokens[i] < hi) list[atomicAdd(listed, 1)] = tokens[i];
}

// ------------------------------------------------------------------------------ trees whose drafts have probabilities
template <int KIND>
__global__ __launch_bounds__(kWide) void verify_walk_kernel(const VerifyArgs a) {
  __shared__ int parents[kMaxTokens], path[kMaxTokens];
  __shared__ double waves[kWide / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
  const Rows r = request(a, b);
  for (int i = tid; i < r.n; i += kWide) parents[i] = a.parents[r.q0 + i];
  __syncthreads();
  int cur = 0, depth = 0, refused = 0;
  double taken = 0.0, total = 1.0;  // C and T
  bool summed = true;               // whether T is C's
  // every thread takes every step alike: what it depends on is read by all
  for (int j = 1; j < r.n && depth < a.depth; ++j) {
    if (parents[j] != cur) continue;
    const int64_t at_t = (int64_t)(r.q0 + cur) * a.t_row, at_d = (int64_t)(r.q0 + cur) * a.d_row;
    if (!summed) {
      double sum = 0.0;
      for (int v = 8 * tid; v < a.V; v += 8 * kWide) {
        float pf[8], qf[8];
        load8<KIND>(a.target, at_t, v, a.V, pf);
        load8<KIND>(a.draft, at_d, v, a.V, qf);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += left_of(prob(pf[i]), prob(qf[i]), taken);
      }
      sum = wave_total(sum);
      if (lane == 0) waves[wave] = sum;
      __syncthreads();
      total = 0.0;
#pragma unroll
      for (int i = 0; i < kWide / 64; ++i) total += waves[i];
      __syncthreads();  // waves[] has been read
      summed = true;
    }
    const int x = a.tokens[r.q0 + j];
    double p = 0.0, q = 0.0;
    if (x >= 0 && x < a.V) {
      q = prob(value<KIND>(a.draft, at_d + x));
      p = left_of(prob(value<KIND>(a.target, at_t + x)), q, taken);
    }
    if ((double)a.accept[r.q0 + j] * q * total < p) {
      if (tid == 0) path[depth] = j;
      cur = j;
      ++depth;
      refused = 0;
      taken = 0.0;
      total = 1.0;
    } else {
      ++refused;
      taken += total;
      summed = !(total > 0.0);  // where nothing is left, nothing will be
    }
  }
  __syncthreads();
  for (int i = tid; i < a.depth; i += kWide) a.accepted[(int64_t)b * a.depth + i] = i < depth ? path[i] : -1;
  if (tid == 0) {
    a.counts[b] = depth;
    a.state[b] = State{r.n > 0 ? r.q0 + cur : -1, refused, taken};
  }
}

// ------------------------------------------------------------------------------ the sums
// WALKED: the walk has been done by a kernel of its own.
template <int KIND, bool DRAFT, bool WALKED>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(const VerifyArgs a) {
  __shared__ Walk w;
  __shared__ int list[kMaxTokens];
  __shared__ int listed;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), b = blockIdx.y, chunk = blockIdx.x;
  const Rows r = request(a, b);
  if (tid == 0) listed = 0;
  if constexpr (WALKED) {
    const State s = a.state[b];
    if (tid == 0) w.row = s.row, w.refused = s.refused, w.taken = s.taken;
    __syncthreads();
  } else {
    if (wave == 0) walk_tests<KIND>(a, r, lane, w);
    __syncthreads();
    if (chunk == 0) {
      for (int i = tid; i < a.depth; i += kThreads) a.accepted[(int64_t)b * a.depth + i] = i < w.depth ? w.path[i] : -1;
      if (!DRAFT)
        for (int i = tid; i < w.refused; i += kThreads) a.refused[r.q0 + i] = w.token[i];
      if (tid == 0) {
        a.counts[b] = w.depth;
        a.state[b] = State{w.row, w.refused, w.taken};
      }
    }
  }
  if (w.row < 0) return;

  const int u0 = chunk * a.chunk, u1 = min(u0 + a.chunk, a.units);
  Left l;
  l.list = list;
  l.refused = uniform(w.refused);
  l.taken = w.taken;
  if (!DRAFT) {
    const int64_t lo = (int64_t)u0 * a.unit, hi = (int64_t)u1 * a.unit;
    pick_listed(w.token, l.refused, (int)lo, (int)min(hi, (int64_t)a.V), list, &listed, tid, kThreads);
    __syncthreads();
    l.listed = uniform(listed);
  }
  const int64_t at_t = (int64_t)w.row * a.t_row, at_d = (int64_t)w.row * a.d_row;
  double* sums = a.sums + (int64_t)b * a.units;
  for (int u = u0 + wave; u < u1; u += kThreads / 64) {
    const double sum = unit_sum<KIND, DRAFT>(a, at_t, at_d, l, u, lane);
    if (lane == 63) sums[u] = sum;
  }
}

// ------------------------------------------------------------------------------ the token
template <int KIND, bool DRAFT>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(const VerifyArgs a) {
  __shared__ int list[kMaxTokens];
  __shared__ int listed, found, last;
  __shared__ double waves[kThreads / 64], base_of;
  constexpr int kPer = kVerifyUnits / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), b = blockIdx.x;
  const Rows r = request(a, b);
  const State s = a.state[b];
  if (s.row < 0) {
    if (tid == 0) a.next[b] = -1;
    return;
  }
  const float random = a.sample[b];
  const int64_t at_t = (int64_t)s.row * a.t_row, at_d = (int64_t)s.row * a.d_row;
  double* sums = a.sums + (int64_t)b * a.units;
  Left l;
  l.list = list;
  l.refused = s.refused;
  l.taken = s.taken;

  // the units' sums, kPer in a row for each thread
  double mine[kPer], before, total;
  for (int again = 0;; again = 1) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      mine[i] = kPer * tid + i < a.units ? sums[kPer * tid + i] : 0.0;
      sum += mine[i];
    }
    const double upto = wave_upto(sum);
    if (lane == 63) waves[wave] = upto;
    if (tid == 0) {
      listed = 0;
      found = a.units;
      last = -1;
    }
    __syncthreads();
    before = lane_before(upto);
    total = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) before += waves[w];
      total += waves[w];
    }
    if (total > 0.0 || again) break;
    // nothing left: the target's row
    l.refused = 0;
    for (int u = wave; u < a.units; u += kThreads / 64) {
      const double x = unit_sum<KIND, DRAFT>(a, at_t, at_d, l, u, lane);
      if (lane == 63) sums[u] = x;
    }
    __syncthreads();  // (the workgroup's own writes, in memory that it alone uses)
  }
  if (!(total > 0.0)) {
    if (tid == 0) a.next[b] = -1;
    return;
  }
  const double share = random < 1.f ? (double)fmaxf(random, 0.f) * total : __builtin_nan("");  // (no sum passes a NaN)
  double upto = before;
  int first = a.units, top = -1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    upto += mine[i];
    if (mine[i] > 0.0) {
      top = kPer * tid + i;
      if (first == a.units && upto > share) first = top;
    }
  }
  if (first < a.units) atomicMin(&found, first);
  if (top >= 0) atomicMax(&last, top);
  __syncthreads();
  const int unit = found < a.units ? found : last;  // none passes the share (a random number of 1, or NaN): the last
  if (tid == unit / kPer) {
    for (int i = 0; i < kPer; ++i)
      if (i < unit % kPer) before += mine[i];
    base_of = before;
  }
  const int lo = unit * a.unit, hi = (int)min((int64_t)lo + a.unit, (int64_t)a.V);
  if (!DRAFT) pick_listed(a.refused + r.q0, l.refused, lo, hi, list, &listed, tid, kThreads);
  __syncthreads();
  if (wave != 0) return;

  // the token
  l.listed = uniform(listed);
  const bool draft = DRAFT && l.refused > 0;
  double base = base_of;
  int token = -1;
  for (int v0 = lo; v0 < hi; v0 += kVerifyStep) {
    const int v = v0 + 8 * lane;
    float pf[8], qf[8];
    double x[8], sum = 0.0;
    load8<KIND>(a.target, at_t, v, hi, pf);
    if (draft) load8<KIND>(a.draft, at_d, v, hi, qf);
    left8(pf, qf, draft, l, v, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += x[i];
    const double all = wave_upto(sum);
    double now = base + lane_before(all);
    int here = -1;  // the first that passes the share, or the last that is above 0
    bool past = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      now += x[i];
      if (x[i] > 0.0 && !past) {
        here = v + i;
        past = now > share;
      }
    }
    const uint64_t hit = __ballot(past), some = __ballot(here >= 0);
    if (hit) {
      token = __builtin_amdgcn_readlane(here, __builtin_ctzll(hit));
      break;
    }
    if (some) token = __builtin_amdgcn_readlane(here, 63 - __builtin_clzll(some));
    base += lane_of(all, 63);
  }
  if (lane == 0) a.next[b] = token;
}

template <int KIND, bool DRAFT>
hipError_t launch(const VerifyArgs& a, int64_t B, int64_t chunks, hipStream_t stream) {
  const dim3 grid((unsigned)chunks, (unsigned)B);
  if (DRAFT && a.parents) {
    hipLaunchKernelGGL((verify_walk_kernel<KIND>), dim3((unsigned)B), dim3(kWide), 0, stream, a);
    hipLaunchKernelGGL((verify_sums_kernel<KIND, DRAFT, DRAFT>), grid, dim3(kThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((verify_sums_kernel<KIND, DRAFT, false>), grid, dim3(kThreads), 0, stream, a);
  }
  hipLaunchKernelGGL((verify_pick_kernel<KIND, DRAFT>), dim3((unsigned)B), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch(const VerifyArgs& a, int64_t B, int64_t chunks, hipStream_t stream) {
  return a.draft ? launch<KIND, true>(a, B, chunks, stream) : launch<KIND, false>(a, B, chunks, stream);
}

}  // namespace

hipError_t launch_verify(const VerifyProblem& p, const VerifyPlan& pl, void* workspace, hipStream_t stream) {
  VerifyArgs a{};
  a.target = p.target; a.draft = p.draft; a.tokens = p.tokens; a.parents = p.parents; a.starts = p.starts;
  a.accept = p.accept; a.sample = p.sample; a.accepted = p.accepted; a.counts = p.counts; a.next = p.next;
  char* ws = (char*)workspace;
  a.state = (State*)ws;
  a.sums = (double*)(ws + pl.sums);
  a.refused = (int32_t*)(ws + pl.refused);
  a.t_row = p.t_row; a.d_row = p.d_row; a.N = (int32_t)p.N; a.V = (int32_t)p.V; a.depth = (int32_t)p.depth;
  a.unit = (int32_t)pl.unit; a.units = (int32_t)pl.units; a.chunk = (int32_t)pl.chunk;
  switch (p.dtype) {
    case WQ_F32: return launch<kF32>(a, p.B, pl.chunks, stream);
    case WQ_F16: return launch<kF16>(a, p.B, pl.chunks, stream);
    default: return launch<kBf16>(a, p.B, pl.chunks, stream);
  }
}

}  // namespace wq
