// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// The tests of a request's tokens need one probability of the target's and one of the draft's each, whatever
// the vocabulary's size; only the row of the last accepted token is read whole, for what is left of it
// after the refused children, r(x) = max(p(x) - q(x), 0) or p(x) without the refused tokens, and the first x
// whose running sum passes u times the whole.
//
//   sums: each workgroup has a chunk of a request's row.  It walks through the tests itself (the wave's lanes hold
//     the tokens, so that a step is a ballot), which takes less than a launch of its own, and sums its
//     chunk of r, and of p, which stands for r where nothing is left of that.
//   pick: a workgroup for each request finds the chunk that the random share falls into and the token in it.
//
// Where drafts of a tree have probabilities, the second child of a token is tested against what the first left,
// divided by its sum: a row to be summed in the middle of the walk.  There a workgroup for each request walks
// first (walk), and the sums take up what it found.
//
// Everything that is compared or summed is fp64, in an order that depends on sizes alone: equal calls give
// equal tokens, and a token differs from the exact one where the random number is within 2^-50 of a
// border of its running sums (of V borders, in fp32 one in a hundred calls would be so near).
#include <algorithm>

#include "serve_device.h"
#include "serve_step_kernels.h"
#include "serve_tile.h"

namespace wq {
namespace {

constexpr int kThreads = 256;       // of the sums
constexpr int kWide = 1024;         // of the pick and the walk of its own
constexpr int kMaxTokens = kVerifyTokens;

struct State {
  int32_t row;      // of the last accepted token; -1: a request without tokens
  int32_t refused;  // children refused since
  int32_t pad[2];
};
static_assert(sizeof(State) == kVerifyStateBytes, "the plan's size of a state");

struct VerifyArgs {
  const void *target, *draft;
  const int32_t *tokens, *parents, *starts;
  const float *accept, *sample;
  int32_t *accepted, *counts, *next;
  State* state;
  double* sums;      // (of r, of p) of each request's chunks
  double* scales;    // with draft: a request's refusals' sums, from its first row on
  int32_t* refused;  // without: the refused tokens
  int64_t t_row, d_row;
  int32_t N, V, depth, chunk, chunks;
};

enum Kind { kF32, kF16, kBf16 };

template <int KIND>
__device__ __forceinline__ float value(const void* base, int64_t i) {
  if constexpr (KIND == kF32) return ((const float*)base)[i];
  else return act_to_f32<KIND == kBf16>(((const uint16_t*)base)[i]);
}
// A probability: negative numbers and NaN are 0.
__device__ __forceinline__ double prob(float v) { return (double)fmaxf(v, 0.f); }

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
  double scale[kMaxTokens];   // the sums that refusals left (trees with draft)
};

__device__ __forceinline__ double shuffled(double v, int lane) { return __shfl(v, lane, 64); }

// The tests of a request's tokens by one wave; `again`(row, refusals): the scale of one more refusal, where the
// next child needs it (trees with draft; all threads of the workgroup take part).
//
// What is left at token x after c refusals, with draft: r_0 = p, r_(i+1) = max(r_i - q, 0) / scale_i.
__device__ __forceinline__ double left_of(double p, double q, const double* scale, int c) {
  for (int i = 0; i < c; ++i) {
    p = fmax(p - q, 0.0);
    p = scale[i] > 0.0 ? p / scale[i] : 0.0;
  }
  return p;
}

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
      const int x = __shfl(token, at, 64);
      const double ux = (double)__shfl(u, at, 64), qx = shuffled(q, at);
      double px = shuffled(p, at);
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

__device__ __forceinline__ double wave_total(double v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// What is left of a row at the 8 elements from v on; list: the refused tokens (without draft) of this chunk.
struct Left {
  const double* scale = nullptr;
  const int* list = nullptr;
  int refused = 0, listed = 0;
};

__device__ __forceinline__ void left8(const float* pf, const float* qf, bool draft, const Left& l, int v, double* r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = prob(pf[i]);
  if (draft) {
    if (l.refused > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = fmax(left_of(r[i], prob(qf[i]), l.scale, l.refused - 1) - prob(qf[i]), 0.0);
    }
  } else {
    for (int k = 0; k < l.listed; ++k) {
      const uint32_t in = (uint32_t)(l.list[k] - v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in == (uint32_t)i) r[i] = 0.0;
    }
  }
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
  __shared__ Walk w;
  __shared__ int parents[kMaxTokens];
  __shared__ double waves[kWide / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
  const Rows r = request(a, b);
  for (int i = tid; i < r.n; i += kWide) parents[i] = a.parents[r.q0 + i];
  __syncthreads();
  int cur = 0, depth = 0, refused = 0, summed = 0;  // summed: refusals whose scales are known
  // every thread takes every step alike: what it depends on is read by all
  for (int j = 1; j < r.n && depth < a.depth; ++j) {
    if (parents[j] != cur) continue;
    const int64_t at_t = (int64_t)(r.q0 + cur) * a.t_row, at_d = (int64_t)(r.q0 + cur) * a.d_row;
    while (summed < refused) {
      double sum = 0.0;
      for (int v = 8 * tid; v < a.V; v += 8 * kWide) {
        float pf[8], qf[8];
        load8<KIND>(a.target, at_t, v, a.V, pf);
        load8<KIND>(a.draft, at_d, v, a.V, qf);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += fmax(left_of(prob(pf[i]), prob(qf[i]), w.scale, summed) - prob(qf[i]), 0.0);
      }
      sum = wave_total(sum);
      __syncthreads();
      if (lane == 0) waves[wave] = sum;
      __syncthreads();
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < kWide / 64; ++i) sum += waves[i];
      if (tid == 0) w.scale[summed] = sum;
      __syncthreads();
      ++summed;
    }
    const int x = a.tokens[r.q0 + j];
    double p = 0.0, q = 0.0;
    if (x >= 0 && x < a.V) {
      q = prob(value<KIND>(a.draft, at_d + x));
      p = left_of(prob(value<KIND>(a.target, at_t + x)), q, w.scale, refused);
    }
    if ((double)a.accept[r.q0 + j] * q < p) {
      if (tid == 0) w.path[depth] = j;
      cur = j;
      ++depth;
      refused = summed = 0;
      __syncthreads();  // the scales have been read
    } else {
      ++refused;
    }
  }
  __syncthreads();
  for (int i = tid; i < refused - 1; i += kWide) a.scales[r.q0 + i] = w.scale[i];
  for (int i = tid; i < a.depth; i += kWide) a.accepted[(int64_t)b * a.depth + i] = i < depth ? w.path[i] : -1;
  if (tid == 0) {
    a.counts[b] = depth;
    a.state[b] = State{r.n > 0 ? r.q0 + cur : -1, refused, {0, 0}};
  }
}

// ------------------------------------------------------------------------------ the sums
// WALKED: the walk has been done by a kernel of its own.
template <int KIND, bool DRAFT, bool WALKED>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(const VerifyArgs a) {
  __shared__ Walk w;
  __shared__ int list[kMaxTokens];
  __shared__ int listed;
  __shared__ double waves[kThreads / 64][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.y, chunk = blockIdx.x;
  const Rows r = request(a, b);
  if (tid == 0) listed = 0;
  if constexpr (WALKED) {
    const State s = a.state[b];
    if (tid == 0) w.row = s.row, w.refused = s.refused;
    for (int i = tid; i < s.refused - 1; i += kThreads) w.scale[i] = a.scales[r.q0 + i];
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
        a.state[b] = State{w.row, w.refused, {0, 0}};
      }
    }
  }
  if (w.row < 0) return;

  const int lo = chunk * a.chunk, hi = min(lo + a.chunk, a.V);
  Left l;
  l.scale = w.scale;
  l.list = list;
  l.refused = uniform(w.refused);
  if (!DRAFT) {
    pick_listed(w.token, l.refused, lo, hi, list, &listed, tid, kThreads);
    __syncthreads();
    l.listed = uniform(listed);
  }
  const int64_t at_t = (int64_t)w.row * a.t_row, at_d = (int64_t)w.row * a.d_row;
  const bool draft = DRAFT && l.refused > 0;  // without a refusal p is all that is read
  double left = 0.0, whole = 0.0;
#pragma unroll 2
  for (int v = lo + 8 * tid; v < hi; v += 8 * kThreads) {
    float pf[8], qf[8];
    double x[8];
    load8<KIND>(a.target, at_t, v, hi, pf);
    if (draft) load8<KIND>(a.draft, at_d, v, hi, qf);
    left8(pf, qf, draft, l, v, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      left += x[i];
      whole += prob(pf[i]);
    }
  }
  left = wave_total(left);
  whole = wave_total(whole);
  if (lane == 0) waves[wave][0] = left, waves[wave][1] = whole;
  __syncthreads();
  if (tid == 0) {
    left = whole = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) left += waves[i][0], whole += waves[i][1];
    double* to = a.sums + ((int64_t)b * a.chunks + chunk) * 2;
    to[0] = left;
    to[1] = whole;
  }
}

// ------------------------------------------------------------------------------ the token
// What stands before this thread of a sum over the workgroup's threads, in their order.
__device__ __forceinline__ double before(double v, double* waves, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  double upto = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double t = __shfl_up(upto, o, 64);
    if (lane >= o) upto += t;
  }
  __syncthreads();
  if (lane == 63) waves[wave] = upto;
  __syncthreads();
  double sum = 0.0;
  for (int w = 0; w < wave; ++w) sum += waves[w];
  const double prior = __shfl_up(upto, 1, 64);
  return sum + (lane ? prior : 0.0);
}

template <int KIND, bool DRAFT>
__global__ __launch_bounds__(kWide) void verify_pick_kernel(const VerifyArgs a) {
  __shared__ double scale[kMaxTokens];
  __shared__ int list[kMaxTokens];
  __shared__ int listed, found, last;
  __shared__ double waves[kWide / 64], total[2], base_of;
  const int tid = threadIdx.x, b = blockIdx.x;
  const Rows r = request(a, b);
  const State s = a.state[b];
  if (s.row < 0) {
    if (tid == 0) a.next[b] = -1;
    return;
  }
  if (tid == 0) {
    listed = 0;
    found = a.chunks;
    last = -1;
  }
  if (DRAFT && a.parents)
    for (int i = tid; i < s.refused - 1; i += kWide) scale[i] = a.scales[r.q0 + i];

  // the chunk: there are at most kWide, one for each thread
  const double* sums = a.sums + ((int64_t)b * a.chunks + tid) * 2;
  double mine[2] = {0.0, 0.0}, pre[2];
  if (tid < a.chunks) mine[0] = sums[0], mine[1] = sums[1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    pre[i] = before(mine[i], waves, tid);
    if (tid == kWide - 1) total[i] = pre[i] + mine[i];
  }
  __syncthreads();
  const int k = total[0] > 0.0 ? 0 : 1;  // nothing left: the target's row
  if (!(total[k] > 0.0)) {
    if (tid == 0) a.next[b] = -1;
    return;
  }
  const float u = a.sample[b];
  const double share = u < 1.f ? (double)fmaxf(u, 0.f) * total[k] : __builtin_nan("");  // (no sum passes a NaN)
  if (pre[k] + mine[k] > share && mine[k] > 0.0) atomicMin(&found, tid);
  if (mine[k] > 0.0) atomicMax(&last, tid);
  __syncthreads();
  const int chunk = found < a.chunks ? found : last;  // none passes the share (a random number of 1, or NaN): the last
  if (tid == chunk) base_of = pre[k];
  __syncthreads();
  double base = base_of;

  // the token
  const int lo = chunk * a.chunk, hi = min(lo + a.chunk, a.V);
  Left l;
  l.scale = scale;
  l.list = list;
  l.refused = k == 0 ? s.refused : 0;
  if (!DRAFT && k == 0) pick_listed(a.refused + r.q0, s.refused, lo, hi, list, &listed, tid, kWide);
  __syncthreads();
  l.listed = listed;
  if (tid == 0) {
    found = a.V;
    last = -1;
  }
  __syncthreads();
  const int64_t at_t = (int64_t)s.row * a.t_row, at_d = (int64_t)s.row * a.d_row;
  const bool draft = DRAFT && l.refused > 0;
  for (int v0 = lo; v0 < hi; v0 += 8 * kWide) {
    const int v = v0 + 8 * tid;
    float pf[8], qf[8];
    double x[8], sum = 0.0;
    load8<KIND>(a.target, at_t, v, hi, pf);
    if (draft) load8<KIND>(a.draft, at_d, v, hi, qf);
    left8(pf, qf, draft, l, v, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += x[i];
    const double pre = base + before(sum, waves, tid);
    double upto = pre;
    int mine = a.V, top = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      upto += x[i];
      if (x[i] > 0.0) {
        top = v + i;
        if (mine == a.V && upto > share) mine = v + i;
      }
    }
    if (mine < a.V) atomicMin(&found, mine);
    if (top >= 0) atomicMax(&last, top);
    __syncthreads();
    if (tid == kWide - 1) base_of = pre + sum;
    __syncthreads();
    base = base_of;
    if (found < a.V) break;
  }
  if (tid == 0) a.next[b] = found < a.V ? found : last;
}

template <int KIND, bool DRAFT>
hipError_t launch(const VerifyArgs& a, int64_t B, hipStream_t stream) {
  const dim3 grid((unsigned)a.chunks, (unsigned)B);
  if (DRAFT && a.parents) {
    hipLaunchKernelGGL((verify_walk_kernel<KIND>), dim3((unsigned)B), dim3(kWide), 0, stream, a);
    hipLaunchKernelGGL((verify_sums_kernel<KIND, DRAFT, DRAFT>), grid, dim3(kThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((verify_sums_kernel<KIND, DRAFT, false>), grid, dim3(kThreads), 0, stream, a);
  }
  hipLaunchKernelGGL((verify_pick_kernel<KIND, DRAFT>), dim3((unsigned)B), dim3(kWide), 0, stream, a);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch(const VerifyArgs& a, int64_t B, hipStream_t stream) {
  return a.draft ? launch<KIND, true>(a, B, stream) : launch<KIND, false>(a, B, stream);
}

}  // namespace

hipError_t launch_verify(const VerifyProblem& p, const VerifyPlan& pl, void* workspace, hipStream_t stream) {
  VerifyArgs a{};
  a.target = p.target; a.draft = p.draft; a.tokens = p.tokens; a.parents = p.parents; a.starts = p.starts;
  a.accept = p.accept; a.sample = p.sample; a.accepted = p.accepted; a.counts = p.counts; a.next = p.next;
  char* ws = (char*)workspace;
  a.state = (State*)ws;
  a.sums = (double*)(ws + pl.sums);
  a.scales = (double*)(ws + pl.refused);
  a.refused = (int32_t*)(ws + pl.refused);
  a.t_row = p.t_row; a.d_row = p.d_row; a.N = (int32_t)p.N; a.V = (int32_t)p.V; a.depth = (int32_t)p.depth;
  a.chunk = (int32_t)pl.chunk; a.chunks = (int32_t)pl.chunks;
  switch (p.dtype) {
    case WQ_F32: return launch<kF32>(a, p.B, stream);
    case WQ_F16: return launch<kF16>(a, p.B, stream);
    default: return launch<kBf16>(a, p.B, stream);
  }
}

}  // namespace wq
