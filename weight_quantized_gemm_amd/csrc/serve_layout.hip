// The paged layout of a step from the requests' lengths: starts of the requests' tokens, and of each token
// its request, cache row, position and row of the tree mask, with the requests' new pages taken from a stack.
//
// Integers only, a few bytes a token: bound by the launch and the chain lengths -> sums -> request -> page -> row.
// One launch does it all: each workgroup sums the lengths of all requests anew (a window of kWindow at a
// time, in LDS, while its tokens fall into the window), which takes less than a second launch would,
// and finds its tokens' requests by bisection there.  Nothing is passed between workgroups, so no
// order of execution shows.
//
// A new page is written to the table by the token that is the first in it; tokens of new pages take
// their page from the stack themselves and never read what another token writes.
#include <algorithm>

#include "serve_device.h"
#include "serve_step_kernels.h"

namespace wq {
namespace {

constexpr int kThreads = 256;
constexpr int kWindow = 4096;   // requests whose sums stand in LDS at a time
constexpr int kPer = kWindow / kThreads;
constexpr int kBehind = 768;    // tokens before a pass's whose parents stand in LDS too

struct LayoutArgs {
  const int32_t *context, *fresh, *free_pages, *free_count, *offsets, *parents;
  int32_t *table, *starts, *requests, *positions, *slots, *free_left;
  uint32_t* mask;
  int32_t B, N, width, words;
  int64_t F;
  int32_t chunk;  // tokens of a workgroup, a multiple of kThreads
  FastDiv by_page;
};

// Sums over the workgroup's threads, at most `most` (saturated sums of numbers >= 0 are associative):
// returns what stands before this thread; total: of all.
__device__ __forceinline__ int sum_before(int v, int most, int* waves, int tid, int& total) {
  const int lane = tid & 63, wave = tid >> 6;
  int upto = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(upto, o, 64);
    if (lane >= o) upto = min(upto + t, most);
  }
  __syncthreads();  // waves[] of the sums before have been read
  if (lane == 63) waves[wave] = upto;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) before = min(before + waves[w], most);
    total = min(total + waves[w], most);
  }
  const int prior = __shfl_up(upto, 1, 64);
  return min(before + (lane ? prior : 0), most);
}

__device__ __forceinline__ int pages_for(int64_t keys, const LayoutArgs& a) {  // at most the table's width
  const uint32_t k = (uint32_t)min(keys, (int64_t)a.width * a.by_page.d);      // below 2^31
  return k == 0 ? 0 : (int)divide(k - 1, a.by_page) + 1;
}

__global__ __launch_bounds__(kThreads) void layout_kernel(const LayoutArgs a) {
  __shared__ int starts[kWindow + 1], ctx[kWindow], taken[kWindow];
  __shared__ int up[kBehind + kThreads];
  __shared__ int waves[kThreads / 64];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, (int64_t)a.N);
  const int count = (int)min(max((int64_t)a.free_count[0], (int64_t)0), a.F);
  int tokens = 0, pages = 0;  // of the windows before

  for (int b0 = 0; b0 < a.B || b0 == 0; b0 += kWindow) {
    const int n = min(kWindow, a.B - b0), per = (n + kThreads - 1) / kThreads, mine = tid * per;
    // tokens: at most N less the ones before, in all
    int c[kPer], f[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool on = i < per && mine + i < n;
      c[i] = on ? max(a.context[b0 + mine + i], 0) : 0;
      f[i] = on ? min(max(a.fresh[b0 + mine + i], 0), a.N) : 0;
      sum = min(sum + f[i], a.N);
    }
    int total;
    int at = sum_before(sum, a.N, waves, tid, total);
    int need = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int from = min(tokens + at, a.N);
      at = min(at + f[i], a.N);
      f[i] = min(tokens + at, a.N) - from;  // what there is room for
      if (i < per && mine + i < n) {
        starts[mine + i] = from;
        ctx[mine + i] = c[i];
        need += pages_for((int64_t)c[i] + f[i], a) - pages_for(c[i], a);
      }
    }
    const int end = min(tokens + total, a.N);
    int all;
    int first = sum_before(need, 0x7fffffff, waves, tid, all);  // at most a page a token: no overflow
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per && mine + i < n) {
        taken[mine + i] = pages + first;
        first += pages_for((int64_t)c[i] + f[i], a) - pages_for(c[i], a);
      }
    if (tid == 0) starts[n] = end;
    __syncthreads();

    // the starts of one window in turn are written by one workgroup
    if ((b0 / kWindow) % gridDim.x == blockIdx.x)
      for (int i = tid; i <= n; i += kThreads)
        if (i < n || b0 + n >= a.B) a.starts[b0 + i] = starts[i];

    const int64_t lo = max(t0, (int64_t)tokens), hi = min(t1, (int64_t)end);
    for (int64_t p0 = t0 + (lo - t0) / kThreads * kThreads; p0 < hi; p0 += kThreads) {
      if (a.parents) {
        __syncthreads();
        for (int i = tid; i < kBehind + kThreads; i += kThreads) {
          const int64_t t = p0 - kBehind + i;
          up[i] = t >= 0 && t < a.N ? a.parents[t] : -1;
        }
        __syncthreads();
      }
      const int64_t t = p0 + tid;
      if (t < lo || t >= hi) continue;
      int l = 0, r = n;  // starts[l] <= t < starts[r]
      while (r - l > 1) {
        const int m = (l + r) >> 1;
        if (starts[m] <= (int)t) l = m;
        else r = m;
      }
      const int b = b0 + l, j = (int)t - starts[l];
      const int64_t key = (int64_t)ctx[l] + j;
      const int64_t offset = a.offsets ? a.offsets[b] : 0;

      // its page: the request's, or a new one
      int entry = -1, in = 0;
      if (key < (int64_t)a.width * a.by_page.d) {
        const int page = (int)divide((uint32_t)key, a.by_page), fresh = page - pages_for(ctx[l], a);
        int32_t* place = a.table + (int64_t)b * a.width + page;
        in = (int)((uint32_t)key - (uint32_t)page * a.by_page.d);
        if (fresh < 0) {
          entry = *place;
        } else {
          const int rank = count - 1 - (taken[l] + fresh);
          entry = rank >= 0 ? a.free_pages[rank] : -1;
          if (in == 0) *place = entry;
        }
      }
      const int64_t slot = (int64_t)entry * a.by_page.d + in;
      a.slots[t] = entry >= 0 && slot <= 0x7fffffff ? (int)slot : -1;
      if (a.requests) a.requests[t] = b;

      int depth = j;
      if (a.parents) {
        // a walk up to the root; ancestors come in descending order, so the words of the mask do too
        uint32_t* row = a.mask + t * a.words;
        int w = a.words - 1, node = j;
        uint32_t bits = 0;
        depth = -1;
        for (;;) {
          const int nw = node >> 5;
          while (w > nw) {
            row[w--] = bits;
            bits = 0;
          }
          if (nw < a.words) bits |= 1u << (node & 31);
          ++depth;
          const int64_t from = starts[l] + node - (p0 - kBehind);
          const int p = from >= 0 ? up[from] : a.parents[starts[l] + node];
          if (p < 0 || p >= node) break;
          node = p;
        }
        while (w >= 0) {
          row[w--] = bits;
          bits = 0;
        }
      }
      const int64_t pos = offset + ctx[l] + depth;
      a.positions[t] = (int)min(max(pos, (int64_t)INT32_MIN), (int64_t)INT32_MAX);
    }
    tokens = end;
    pages += all;
    __syncthreads();  // the window has been read
  }

  if (blockIdx.x == 0 && tid == 0) *a.free_left = count - pages;
  for (int64_t t = max(t0, (int64_t)tokens) + tid; t < t1; t += kThreads) {
    a.slots[t] = -1;
    a.positions[t] = 0;
    if (a.requests) a.requests[t] = -1;
    for (int w = 0; w < a.words; ++w) a.mask[t * a.words + w] = 0;
  }
}

}  // namespace

hipError_t launch_layout(const LayoutProblem& p, hipStream_t stream) {
  LayoutArgs a{};
  a.context = p.context; a.fresh = p.fresh; a.table = p.table; a.free_pages = p.free_pages; a.free_count = p.free_count;
  a.offsets = p.offsets; a.parents = p.parents; a.starts = p.starts; a.requests = p.requests;
  a.positions = p.positions; a.slots = p.slots; a.mask = p.mask; a.free_left = p.free_left;
  a.B = (int32_t)p.B; a.N = (int32_t)p.N; a.F = p.F; a.width = (int32_t)p.width; a.words = (int32_t)p.words;
  a.by_page = fast_div((uint32_t)p.page);
  // at most 1024 workgroups: each looks at all requests
  const int64_t passes = (p.N + kThreads - 1) / kThreads, each = std::max<int64_t>(1, (passes + 1023) / 1024);
  a.chunk = (int32_t)(each * kThreads);
  const int64_t blocks = std::max<int64_t>(1, (passes + each - 1) / each);
  hipLaunchKernelGGL(layout_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace wq
