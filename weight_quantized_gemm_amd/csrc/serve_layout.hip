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
//
// Measured (kernel trace): one token of each of 48 requests 4.9 us; 64 trees of up to 48 tokens, with the walks up the
// parents in LDS, 9.2; 4096 requests of 86237 tokens 7.6, 1.1 MB moved in twice the time of a
// bare launch.
#include <algorithm>

#include "serve_device.h"
#include "serve_step_kernels.h"

namespace wq {
namespace {

constexpr int kWindow = 4096;   // requests whose sums stand in LDS at a time
constexpr int kBehind = 768;    // tokens before a pass's whose parents stand in LDS too
typedef int32_t i32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

struct LayoutArgs {
  const int32_t *context, *fresh, *free_pages, *free_count, *offsets, *parents;
  int32_t *table, *starts, *requests, *positions, *slots, *free_left;
  uint32_t* mask;
  int32_t B, N, width, words;
  int64_t F;
  int32_t chunk;  // tokens of a workgroup, a multiple of its threads
  FastDiv by_page;
};

template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int v) {  // from another lane, 0 where there is none
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
// The sum of lanes 0 .. this one of numbers >= 0, at most `most` (saturated sums are associative).
__device__ __forceinline__ int wave_upto(int v, int most) {
  v = min(v + moved<0x111, 0xf>(v), most);
  v = min(v + moved<0x112, 0xf>(v), most);
  v = min(v + moved<0x114, 0xf>(v), most);
  v = min(v + moved<0x118, 0xf>(v), most);
  v = min(v + moved<0x142, 0xa>(v), most);     // lane 15 of rows 0 and 2 to rows 1 and 3
  return min(v + moved<0x143, 0xc>(v), most);  // lane 31 to rows 2 and 3
}
// The same without a limit, modulo 2^32.
__device__ __forceinline__ uint32_t wave_upto(uint32_t v) {
  v += moved<0x111, 0xf>((int)v);
  v += moved<0x112, 0xf>((int)v);
  v += moved<0x114, 0xf>((int)v);
  v += moved<0x118, 0xf>((int)v);
  v += moved<0x142, 0xa>((int)v);
  return v + moved<0x143, 0xc>((int)v);
}

__device__ __forceinline__ int pages_for(int64_t keys, const LayoutArgs& a) {  // at most the table's width
  const uint32_t k = (uint32_t)min(keys, (int64_t)a.width * a.by_page.d);      // below 2^31
  return k == 0 ? 0 : (int)divide(k - 1, a.by_page) + 1;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void layout_kernel(const LayoutArgs a) {
  constexpr int kPer = kWindow / THREADS, kWaves = THREADS / 64;
  __shared__ int starts[kWindow + 1], ctx[kWindow], taken[kWindow];
  __shared__ int up[kBehind + THREADS];
  __shared__ int waves[kWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, (int64_t)a.N);
  const int count = (int)min(max((int64_t)a.free_count[0], (int64_t)0), a.F);
  auto stage_parents = [&](int64_t p0) {
    for (int i = tid; i < kBehind + THREADS; i += THREADS) {
      const int64_t t = p0 - kBehind + i;
      up[i] = t >= 0 && t < a.N ? a.parents[t] : -1;
    }
  };
  int64_t staged = t0;
  if (a.parents) stage_parents(t0);  // on their way while the lengths are summed
  int tokens = 0, pages = 0;         // of the windows before
  const int most = a.N + 1;          // where sums of tokens stop

  for (int b0 = 0; b0 < a.B || b0 == 0; b0 += kWindow) {
    const int n = min(kWindow, a.B - b0);
    const int per = n <= THREADS ? 1 : (n + 4 * THREADS - 1) / (4 * THREADS) * 4, mine = tid * per;
    int c[kPer], f[kPer], sum = 0;
#pragma unroll
    for (int g = 0; g < kPer; g += 4) {
      if (per > 1 && g < per && mine + g + 3 < n) {
        const i32x4_any_t x = *(const i32x4_any_t*)(a.context + b0 + mine + g);
        const i32x4_any_t y = *(const i32x4_any_t*)(a.fresh + b0 + mine + g);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[g + i] = x[i], f[g + i] = y[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool on = g + i < per && mine + g + i < n;
          c[g + i] = on ? a.context[b0 + mine + g + i] : 0;
          f[g + i] = on ? a.fresh[b0 + mine + g + i] : 0;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = max(c[i], 0);
      f[i] = min(max(f[i], 0), most);
      sum = min(sum + f[i], most);
    }
    // Tokens and pages before this thread's requests in one step; again, where there are more tokens than room, with
    // what there is room for.
    int end, from = 0;
    uint32_t first, all;
    for (int clipped = 0;; clipped = 1) {
      uint32_t need = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < per) need += (uint32_t)(pages_for((int64_t)c[i] + f[i], a) - pages_for(c[i], a));
      const int upto = wave_upto(sum, most);
      const uint32_t need_upto = wave_upto(need);
      if (lane == 63) waves[wave][0] = upto, waves[wave][1] = (int)need_upto;
      __syncthreads();
      int before = 0, total = 0;
      all = 0;
      first = need_upto - need;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before = min(before + waves[w][0], most), first += (uint32_t)waves[w][1];
        total = min(total + waves[w][0], most);
        all += (uint32_t)waves[w][1];
      }
      from = min(tokens + before + moved<0x138, 0xf>(upto), a.N);
      end = min(tokens + total, a.N);
      if (clipped || tokens + total <= a.N) break;
      sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        f[i] = min(f[i], a.N - from - sum);
        sum += f[i];
      }
      __syncthreads();  // waves[] has been read
    }
    first += (uint32_t)pages;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per && mine + i < n) {
        starts[mine + i] = from;
        ctx[mine + i] = c[i];
        taken[mine + i] = (int)first;
        from += f[i];
        first += (uint32_t)(pages_for((int64_t)c[i] + f[i], a) - pages_for(c[i], a));
      }
    if (tid == 0) starts[n] = end;
    __syncthreads();

    // the starts of one window in turn are written by one workgroup
    if ((b0 / kWindow) % gridDim.x == blockIdx.x)
      for (int i = tid; i <= n; i += THREADS)
        if (i < n || b0 + n >= a.B) a.starts[b0 + i] = starts[i];

    const int64_t lo = max(t0, (int64_t)tokens), hi = min(t1, (int64_t)end);
    for (int64_t p0 = t0 + (lo - t0) / THREADS * THREADS; p0 < hi; p0 += THREADS) {
      if (a.parents && p0 != staged) {
        __syncthreads();
        stage_parents(staged = p0);
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
    pages += (int)all;
    __syncthreads();  // the window has been read
  }

  if (blockIdx.x == 0 && tid == 0) *a.free_left = count - pages;
  for (int64_t t = max(t0, (int64_t)tokens) + tid; t < t1; t += THREADS) {
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
  // Workgroups of 1024 threads where there are many requests for each to look at (4096 requests of 86237 tokens:
  // 17.2 us with 256 threads, 7.7 with 1024); of 256 where there are few, which start sooner.
  const bool wide = p.B > 1024;
  const int64_t threads = wide ? 1024 : 256;
  // at most 1024 workgroups, since each looks at all requests
  const int64_t passes = (p.N + threads - 1) / threads, each = std::max<int64_t>(1, (passes + 1023) / 1024);
  a.chunk = (int32_t)(each * threads);
  const dim3 grid((unsigned)std::max<int64_t>(1, (passes + each - 1) / each));
  if (wide) hipLaunchKernelGGL(layout_kernel<1024>, grid, dim3(1024), 0, stream, a);
  else hipLaunchKernelGGL(layout_kernel<256>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace wq
