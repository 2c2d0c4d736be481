// Norms of the heads of q and k, rotary positions of one or several axes, and the append of k and v to
// rows of a cache, in one pass:
//
//   x <- x / sqrt(mean(x^2) + eps) * weight      over a head (without a weight: x)
//   (u, v) -> factor * (u cos w - v sin w, v cos w + u sin w),   w = position of pair j's axis * inv_freq[j]
//
// Bound by memory: every element is read and written once.  G lanes of a wave hold a head, two pieces of 16 bytes
// each, so that its sum of squares is log2(G) cross-lane additions away and nothing but the angles goes
// through LDS.  In the half layout the two pieces turn with each other; interleaved, and past the rotated part, the
// second piece is any other.  Where the halves are not whole pieces, a lane finds the partners of its
// elements in LDS.  A head of v, and elements past the rotated part, are copied.
//
// The workgroup computes the cosines and sines of its tokens once, in LDS, for all heads; angles are products in fp64,
// taken in turns and reduced to half a turn before they become fp32.
//
// Measured (kernel trace): 16384 tokens of 32 + 8 + 8 heads of 128 in bf16 78.9 us, 5.1 TB/s of reads and writes, where a
// copy has 5.2 (87.9 with one piece a lane), and 89.0 with 20 elements that turn (kOdd); 6001 tokens of three axes,
// interleaved, heads of 96, 26.0 us (113 MB at 4.3 TB/s, within the 256 MB cache); 8 tokens 4.2 us.  Without weights this is
// rope's formula; calls of 16384 tokens as above, in us, rope's kernel first: 128 elements that turn 76.4 and 76.6,
// interleaved 74.8 and 76.4, 64 elements 81.6 and 75.2, 20 elements 377 and 79.8.
#include <algorithm>

#include "serve_device.h"
#include "serve_step_kernels.h"

namespace wq {
namespace {

constexpr double kInvTwoPi = 0.15915494309189533577;
enum Mode { kHalf, kPairs, kOdd };  // half layout in whole 8s; interleaved; half layout otherwise

struct NormRopeArgs {
  // of q, k and v
  const uint16_t* src[3];
  uint16_t* dst[3];
  const void* weight[3];
  int64_t src_t[3], src_h[3], dst_t[3], dst_h[3];
  int32_t wide[3];                        // weights in fp32
  const int32_t *positions, *slots, *axis_of;
  const float* inv_freq;
  int64_t T, S;
  int64_t t_base;                         // the launch's first token, and the first of its heads
  int32_t h_base;
  int32_t hq, hkv, heads, half, d, axes;  // heads: of a token, v's among them
  int32_t turn_units, units, second;      // lanes of a head whose pieces turn (kHalf), all of them; pieces to the second
  FastDiv by_heads, by_half;
  float factor, eps, inv_d;
};

// The sum over the G lanes of an aligned group, in all of them.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  auto add = [&](auto ctrl) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  add(std::integral_constant<int, 0xb1>());                         // lane ^ 1
  add(std::integral_constant<int, 0x4e>());                         // lane ^ 2
  if constexpr (G >= 8) add(std::integral_constant<int, 0x141>());  // the other 4 of 8
  if constexpr (G >= 16) add(std::integral_constant<int, 0x140>()); // the other 8 of 16
  return v;
}

template <bool BF16>
__device__ __forceinline__ void widen(const u32x4_t& x, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = act_to_f32<BF16>((uint16_t)x[i]);
    f[2 * i + 1] = act_to_f32<BF16>((uint16_t)(x[i] >> 16));
  }
}

template <bool BF16>
__device__ __forceinline__ u32x4_t narrow(const float* f) {
  return u32x4_t{pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]), pack2<BF16>(f[6], f[7])};
}

// weight[e .. e + 7]
template <bool BF16>
__device__ __forceinline__ void load_weight(const void* weight, bool wide, int e, float* w) {
  if (wide) {
    const f32x4_t lo = *(const f32x4_t*)((const float*)weight + e), hi = *(const f32x4_t*)((const float*)weight + e + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lo[i], w[4 + i] = hi[i];
  } else {
    widen<BF16>(*(const u32x4_t*)((const uint16_t*)weight + e), w);
  }
}

template <class T>
__device__ __forceinline__ T pick(const T* of, int kind) { return kind == 0 ? of[0] : kind == 1 ? of[1] : of[2]; }

template <bool BF16, int G, int MODE>
__global__ __launch_bounds__(256) void norm_rope_kernel(const NormRopeArgs a) {
  extern __shared__ __align__(16) float2 turns[];  // (cos, sin) of each token of the workgroup and each pair
  __shared__ __align__(16) float rows[MODE == kOdd ? 256 * 16 : 1];
  constexpr int Groups = 256 / G;
  const int tid = threadIdx.x, unit = tid % G, group = tid / G;
  // one head for a group of lanes; a launch has fewer than 2^30
  const uint32_t first = (uint32_t)a.h_base + blockIdx.x * Groups, before = divide(first, a.by_heads);
  const int64_t t0 = a.t_base + before;
  const int h0 = (int)(first - before * (uint32_t)a.heads);
  const uint32_t left = (uint32_t)min(a.T - t0, (int64_t)1 << 20);  // tokens from t0 on
  const int tokens = (int)min(left, divide((uint32_t)(h0 + Groups - 1), a.by_heads) + 1);

  // this lane's head, its token of the workgroup's, and its pieces
  const uint32_t x0 = (uint32_t)(h0 + group), token = divide(x0, a.by_heads);
  const int head = (int)(x0 - token * (uint32_t)a.heads);
  const int kind = head < a.hq ? 0 : head < a.hq + a.hkv ? 1 : 2;
  const int h = head - (kind == 0 ? 0 : kind == 1 ? a.hq : a.hq + a.hkv);
  const bool turning = MODE != kHalf || unit < a.turn_units;
  const int piece = turning ? unit : unit + a.turn_units;       // kHalf: past both halves
  const int lo = 8 * piece, hi = lo + 8 * (turning ? a.second : (a.units - a.turn_units));
  const bool one = unit < a.units && token < left, two = one && hi < a.d;
  const void* weight = pick(a.weight, kind);
  const bool wide = pick(a.wide, kind);

  const int64_t src_t = pick(a.src_t, kind);
  const uint16_t* src = pick(a.src, kind) + t0 * src_t + (uint64_t)token * src_t + (uint64_t)(uint32_t)h * pick(a.src_h, kind);
  uint16_t* dst = nullptr;  // null: no token, or one whose slot drops its k and v
  u32x4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
  if (one) {
    x = *(const u32x4_t*)(src + lo);
    if (two) y = *(const u32x4_t*)(src + hi);
    int64_t row = t0 + token;
    if (kind != 0 && a.slots) row = a.slots[row];
    if (kind == 0 || (row >= 0 && row < a.S))
      dst = pick(a.dst, kind) + row * pick(a.dst_t, kind) + (uint64_t)(uint32_t)h * pick(a.dst_h, kind);
  }
  float wl[8], wh[8];
  if (weight && one) {
    load_weight<BF16>(weight, wide, lo, wl);
    if (two) load_weight<BF16>(weight, wide, hi, wh);
  }

  for (int i = tid; i < tokens * a.half; i += 256) {
    const int tk = (int)divide((uint32_t)i, a.by_half), j = i - tk * a.half;
    const uint32_t axis = a.axis_of ? (uint32_t)a.axis_of[j] : 0;
    const int pos = axis < (uint32_t)a.axes ? a.positions[axis * a.T + t0 + tk] : 0;
    const double turn = (double)pos * (double)a.inv_freq[j] * kInvTwoPi;
    float s, c;
    sincospif(2.f * (float)(turn - rint(turn)), &s, &c);
    turns[i] = make_float2(a.factor * c, a.factor * s);
  }
  __syncthreads();

  float f[8], g[8];
  widen<BF16>(x, f);
  widen<BF16>(y, g);
  if (weight) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], fmaf(g[i], g[i], sum));
    sum = group_sum<G>(sum);
    const float mean = fmaf(sum, a.inv_d, a.eps);
    float by = __builtin_amdgcn_rsqf(mean);
    if (BF16 && !(mean < __builtin_inff())) {  // squares of bf16 pass fp32: with a factor of 2^-70
      constexpr float kDown = 0x1p-70f;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] *= kDown;
        g[i] *= kDown;
        sum = fmaf(f[i], f[i], fmaf(g[i], g[i], sum));
      }
      by = __builtin_amdgcn_rsqf(fmaf(group_sum<G>(sum), a.inv_d, a.eps * kDown * kDown));
    }
    if (one)
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // the norm first: of a head and a weight far from 1, by * weight leaves fp32
        f[i] = f[i] * by * wl[i];
        if (two) g[i] = g[i] * by * wh[i];
      }
  }
  const float2* cs = turns + token * a.half;
  if constexpr (MODE == kOdd) {
    float* row = rows + 16 * G * group;
    if (kind < 2 && one) {
      *(f32x4_t*)(row + lo) = f32x4_t{f[0], f[1], f[2], f[3]};
      *(f32x4_t*)(row + lo + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
      if (two) {
        *(f32x4_t*)(row + hi) = f32x4_t{g[0], g[1], g[2], g[3]};
        *(f32x4_t*)(row + hi + 4) = f32x4_t{g[4], g[5], g[6], g[7]};
      }
    }
    // the group's lanes are of one wave: what they wrote is there once its LDS writes are done
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
    __builtin_amdgcn_wave_barrier();
    auto turned = [&](float mine, int at) {
      if (at >= 2 * a.half) return mine;
      const bool low = at < a.half;
      const float other = row[low ? at + a.half : at - a.half];
      const float2 z = cs[low ? at : at - a.half];
      return low ? mine * z.x - other * z.y : mine * z.x + other * z.y;
    };
    if (kind < 2 && one && dst)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = turned(f[i], lo + i);
        if (two) g[i] = turned(g[i], hi + i);
      }
  } else if constexpr (MODE == kPairs) {
    auto turn = [&](float* v, int at) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (at / 2 + p < a.half) {
          const float2 z = cs[at / 2 + p];
          const float u = v[2 * p], w = v[2 * p + 1];
          v[2 * p] = u * z.x - w * z.y;
          v[2 * p + 1] = w * z.x + u * z.y;
        }
    };
    if (kind < 2 && dst) {
      turn(f, lo);
      if (two) turn(g, hi);
    }
  } else if (kind < 2 && turning && dst) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 z = cs[lo + i];
      const float u = f[i], v = g[i];
      f[i] = u * z.x - v * z.y;
      g[i] = v * z.x + u * z.y;
    }
  }
  if (!dst) return;
  *(u32x4_t*)(dst + lo) = kind < 2 ? narrow<BF16>(f) : x;
  if (two) *(u32x4_t*)(dst + hi) = kind < 2 ? narrow<BF16>(g) : y;
}

template <bool BF16, int MODE>
hipError_t launch(NormRopeArgs a, hipStream_t stream) {
  const int g = a.units <= 4 ? 4 : a.units <= 8 ? 8 : 16;
  void (*kern)(NormRopeArgs) = nullptr;
  switch (g) {
    case 4: kern = norm_rope_kernel<BF16, 4, MODE>; break;
    case 8: kern = norm_rope_kernel<BF16, 8, MODE>; break;
    default: kern = norm_rope_kernel<BF16, 16, MODE>; break;
  }
  const int64_t groups = 256 / g, blocks = (a.T * a.heads + groups - 1) / groups;
  // tokens that this many heads in a row can touch: at most 20 KB of LDS
  const int64_t tokens = std::min<int64_t>(a.T, groups / a.heads + 2);
  const size_t lds = (size_t)tokens * a.half * sizeof(float2);
  constexpr int64_t kMost = 1 << 23;  // workgroups of one launch: its threads stay below 2^32
  for (int64_t b = 0; b < blocks; b += kMost) {
    a.t_base = b * groups / a.heads;
    a.h_base = (int32_t)(b * groups % a.heads);
    hipLaunchKernelGGL(kern, dim3((unsigned)std::min(kMost, blocks - b)), dim3(256), lds, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeProblem& n, hipStream_t stream) {
  const RopeProblem& p = n.rope;
  NormRopeArgs a{};
  a.src[0] = (const uint16_t*)p.q; a.src[1] = (const uint16_t*)p.k; a.src[2] = (const uint16_t*)p.v;
  a.dst[0] = (uint16_t*)p.qo; a.dst[1] = (uint16_t*)p.ko; a.dst[2] = (uint16_t*)p.vo;
  a.weight[0] = n.q_weight; a.weight[1] = n.k_weight; a.wide[0] = n.q_weight32; a.wide[1] = n.k_weight32;
  a.src_t[0] = p.q_t; a.src_t[1] = p.k_t; a.src_t[2] = p.v_t; a.src_h[0] = p.q_h; a.src_h[1] = p.k_h; a.src_h[2] = p.v_h;
  a.dst_t[0] = p.qo_t; a.dst_t[1] = p.ko_t; a.dst_t[2] = p.vo_t;
  a.dst_h[0] = p.qo_h; a.dst_h[1] = p.ko_h; a.dst_h[2] = p.vo_h;
  a.positions = p.positions; a.slots = p.slots; a.inv_freq = p.inv_freq; a.axis_of = n.axis_of;
  a.T = p.T; a.S = p.S; a.hq = p.hq; a.hkv = p.hkv; a.half = p.half; a.d = p.d; a.axes = n.axes;
  a.heads = p.hq + p.hkv + (p.v ? p.hkv : 0);
  a.factor = p.factor; a.eps = n.eps; a.inv_d = 1.f / (float)p.d;
  a.by_heads = fast_div((uint32_t)a.heads); a.by_half = fast_div((uint32_t)p.half);
  const bool bf16 = p.act == WQ_BF16;
  if (!p.interleaved && p.half % 8 == 0) {  // pairs of pieces that turn with each other, then pairs of the others
    a.turn_units = a.second = p.half / 8;
    a.units = a.turn_units + ((p.d - 2 * p.half) / 8 + 1) / 2;
    return bf16 ? launch<true, kHalf>(a, stream) : launch<false, kHalf>(a, stream);
  }
  a.units = a.second = (p.d / 8 + 1) / 2;
  if (p.interleaved) return bf16 ? launch<true, kPairs>(a, stream) : launch<false, kPairs>(a, stream);
  return bf16 ? launch<true, kOdd>(a, stream) : launch<false, kOdd>(a, stream);
}

}  // namespace wq
