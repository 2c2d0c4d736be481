// Norms of the heads of q and k, rotary positions of one or several axes, and the append of k and v to
// rows of a cache, in one pass:
//
//   x <- x / sqrt(mean(x^2) + eps) * weight      over a head (without a weight: x)
//   (u, v) -> factor * (u cos w - v sin w, v cos w + u sin w),   w = position of pair j's axis * inv_freq[j]
//
// Bound by memory: every element is read and written once.  G lanes of a wave hold a head, 16 or 32 bytes each, so
// that its sum of squares is log2(G) cross-lane additions away and nothing but the angles goes through LDS.
// In the half layout a lane holds 8 elements of the first half and the 8 that turn with them; interleaved, 8
// elements in a row.  Where the halves are not whole 8s, a lane holds 8 in a row and finds the partners in
// LDS (16384 tokens).  A head of v, and elements past the rotated part, are copied.
//
// The workgroup computes the cosines and sines of its tokens once, in LDS, for all heads; angles are products in fp64,
// taken in turns and reduced to half a turn before they become fp32.
#include <algorithm>

#include "serve_device.h"
#include "serve_step_kernels.h"

namespace wq {
namespace {

constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr int kItems = 2;  // heads of a group of lanes
enum Mode { kHalf, kPairs, kOdd };  // half layout in whole 8s; interleaved; half layout otherwise

struct NormRopeArgs {
  const uint16_t *q, *k, *v;
  uint16_t *qo, *ko, *vo;
  const int32_t *positions, *slots, *axis_of;
  const float* inv_freq;
  const void *q_weight, *k_weight;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, qo_t, qo_h, ko_t, ko_h, vo_t, vo_h;
  int64_t T, S, block0;
  int32_t hq, hkv, heads, half, d, axes;  // heads: of a token, v's among them
  int32_t turn_units, head_units;         // kHalf: units (of 16 elements) that turn, and all of a head
  int32_t q_weight32, k_weight32;
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
  if constexpr (G >= 32) {
    const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  }
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

// f *= weight[e .. e + 7] * by
template <bool BF16>
__device__ __forceinline__ void weigh(const void* weight, bool wide, int e, float by, float* f) {
  float w[8];
  if (wide) {
    const f32x4_t lo = *(const f32x4_t*)((const float*)weight + e), hi = *(const f32x4_t*)((const float*)weight + e + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lo[i], w[4 + i] = hi[i];
  } else {
    widen<BF16>(*(const u32x4_t*)((const uint16_t*)weight + e), w);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= by * w[i];
}

// What a group of lanes works on.
struct Item {
  const uint16_t* src = nullptr;
  uint16_t* dst = nullptr;  // null: no item, or a token whose slot drops it
  const void* weight = nullptr;
  int token = 0;            // of the workgroup
  bool wide = false, turns = false;
};

__device__ __forceinline__ Item find_item(const NormRopeArgs& a, int64_t t0, int h0, int i, int64_t last) {
  Item w;
  if (t0 * a.heads + h0 + i >= last) return w;
  const uint32_t x = (uint32_t)(h0 + i);
  w.token = (int)divide(x, a.by_heads);
  const int h = (int)(x - (uint32_t)w.token * (uint32_t)a.heads);
  const int64_t t = t0 + w.token;
  if (h < a.hq) {
    w.src = a.q + t * a.q_t + h * a.q_h;
    w.dst = a.qo + t * a.qo_t + h * a.qo_h;
    w.weight = a.q_weight;
    w.wide = a.q_weight32;
    w.turns = true;
    return w;
  }
  const int64_t row = a.slots ? a.slots[t] : t;
  const bool on = row >= 0 && row < a.S;
  if (h < a.hq + a.hkv) {
    w.src = a.k + t * a.k_t + (h - a.hq) * a.k_h;
    if (on) w.dst = a.ko + row * a.ko_t + (h - a.hq) * a.ko_h;
    w.weight = a.k_weight;
    w.wide = a.k_weight32;
    w.turns = true;
  } else {
    w.src = a.v + t * a.v_t + (h - a.hq - a.hkv) * a.v_h;
    if (on) w.dst = a.vo + row * a.vo_t + (h - a.hq - a.hkv) * a.vo_h;
  }
  return w;
}

template <bool BF16, int G, int MODE>
__global__ __launch_bounds__(256) void norm_rope_kernel(const NormRopeArgs a) {
  extern __shared__ __align__(16) float2 turns[];  // (cos, sin) of each token of the workgroup and each pair
  __shared__ __align__(16) float rows[MODE == kOdd ? 256 * 8 : 1];
  constexpr int Groups = 256 / G, E = kItems;
  const int tid = threadIdx.x, unit = tid % G, group = tid / G;
  const int64_t first = (a.block0 + blockIdx.x) * (Groups * E), last = a.T * a.heads;
  const int64_t t0 = first / a.heads;
  const int h0 = (int)(first - t0 * a.heads);
  const int tokens = (int)((min(first + Groups * E, last) - 1) / a.heads - t0) + 1;

  // a lane's elements: 8 from lo on and, where it turns in the half layout, 8 from lo + half on
  const bool two = MODE == kHalf && unit < a.turn_units;
  const bool has = MODE == kHalf ? unit < a.head_units : 8 * unit < a.d;
  const int lo = MODE == kHalf && !two ? 2 * a.half + 8 * (unit - a.turn_units) : 8 * unit;
  Item w[E];
  u32x4_t x[E], y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    w[e] = find_item(a, t0, h0, group + Groups * e, last);
    x[e] = y[e] = u32x4_t{0, 0, 0, 0};
    if (!w[e].dst || !has) continue;
    x[e] = *(const u32x4_t*)(w[e].src + lo);
    if (two) y[e] = *(const u32x4_t*)(w[e].src + lo + a.half);
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

#pragma unroll
  for (int e = 0; e < E; ++e) {
    float f[8], g[8];
    widen<BF16>(x[e], f);
    widen<BF16>(y[e], g);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], fmaf(g[i], g[i], sum));
    sum = group_sum<G>(sum);
    float by = 1.f / sqrtf(fmaf(sum, a.inv_d, a.eps));
    if (BF16 && w[e].weight && !(sum < __builtin_inff())) {  // squares of bf16 pass fp32: with a factor of 2^-70
      constexpr float kDown = 0x1p-70f;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] *= kDown;
        g[i] *= kDown;
        sum = fmaf(f[i], f[i], fmaf(g[i], g[i], sum));
      }
      by = 1.f / sqrtf(group_sum<G>(sum) * a.inv_d);
    }
    if (w[e].weight && w[e].dst && has) {
      weigh<BF16>(w[e].weight, w[e].wide, lo, by, f);
      if (two) weigh<BF16>(w[e].weight, w[e].wide, lo + a.half, by, g);
    }
    const float2* cs = turns + w[e].token * a.half;
    if constexpr (MODE == kOdd) {
      float* row = rows + 8 * G * group;
      if (w[e].turns) {
        *(f32x4_t*)(row + 8 * unit) = f32x4_t{f[0], f[1], f[2], f[3]};
        *(f32x4_t*)(row + 8 * unit + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
      }
      // the group's lanes are of one wave: what they wrote is there once its LDS writes are done
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
      __builtin_amdgcn_wave_barrier();
      if (w[e].turns && has)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = lo + i;
          if (at < 2 * a.half) {
            const bool low = at < a.half;
            const float other = row[low ? at + a.half : at - a.half];
            const float2 z = cs[low ? at : at - a.half];
            f[i] = low ? f[i] * z.x - other * z.y : f[i] * z.x + other * z.y;
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
      __builtin_amdgcn_wave_barrier();
    } else if constexpr (MODE == kPairs) {
      if (w[e].turns && has)
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if (lo / 2 + p < a.half) {
            const float2 z = cs[lo / 2 + p];
            const float u = f[2 * p], v = f[2 * p + 1];
            f[2 * p] = u * z.x - v * z.y;
            f[2 * p + 1] = v * z.x + u * z.y;
          }
    } else if (w[e].turns && two) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 z = cs[lo + i];
        const float u = f[i], v = g[i];
        f[i] = u * z.x - v * z.y;
        g[i] = v * z.x + u * z.y;
      }
    }
    if (!w[e].dst || !has) continue;
    if (w[e].turns) x[e] = narrow<BF16>(f);
    *(u32x4_t*)(w[e].dst + lo) = x[e];
    if (two) {
      if (w[e].turns) y[e] = narrow<BF16>(g);
      *(u32x4_t*)(w[e].dst + lo + a.half) = y[e];
    }
  }
}

template <bool BF16, int MODE>
hipError_t launch(NormRopeArgs a, int units, hipStream_t stream) {
  const int g = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
  void (*kern)(NormRopeArgs) = nullptr;
  switch (g) {
    case 4: kern = norm_rope_kernel<BF16, 4, MODE>; break;
    case 8: kern = norm_rope_kernel<BF16, 8, MODE>; break;
    case 16: kern = norm_rope_kernel<BF16, 16, MODE>; break;
    default: kern = norm_rope_kernel<BF16, 32, MODE>; break;
  }
  const int64_t items = 256 / g * kItems, blocks = (a.T * a.heads + items - 1) / items;
  // tokens that this many heads in a row can touch: at most 40 KB of LDS
  const int64_t tokens = std::min<int64_t>(a.T, items / a.heads + 2);
  const size_t lds = (size_t)tokens * a.half * sizeof(float2);
  constexpr int64_t kMost = 1 << 23;  // workgroups of one launch: its threads stay below 2^32
  for (a.block0 = 0; a.block0 < blocks; a.block0 += kMost) {
    hipLaunchKernelGGL(kern, dim3((unsigned)std::min(kMost, blocks - a.block0)), dim3(256), lds, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeProblem& n, hipStream_t stream) {
  const RopeProblem& p = n.rope;
  NormRopeArgs a{};
  a.q = (const uint16_t*)p.q; a.k = (const uint16_t*)p.k; a.v = (const uint16_t*)p.v;
  a.qo = (uint16_t*)p.qo; a.ko = (uint16_t*)p.ko; a.vo = (uint16_t*)p.vo;
  a.positions = p.positions; a.slots = p.slots; a.inv_freq = p.inv_freq; a.axis_of = n.axis_of;
  a.q_weight = n.q_weight; a.k_weight = n.k_weight; a.q_weight32 = n.q_weight32; a.k_weight32 = n.k_weight32;
  a.q_t = p.q_t; a.q_h = p.q_h; a.k_t = p.k_t; a.k_h = p.k_h; a.v_t = p.v_t; a.v_h = p.v_h;
  a.qo_t = p.qo_t; a.qo_h = p.qo_h; a.ko_t = p.ko_t; a.ko_h = p.ko_h; a.vo_t = p.vo_t; a.vo_h = p.vo_h;
  a.T = p.T; a.S = p.S; a.hq = p.hq; a.hkv = p.hkv; a.half = p.half; a.d = p.d; a.axes = n.axes;
  a.heads = p.hq + p.hkv + (p.v ? p.hkv : 0);
  a.factor = p.factor; a.eps = n.eps; a.inv_d = 1.f / (float)p.d;
  a.by_heads = fast_div((uint32_t)a.heads); a.by_half = fast_div((uint32_t)p.half);
  a.turn_units = p.half / 8;
  a.head_units = a.turn_units + (p.d - 2 * p.half) / 8;
  const bool bf16 = p.act == WQ_BF16;
  if (p.interleaved)
    return bf16 ? launch<true, kPairs>(a, p.d / 8, stream) : launch<false, kPairs>(a, p.d / 8, stream);
  if (p.half % 8 == 0)
    return bf16 ? launch<true, kHalf>(a, a.head_units, stream) : launch<false, kHalf>(a, a.head_units, stream);
  return bf16 ? launch<true, kOdd>(a, p.d / 8, stream) : launch<false, kOdd>(a, p.d / 8, stream);
}

}  // namespace wq
