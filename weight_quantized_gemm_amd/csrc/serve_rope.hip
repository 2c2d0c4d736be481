// Rotary positions of q and k, with k and v written to rows of a cache:
//
//   (u, v) -> factor * (u cos w - v sin w, v cos w + u sin w),   w = position * inv_freq[j]
//
// Bound by memory: every element is read and written once.  A unit is what one thread moves:
// 16 bytes of a head's first half and 16 of its second (half layout), 16 bytes of adjacent
// pairs (interleaved), or 16 bytes that are only copied (v, and a head's tail past the rotated
// part).  The units of all tokens form one row, token by token; a workgroup takes 512 of
// them, two a thread, whether they are a part of one token or many tokens.  Both loads are
// issued before the angles are ready, so that their latency covers the angles' arithmetic.
//
// The workgroup computes the cosines and sines of its tokens once, in LDS, for all heads.  An
// angle is a product of up to 2^31 and a frequency; fp32 would lose it (at position 131071 an
// ulp is 1/128 radian), so the product is taken in fp64 in turns, reduced to half a turn
// there, and only the remainder is fp32.
//
// Measured (MI355X): 16384 tokens, 32 + 8 + 8 heads of 128, bf16: 76.2 us for 403 MB, 5.28 TB/s, the rate of
// a large copy; 509 tokens (25 MB): 6.6 us, 3.8 TB/s; 4 tokens: 5.2 us, of which the kernel takes 3.2
// and the rest is the launch.  Where the rotated part is not whole 16-byte units, a unit is a pair of 2-byte
// elements: 378 us for the same tokens with 20 elements rotated, 1.07 TB/s.
#include <algorithm>

#include "serve_device.h"
#include "serve_kernels.h"

namespace wq {
namespace {

constexpr int kUnits = 512;  // units of a workgroup
constexpr double kInvTwoPi = 0.15915494309189533577;

struct RopeArgs {
  const uint16_t *q, *k, *v;
  uint16_t *qo, *ko, *vo;
  const int32_t *positions, *slots;
  const float* inv_freq;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, qo_t, qo_h, ko_t, ko_h, vo_t, vo_h;
  int64_t T, S;
  int64_t block0;                  // the launch's first workgroup among all of the call's
  int32_t hq, hkv, half;
  int32_t turn_units, head_units;  // units of a head: rotated ones, all of them
  int32_t units;                   // units of a token
  int32_t copy_units;              // units of a v head
  FastDiv by_units, by_head, by_copy, by_half;
  float factor;
};

// What a unit works on.  lo: its first element, within a head; pair: its first pair, if it turns
// (otherwise it is copied).
struct Unit {
  const uint16_t* src = nullptr;
  uint16_t* dst = nullptr;  // null: no unit, or a token whose slot drops it
  int token = 0;            // of the workgroup
  int lo = 0, pair = 0;
  bool turn = false;
};

// VEC: a unit is 8 elements (half layout: twice 8), which the rotated part divides into;
// otherwise it is one pair (or one copied element).
template <bool VEC, bool INTER>
__device__ __forceinline__ Unit find_unit(const RopeArgs& a, int64_t t0, int u0, int i, int64_t last) {
  Unit w;
  const int64_t all = t0 * a.units + u0 + i;
  if (all >= last) return w;
  const uint32_t x = (uint32_t)(u0 + i);
  w.token = (int)divide(x, a.by_units);
  int u = (int)(x - (uint32_t)w.token * (uint32_t)a.units);
  const int64_t t = t0 + w.token;
  const int rotated = (a.hq + a.hkv) * a.head_units;
  if (u < rotated) {
    const int h = (int)divide((uint32_t)u, a.by_head);
    u -= h * a.head_units;
    w.turn = u < a.turn_units;
    const int rest = 2 * a.half + (VEC ? 8 : 1) * (u - a.turn_units);
    if (w.turn) {
      w.lo = VEC ? 8 * u : INTER ? 2 * u : u;
      w.pair = INTER ? w.lo / 2 : w.lo;
    } else {
      w.lo = rest;
    }
    if (h < a.hq) {
      w.src = a.q + t * a.q_t + h * a.q_h;
      w.dst = a.qo + t * a.qo_t + h * a.qo_h;
    } else {
      const int64_t row = a.slots ? a.slots[t] : t;
      w.src = a.k + t * a.k_t + (h - a.hq) * a.k_h;
      if (row >= 0 && row < a.S) w.dst = a.ko + row * a.ko_t + (h - a.hq) * a.ko_h;
    }
  } else {
    u -= rotated;
    const int h = (int)divide((uint32_t)u, a.by_copy);
    const int64_t row = a.slots ? a.slots[t] : t;
    w.lo = (VEC ? 8 : 1) * (u - h * a.copy_units);
    w.src = a.v + t * a.v_t + h * a.v_h;
    if (row >= 0 && row < a.S) w.dst = a.vo + row * a.vo_t + h * a.vo_h;
  }
  return w;
}

template <bool BF16, bool VEC, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs a) {
  extern __shared__ float2 turns[];  // (cos, sin) of each token of the workgroup and each pair
  const int tid = threadIdx.x;
  const int64_t first = (a.block0 + blockIdx.x) * kUnits, last = a.T * a.units;
  const int64_t t0 = first / a.units;
  const int u0 = (int)(first - t0 * a.units);
  const int tokens = (int)((min(first + kUnits, last) - 1) / a.units - t0) + 1;

  Unit w[2];
  u32x4_t x[2], y[2];
  uint16_t xs[2] = {0, 0}, ys[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    w[e] = find_unit<VEC, INTER>(a, t0, u0, tid + 256 * e, last);
    if (!w[e].dst) continue;
    if constexpr (VEC) {
      x[e] = *(const u32x4_t*)(w[e].src + w[e].lo);
      if (!INTER && w[e].turn) y[e] = *(const u32x4_t*)(w[e].src + w[e].lo + a.half);
    } else {
      xs[e] = w[e].src[w[e].lo];
      if (w[e].turn) ys[e] = w[e].src[w[e].lo + (INTER ? 1 : a.half)];
    }
  }

  for (int i = tid; i < tokens * a.half; i += 256) {
    const int tk = (int)divide((uint32_t)i, a.by_half), j = i - tk * a.half;
    const double turn = (double)a.positions[t0 + tk] * (double)a.inv_freq[j] * kInvTwoPi;
    float s, c;
    sincospif(2.f * (float)(turn - rint(turn)), &s, &c);
    turns[i] = make_float2(a.factor * c, a.factor * s);
  }
  __syncthreads();

#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!w[e].dst) continue;
    const float2* cs = turns + w[e].token * a.half + w[e].pair;
    if constexpr (!VEC) {
      uint16_t o = xs[e];
      if (w[e].turn) {
        const float u = act_to_f32<BF16>(xs[e]), v = act_to_f32<BF16>(ys[e]);
        o = f32_to_act<BF16>(u * cs[0].x - v * cs[0].y);
        w[e].dst[w[e].lo + (INTER ? 1 : a.half)] = f32_to_act<BF16>(v * cs[0].x + u * cs[0].y);
      }
      w[e].dst[w[e].lo] = o;
    } else if (!w[e].turn) {
      *(u32x4_t*)(w[e].dst + w[e].lo) = x[e];
    } else if constexpr (INTER) {
      u32x4_t o;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float u = act_to_f32<BF16>((uint16_t)x[e][p]), v = act_to_f32<BF16>((uint16_t)(x[e][p] >> 16));
        o[p] = pack2<BF16>(u * cs[p].x - v * cs[p].y, v * cs[p].x + u * cs[p].y);
      }
      *(u32x4_t*)(w[e].dst + w[e].lo) = o;
    } else {
      u32x4_t o, r;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float u0f = act_to_f32<BF16>((uint16_t)x[e][p]), v0f = act_to_f32<BF16>((uint16_t)y[e][p]);
        const float u1f = act_to_f32<BF16>((uint16_t)(x[e][p] >> 16)), v1f = act_to_f32<BF16>((uint16_t)(y[e][p] >> 16));
        const float2 c0 = cs[2 * p], c1 = cs[2 * p + 1];
        o[p] = pack2<BF16>(u0f * c0.x - v0f * c0.y, u1f * c1.x - v1f * c1.y);
        r[p] = pack2<BF16>(v0f * c0.x + u0f * c0.y, v1f * c1.x + u1f * c1.y);
      }
      *(u32x4_t*)(w[e].dst + w[e].lo) = o;
      *(u32x4_t*)(w[e].dst + w[e].lo + a.half) = r;
    }
  }
}

template <bool BF16, bool VEC>
hipError_t launch(RopeArgs a, bool interleaved, hipStream_t stream) {
  const int64_t blocks = (a.T * a.units + kUnits - 1) / kUnits;
  // tokens that 512 units in a row can touch; a token has at least half / 8 units, so this is
  // at most 34 KB
  const int64_t tokens = std::min<int64_t>(a.T, kUnits / a.units + 2);
  const size_t lds = (size_t)tokens * a.half * sizeof(float2);
  auto kern = interleaved ? rope_kernel<BF16, VEC, true> : rope_kernel<BF16, VEC, false>;
  constexpr int64_t kMost = 1 << 23;  // workgroups of one launch: its threads stay below 2^32
  for (a.block0 = 0; a.block0 < blocks; a.block0 += kMost) {
    hipLaunchKernelGGL(kern, dim3((unsigned)std::min(kMost, blocks - a.block0)), dim3(256), lds, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const RopeProblem& p, hipStream_t stream) {
  RopeArgs a{};
  a.q = (const uint16_t*)p.q; a.k = (const uint16_t*)p.k; a.v = (const uint16_t*)p.v;
  a.qo = (uint16_t*)p.qo; a.ko = (uint16_t*)p.ko; a.vo = (uint16_t*)p.vo;
  a.positions = p.positions; a.slots = p.slots; a.inv_freq = p.inv_freq;
  a.q_t = p.q_t; a.q_h = p.q_h; a.k_t = p.k_t; a.k_h = p.k_h; a.v_t = p.v_t; a.v_h = p.v_h;
  a.qo_t = p.qo_t; a.qo_h = p.qo_h; a.ko_t = p.ko_t; a.ko_h = p.ko_h; a.vo_t = p.vo_t; a.vo_h = p.vo_h;
  a.T = p.T; a.S = p.S; a.hq = p.hq; a.hkv = p.hkv; a.half = p.half; a.factor = p.factor;
  // 16-byte units where the rotated part is whole units: half layout, both halves start on one
  // and hold whole ones; interleaved, the rotated part ends on one.  Otherwise single pairs.
  const bool vec = p.interleaved ? p.half % 4 == 0 : p.half % 8 == 0;
  if (vec) {
    a.turn_units = p.interleaved ? p.half / 4 : p.half / 8;
    a.head_units = a.turn_units + (p.d - 2 * p.half) / 8;
    a.copy_units = p.d / 8;
  } else {
    a.turn_units = p.half;
    a.head_units = p.half + (p.d - 2 * p.half);
    a.copy_units = p.d;
  }
  a.units = (a.hq + a.hkv) * a.head_units + (p.v ? a.hkv * a.copy_units : 0);
  a.by_units = fast_div((uint32_t)a.units);
  a.by_head = fast_div((uint32_t)a.head_units);
  a.by_copy = fast_div((uint32_t)a.copy_units);
  a.by_half = fast_div((uint32_t)a.half);
  const bool bf16 = p.act == WQ_BF16;
  if (vec) return bf16 ? launch<true, true>(a, p.interleaved, stream) : launch<false, true>(a, p.interleaved, stream);
  return bf16 ? launch<true, false>(a, p.interleaved, stream) : launch<false, false>(a, p.interleaved, stream);
}

}  // namespace wq
