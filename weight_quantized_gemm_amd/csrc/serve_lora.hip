// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = x3[t] + scale[i] * ((x1[t] @ A_i^T) @ B_i^T),   i = indices[t]
//
// Two kernels, h = x1 @ A_i^T (fp32, k split over workgroups) and out = x3 + h @ B_i^T.
//
// Tokens of one adapter need not stand together, and nothing is sorted: the token rows are
// cut into windows of 16 or 64, and a work item is one (window, distinct adapter of it)
// pair.  Every wave finds the window's distinct adapters with one load of 64 indices and
// ballots; the item's product is taken for whole 16-row blocks of the window and only the
// rows of its adapter are stored, so a row never depends on its neighbours.  A sort would
// read an adapter once for all its tokens where the pairs read it once per window, but costs
// a dependent launch; adapters are a few hundred KB and stay in the L2s.
#include <algorithm>

#include "serve_device.h"
#include "serve_kernels.h"
#include "serve_tile.h"

namespace wq {
namespace {

struct LoraArgs {
  const uint16_t* x1;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* indices;
  const float* scale;
  const int32_t* ranks;
  const uint16_t* x3;
  uint16_t* out;
  float* h;               // [splits][m][r]
  int64_t m, n, sx, s3, so;
  int32_t k, r, L, splits, kchunk, slots;
};

// The adapter of this lane's row of the window at w0 (rows past m and lanes past the window:
// -2, no row; a row without adapter: -1).
template <int W>
__device__ __forceinline__ int lane_key(const LoraArgs& p, int64_t w0, int lane) {
  if (lane >= W || w0 + lane >= p.m) return -2;
  const int i = p.indices[w0 + lane];
  return (uint32_t)i < (uint32_t)p.L ? i : -1;
}

__device__ __forceinline__ int adapter_rank(const LoraArgs& p, int i) {
  return p.ranks ? min(max(p.ranks[i], 0), p.r) : p.r;
}

// ------------------------------------------------------------------------------- h = x1 A^T
// One item's h for up to kLoraRankTiles 16-rank tiles from rank r0 and the workgroup's k
// chunk.  MT 16-row blocks from row w0 + 16 * m0.  The four waves take 64-k steps in turn
// (two 16x16x32 MFMAs: rows of x1 against rows of A_i, both k-contiguous, 16 bytes a lane
// straight from global memory) and their sums meet in LDS, in wave order.
template <bool BF16, int MT>
__device__ __forceinline__ void shrink_item(const LoraArgs& p, float* red, int64_t w0, int m0, int key, uint64_t rows,
                                            int r0, int kb, int ke, float* h) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int nt = min(kLoraRankTiles, (p.r - r0 + 15) / 16);
  const uint16_t* xr[MT];
  const uint16_t* ar[kLoraRankTiles];
#pragma unroll
  for (int t = 0; t < MT; ++t) xr[t] = p.x1 + min(w0 + 16 * (m0 + t) + l16, p.m - 1) * p.sx + 8 * g;
#pragma unroll
  for (int j = 0; j < kLoraRankTiles; ++j)
    ar[j] = p.a + ((int64_t)key * p.r + min(r0 + 16 * j + l16, p.r - 1)) * p.k + 8 * g;
  f32x4_t acc[MT][kLoraRankTiles];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < kLoraRankTiles; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  int k0 = kb + 64 * wave;
#pragma unroll 2
  for (; k0 + 64 <= ke; k0 += 256) {
    u32x4_t xf[MT][2], af[kLoraRankTiles][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int t = 0; t < MT; ++t) xf[t][s] = *(const u32x4_t*)(xr[t] + k0 + 32 * s);
#pragma unroll
      for (int j = 0; j < kLoraRankTiles; ++j)
        if (j < nt) af[j][s] = *(const u32x4_t*)(ar[j] + k0 + 32 * s);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < kLoraRankTiles; ++j)
        if (j < nt)
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[t][j] = mfma16x16x32<BF16>(xf[t][s], af[j][s], acc[t][j]);
  }
  if (k0 < ke) {  // the k tail: 8-k pieces past ke are zeros on both sides
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool in = k0 + 32 * s + 8 * g < ke;
      u32x4_t xf[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) xf[t] = in ? *(const u32x4_t*)(xr[t] + k0 + 32 * s) : u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kLoraRankTiles; ++j)
        if (j < nt) {
          const u32x4_t af = in ? *(const u32x4_t*)(ar[j] + k0 + 32 * s) : u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[t][j] = mfma16x16x32<BF16>(xf[t], af, acc[t][j]);
        }
    }
  }
  // block t of row blocks: element i of a lane is row 4 g + i, rank l16
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kLoraRankTiles; ++j)
      if (j < nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[(wave * 16 + 4 * g + i) * (16 * kLoraRankTiles) + 16 * j + l16] = acc[t][j][i];
    __syncthreads();
    const int c = tid & 63;
    if (c < 16 * nt && r0 + c < p.r) {
      for (int row = tid >> 6; row < 16; row += 4) {
        const int wr = 16 * (m0 + t) + row;
        if (!((rows >> wr) & 1)) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) v += red[(w * 16 + row) * (16 * kLoraRankTiles) + c];
        h[(w0 + wr) * p.r + r0 + c] = v;
      }
    }
  }
}

// Grid x: windows, y: slots x blocks of kLoraRankTiles rank tiles, z: k splits.
template <bool BF16, int W>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const LoraArgs p) {
  __shared__ float red[4 * 16 * 16 * kLoraRankTiles];
  const int lane = threadIdx.x & 63;
  const int64_t w0 = (int64_t)blockIdx.x * W;
  const int slot = blockIdx.y % p.slots, r0 = (blockIdx.y / p.slots) * 16 * kLoraRankTiles;
  const int kb = blockIdx.z * p.kchunk, ke = min(p.k, kb + p.kchunk);
  float* h = p.h + (int64_t)blockIdx.z * p.m * p.r;
  const int mine = lane_key<W>(p, w0, lane);
  uint64_t left = __ballot(mine >= 0);
  for (int s = 0; left; ++s) {
    const int key = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t rows = __ballot(mine == key);
    left &= ~rows;
    if (s % p.slots != slot || r0 >= adapter_rank(p, key)) continue;
    if constexpr (W == 16) {
      shrink_item<BF16, 1>(p, red, w0, 0, key, rows, r0, kb, ke, h);
    } else {
      // rows inside one 16-row block (single tokens, the ends of prompts) read that block only
      const int lo = __builtin_ctzll(rows) >> 4, hi = (63 - __builtin_clzll(rows)) >> 4;
      if (lo == hi) shrink_item<BF16, 1>(p, red, w0, lo, key, rows, r0, kb, ke, h);
      else shrink_item<BF16, 4>(p, red, w0, 0, key, rows, r0, kb, ke, h);
    }
  }
}

// ------------------------------------------------------------------------- out = x3 + h B^T
// Both factors of this product are 16-bit in the matrix cores, but h is fp32: it is taken as
// the sum of two 16-bit numbers, hi + lo, which keep 16 (bf16) or 22 (fp16) of its bits.  A
// row is first scaled by a power of two to a largest magnitude in [1, 2), so that fp16 can
// hold it; the power comes back in fp32 at the end.  The contraction of one 16x16x32 MFMA
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

// Grid x: windows, y: blocks of NC * 4 columns (NC per wave), z: slots.  Dynamic LDS: W rows of
// hp = (r rounded up to 16) + 4 packed values, then W row factors.
template <bool BF16, int W, int NC>
__global__ __launch_bounds__(256) void lora_expand_kernel(const LoraArgs p) {
  extern __shared__ uint32_t lds[];
  constexpr int MT = W / 16, NP = NC / 32;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t w0 = (int64_t)blockIdx.x * W;
  const int64_t n0 = (int64_t)blockIdx.y * (4 * NC) + wave * NC;
  const int r16 = (p.r + 15) & ~15, hp = r16 + 4;
  float* factor = (float*)(lds + W * hp);
  const int mine = lane_key<W>(p, w0, lane);
  uint64_t left = __ballot(mine >= -1);
  for (int s = 0; left; ++s) {
    const int key = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t rows = __ballot(mine == key);
    left &= ~rows;
    if (s % p.slots != (int)blockIdx.z) continue;
    const int rank = key < 0 ? 0 : adapter_rank(p, key);
    const int nk = (rank + 15) / 16;
    if (rank == 0 && p.x3 == p.out) continue;  // nothing to add in place

    if (rank) {  // h of the adapter's rows: splits added in order, scaled, split into hi + lo
      __syncthreads();
      constexpr int TPR = 256 / W;  // threads of a row
      const int row = tid / TPR, c0 = tid % TPR;
      const bool have = (rows >> row) & 1;
      const float sc = p.scale ? p.scale[key] : 1.f;
      float big = 0.f;
      for (int c = c0; c < 16 * nk; c += TPR) {
        float v = 0.f;
        if (have && c < rank) {
          const float* hr = p.h + (w0 + row) * p.r + c;
          for (int z = 0; z < p.splits; ++z) v += hr[(int64_t)z * p.m * p.r];
          v *= sc;
        }
        if (__builtin_isfinite(v)) big = fmaxf(big, fabsf(v));  // infinities and NaN stay what they are
        lds[row * hp + c] = __float_as_uint(v);
      }
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) big = fmaxf(big, __shfl_xor(big, o, 64));
      // 2^-e: exponent of the largest magnitude, kept where 2^-e and 2^e are normal numbers
      int e = big > 0.f ? (int)(__float_as_uint(big) >> 23) - 127 : 0;
      e = min(max(e, -126), 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      if (c0 == 0) factor[row] = __uint_as_float((uint32_t)(127 + e) << 23);
      for (int c = c0; c < 16 * nk; c += TPR)
        lds[row * hp + c] = split_hi_lo<BF16>(__uint_as_float(lds[row * hp + c]) * down);
      __syncthreads();
    }

    f32x4_t acc[NP][2][MT];
#pragma unroll
    for (int q = 0; q < NP; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[q][e][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const uint16_t* bk = p.b + (int64_t)max(key, 0) * p.n * p.r;
    for (int j = 0; j < nk; ++j) {
      const int c = 16 * j + 8 * (g & 1);  // this lane's 8 ranks
      u32x4_t hf[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const u32x4_t* src = (const u32x4_t*)(lds + (16 * t + l16) * hp + c);
        const u32x4_t u = src[0], v = src[1];
        const uint32_t sel = g < 2 ? 0x05040100u : 0x07060302u;  // the hi or the lo halves
        hf[t] = u32x4_t{__builtin_amdgcn_perm(u[1], u[0], sel), __builtin_amdgcn_perm(u[3], u[2], sel),
                        __builtin_amdgcn_perm(v[1], v[0], sel), __builtin_amdgcn_perm(v[3], v[2], sel)};
      }
#pragma unroll
      for (int q = 0; q < NP; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int64_t n = n0 + 32 * q + 8 * (l16 >> 2) + 4 * e + (l16 & 3);
          u32x4_t bf = u32x4_t{0, 0, 0, 0};
          if (n < p.n && c < rank) {
            bf = *(const u32x4_t*)(bk + n * p.r + c);
            if (c + 8 > rank) {  // columns past the rank hold anything
#pragma unroll
              for (int d = 0; d < 4; ++d)
                bf[d] &= (c + 2 * d < rank ? 0x0000ffffu : 0u) | (c + 2 * d + 1 < rank ? 0xffff0000u : 0u);
            }
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[q][e][t] = mfma16x16x32<BF16>(bf, hf[t], acc[q][e][t]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int wr = 16 * t + l16;
      if (!((rows >> wr) & 1)) continue;
      const int64_t row = w0 + wr;
      const float f = rank ? factor[wr] : 0.f;
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const int64_t n = n0 + 32 * q + 8 * g;
        if (n >= p.n) continue;
        u32x4_t x = u32x4_t{0, 0, 0, 0};
        if (p.x3) x = *(const u32x4_t*)(p.x3 + row * p.s3 + n);
        if (rank) {
          u32x4_t o;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const f32x4_t& y = acc[q][d >> 1][t];
            const float lo = act_to_f32<BF16>((uint16_t)x[d]) + f * y[2 * (d & 1)];
            const float hi = act_to_f32<BF16>((uint16_t)(x[d] >> 16)) + f * y[2 * (d & 1) + 1];
            o[d] = pack2<BF16>(lo, hi);
          }
          x = o;
        }
        *(u32x4_t*)(p.out + row * p.so + n) = x;
      }
    }
  }
}

template <bool BF16, int W>
hipError_t launch(const LoraArgs& a, const LoraPlan& pl, hipStream_t stream) {
  const int rank_blocks = (a.r + 16 * kLoraRankTiles - 1) / (16 * kLoraRankTiles);
  hipLaunchKernelGGL((lora_shrink_kernel<BF16, W>),
                     dim3((unsigned)pl.windows, (unsigned)(pl.slots * rank_blocks), (unsigned)pl.splits), dim3(256), 0,
                     stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int NC = W == 16 ? 32 : 64;
  const size_t lds = (size_t)W * (((a.r + 15) & ~15) + 4 + 1) * 4;
  auto kern = lora_expand_kernel<BF16, W, NC>;
  e = raise_lds_limit((const void*)kern, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)pl.windows, (unsigned)((a.n + 4 * NC - 1) / (4 * NC)), (unsigned)pl.slots),
                     dim3(256), lds, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraProblem& p, const LoraPlan& pl, void* workspace, hipStream_t stream) {
  LoraArgs a{};
  a.x1 = (const uint16_t*)p.x1; a.a = (const uint16_t*)p.a; a.b = (const uint16_t*)p.b;
  a.indices = p.indices; a.scale = p.scale; a.ranks = p.ranks;
  a.x3 = (const uint16_t*)p.x3; a.out = (uint16_t*)p.out; a.h = (float*)workspace;
  a.m = p.m; a.n = p.n; a.sx = p.sx; a.s3 = p.s3; a.so = p.so;
  a.k = p.k; a.r = p.r; a.L = (int32_t)p.L; a.splits = pl.splits; a.kchunk = pl.kchunk; a.slots = pl.slots;
  const bool bf16 = p.act == WQ_BF16;
  if (pl.window == 16) return bf16 ? launch<true, 16>(a, pl, stream) : launch<false, 16>(a, pl, stream);
  return bf16 ? launch<true, 64>(a, pl, stream) : launch<false, 64>(a, pl, stream);
}

}  // namespace wq
