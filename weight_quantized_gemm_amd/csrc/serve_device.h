// Device-side helpers of the serving operators, on top of wq_device.h: 16x16 matrix
// instructions, packed rounding, 16-bit transpose reads and 64-bit direct-to-LDS loads.
#pragma once
#include "serve_problem.h"
#include "wq_device.h"

namespace wq {

// Raise a kernel's dynamic LDS limit; done once per (kernel, device, size) in a process.
hipError_t raise_lds_limit(const void* kernel, int bytes);

// D (16 x 16) += A (16 x 32) B (32 x 16).  Lane l holds row (A) or column (B) l % 16 at
// contraction indices 8 (l / 16) .. + 7; element i of D is row 4 (l / 16) + i, column l % 16.
template <bool BF16>
__device__ __forceinline__ f32x4_t mfma16x16x32(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                  0, 0, 0);
}

// Two fp32 values rounded to nearest even, the first in bits 0-15.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
  else return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});
}

// x / d for 0 <= x < 2^31
__device__ __forceinline__ uint32_t divide(uint32_t x, const FastDiv& f) {
  return f.d == 1 ? x : __umulhi(x, f.mul) >> f.shift;
}

// gfx950 16-bit transpose read: within each group of 16 lanes, element j of lane L is element
// L % 4 of the 8 bytes addressed by lane 4 j + L / 4.  Lanes addressing (row j = L / 4, 4 columns
// from 4 (L % 4)) of a row-major tile give every lane one column and 4 consecutive rows.
__device__ __forceinline__ u32x2_t lds_read_tr16(const uint8_t* p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((WQ_LDS i16x4_t*)(p)));
}

// The LDS address of a pointer into it, as direct-to-LDS loads take it (for offsets to be added to).
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(WQ_LDS const void*)p; }

// One 16-byte-per-lane direct-to-LDS load from 64-bit addresses (a cache passes 4 GiB): lane
// l's 16 bytes land at LDS address lds + 16 * l.  Self-contained like dma16 (wq_device.h); the caller
// counts it in its vmcnt waits.
__device__ __forceinline__ void dma16_global(const void* src, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %2, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"((uint32_t)__builtin_amdgcn_readfirstlane((int)lds)), "v"((uint64_t)src)
      : "memory");
}

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)v) | ((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32));
}

}  // namespace wq
