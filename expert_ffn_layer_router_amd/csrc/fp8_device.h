// Device code shared by the products of e4m3 codes.
#pragma once

#include "fp8.h"
#include "product_core.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 x 16 of A (lane l: row l % 16, 32 values of the contraction that depend
// on l / 16) times B (the same values of its columns), from zero: D holds
// column l % 16, rows 4 (l / 16) + i.  Which 32 values a lane holds does not
// matter as long as A's and B's agree: the block of 128 has one scale.
__device__ __forceinline__ f32x4 block_product(i32x8 a, i32x8 b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8 join_halves(u32x4 lo, u32x4 hi) {
  return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ float load_scale(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, voff, 0, 0));
}
// Descriptor of `count` scales from `base`; what lies past them reads as 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scales_at(const float* base, int count) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(base), 0, count * 4, 0x00020000);
}

}  // namespace moe
