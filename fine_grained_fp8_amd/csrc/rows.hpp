// Device helpers of the kernels that own a row of values in the lanes of a wave:
// sums over lanes, 1 / sqrt, BF16 packing.
#pragma once

#include "device.hpp"

namespace fp8bs {

// two FP32 values to packed BF16 in one instruction
__device__ __forceinline__ int bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(int, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xF, 0xF, true));
}
// Sum over each run of n consecutive lanes (n a power of two up to 64), in
// every lane, on the vector unit alone.
template <int n>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (n >= 2) v = add_dpp<0xB1>(v);     // quad_perm 1,0,3,2
  if constexpr (n >= 4) v = add_dpp<0x4E>(v);     // quad_perm 2,3,0,1
  if constexpr (n >= 8) v = add_dpp<0x141>(v);    // row_half_mirror
  if constexpr (n >= 16) v = add_dpp<0x140>(v);   // row_mirror
  if constexpr (n >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (n >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// 1 / sqrt(v): the hardware estimate and one Newton step (within 2 ulp), or
// the plain operations where the estimate's step has no finite result.
__device__ __forceinline__ float rsqrt_refined(float v) {
  if (!(v > 1e-30f && v < 1e30f)) return 1.0f / sqrtf(v);
  const float r = __builtin_amdgcn_rsqf(v);
  const float e = __builtin_fmaf(-v * r, r, 1.0f);
  return __builtin_fmaf(0.5f * e, r, r);
}

}  // namespace fp8bs
