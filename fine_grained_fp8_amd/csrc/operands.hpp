// E4M3 operand blocks in a lane's registers, and their exact products (codes as BF16,
// FP32 sums), for the kernels that take a few tokens.
#pragma once

#include "device.hpp"

namespace fp8bs {

// 8 E4M3 codes (two dwords) as BF16, exactly
__device__ __forceinline__ v8bf codes_to_bf16(int lo, int hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One 128-wide K block of a 16-row operand: a lane's 32 codes (bytes 16 g.. and
// 64 + 16 g.. of the block for lane group g), as the framework's tiles and
// its FP8 MFMA order them.
struct Block {
  int __attribute__((ext_vector_type(4))) lo, hi;
};
struct Bf16Block {
  v8bf f[4];
};
__device__ __forceinline__ Bf16Block to_bf16(const Block& b) {
  return Bf16Block{{codes_to_bf16(b.lo[0], b.lo[1]), codes_to_bf16(b.lo[2], b.lo[3]),
                    codes_to_bf16(b.hi[0], b.hi[1]), codes_to_bf16(b.hi[2], b.hi[3])}};
}
// partial sums of one K block with exact products and FP32 additions
__device__ __forceinline__ v4f block_product(const Bf16Block& a, const Bf16Block& b) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma_bf16_16x16x32(a.f[i], b.f[i], c);
  return c;
}

}  // namespace fp8bs
