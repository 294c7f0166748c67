// gmm_mx.hpp -- conversions of microscaled fp4 values on gfx950.
#pragma once

#include "gmm_device.hpp"

namespace gmmk {

// The binary32 whose exponent field is an E8M0 scale byte, as the scaled
// conversions take it (they read the exponent alone: byte 0 is 2^-127).
__device__ __forceinline__ float e8m0_operand(int byte) { return __int_as_float(byte << 23); }

// 8 fp4 e2m1 values (as nib8_to_bf16x8) times 2^(byte - 127): exact in bf16
// (subnormals included) up to byte 252, infinities where a product passes
// the largest bf16, NaN for byte 255 (checked for every byte and code).
__device__ __forceinline__ i32x4 fp4x8_scaled_bf16(unsigned w, int byte) {
  const float s = e8m0_operand(byte);
  i32x4 r;
  r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return r;
}

}  // namespace gmmk
