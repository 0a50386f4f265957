// mxfp4.h -- device helpers of the 4-bit microscaled format (MXFP4).
//
// A row of K values (K a multiple of 32) is K/2 code bytes and K/32 scale
// bytes.  Code of element k: byte k/2, low half for even k; bit 3 is the sign,
// bits 2..0 one of the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Scale byte s of
// 32 consecutive values is worth 2^(s - 127); s = 255 makes its block NaN.
#pragma once

#include "common.h"
#include "launch.h"

namespace int8w {

constexpr uint32_t kMxBlock = 32;  // values a scale

// A scale byte as the f32 operand of the fp4 converters, which take its
// exponent field alone (byte 0 so stands for 2^-127 there as well, and 255
// gives NaN): checked on all 256 bytes times 16 codes.
__device__ __forceinline__ float mx_scale_f32(uint32_t s) { return __uint_as_float(s << 23); }

// Eight codes (one dword, element 0 in the low half of byte 0) -> eight BF16
// values with the scale applied.  Exact below 2^128, since a magnitude has two significant
// bits; at and above it (scale byte 253 with magnitudes 4 and 6, 254 with 2 and up), where
// fp32 ends too, infinity.
__device__ __forceinline__ uint4 mx_to_bf16x8(uint32_t q, float s) {
  const bf16x2 a = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
  const bf16x2 b = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
  const bf16x2 c = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
  const bf16x2 d = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  return make_uint4(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                    __builtin_bit_cast(uint32_t, d));
}

}  // namespace int8w
