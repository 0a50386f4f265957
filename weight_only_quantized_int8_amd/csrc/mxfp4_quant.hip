// mxfp4_quant.hip -- BF16 or f32 values -> MXFP4 codes and scales, and MXFP4 ->
// BF16 values (format: mxfp4.h).
//
// Per block of 32 values with largest magnitude a:
//   s = max(E(a) - 2, 0), E the 8-bit exponent field of a in f32 (so s - 127 =
//   floor(log2 a) - 2 for normal a, and 0 where the block is zero or below
//   2^-124); the largest value then lies below 8 and is rounded to at most 6;
//   code = v / 2^(s-127) to the nearest code, ties to the even one, magnitudes
//   above 6 to 6, the sign kept (also of a zero).
//   A block with an infinity or NaN gets s = 255 and codes 0: it reads as NaN.
// v / 2^(s-127) is exact and the hardware converter rounds it once to the
// nearest even code and saturates, so the codes are the definition's.
//
// Both kernels are HBM-bound: values and codes are flat streams (K % 32 == 0,
// so no block crosses a row).  A lane takes 8 consecutive values, the 4 lanes
// of a block meet in two quad-permute maxima of the magnitude bits, and a wave
// has four such items in flight.  14336x4096 in BF16, 149 MB either way: quantize
// 25.0 us (6.0 TB/s), dequantize 22.4 us (6.6 TB/s).
#include "launch.h"
#include "mxfp4.h"

namespace int8w {

namespace {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // lane ^ 1
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // lane ^ 2
  return v > o ? v : o;
}

template <bool F32>
struct Values8 {
  u32x4 v[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ uint32_t exponent8(const Values8<F32> &x) {  // exponent field of the largest magnitude
  if constexpr (F32) {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = x.v[h][i] & 0x7FFFFFFFu;
        m = m > a ? m : a;
      }
    return quad_max(m) >> 23;
  } else {
    u16x2 m = __builtin_bit_cast(u16x2, x.v[0][0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x.v[0][i] & 0x7FFF7FFFu));
    return quad_max(m.x > m.y ? m.x : m.y) >> 7;
  }
}

template <bool F32>
__device__ __forceinline__ uint32_t codes8(const Values8<F32> &x, float s) {
  uint32_t q = 0;
  if constexpr (F32) {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(x.v[0][0]), __uint_as_float(x.v[0][1]), s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(x.v[0][2]), __uint_as_float(x.v[0][3]), s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(x.v[1][0]), __uint_as_float(x.v[1][1]), s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(x.v[1][2]), __uint_as_float(x.v[1][3]), s, 3);
  } else {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][0]), s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][1]), s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][2]), s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][3]), s, 3);
  }
  return q;
}

constexpr int kItems = 4;  // items of 8 values a lane has in flight

// items: whole groups of 8 values; a workgroup takes 256 * kItems of them.
template <bool F32>
__global__ __launch_bounds__(256) void k_mx_quantize(const u32x4 *__restrict__ x, uint64_t items,
                                                     uint32_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const uint64_t first = (uint64_t)blockIdx.x * (256u * kItems) + threadIdx.x;
  Values8<F32> v[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const uint64_t i = first + 256u * j;
    if (i < items) {
      if constexpr (F32) {
        v[j].v[0] = __builtin_nontemporal_load(x + 2 * i);
        v[j].v[1] = __builtin_nontemporal_load(x + 2 * i + 1);
      } else {
        v[j].v[0] = __builtin_nontemporal_load(x + i);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const uint64_t i = first + 256u * j;
    if (i < items) {  // the four lanes of a block agree: items come in fours
      const uint32_t e = exponent8<F32>(v[j]);
      const bool bad = e == 255u;
      const uint32_t s = bad ? 255u : e > 2u ? e - 2u : 0u;
      const uint32_t q = codes8<F32>(v[j], mx_scale_f32(bad ? 127u : s));
      codes[i] = bad ? 0u : q;
      if ((i & 3u) == 0) scales[i >> 2] = (uint8_t)s;
    }
  }
}

__global__ __launch_bounds__(256) void k_mx_dequantize(const uint32_t *__restrict__ codes,
                                                       const uint8_t *__restrict__ scales, uint64_t items,
                                                       uint4 *__restrict__ out) {
  const uint64_t first = (uint64_t)blockIdx.x * (256u * kItems) + threadIdx.x;
  uint32_t q[kItems], s[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const uint64_t i = first + 256u * j;
    if (i < items) {
      q[j] = __builtin_nontemporal_load(codes + i);
      s[j] = scales[i >> 2];
    }
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const uint64_t i = first + 256u * j;
    if (i < items) store_nt(mx_to_bf16x8(q[j], mx_scale_f32(s[j])), out + i);
  }
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, bool f32, uint32_t rows, uint32_t K, uint8_t *codes, uint8_t *scales,
                              hipStream_t stream) {
  const uint64_t items = (uint64_t)rows * K / 8u;
  const uint32_t grid = (uint32_t)((items + 256u * kItems - 1) / (256u * kItems));
  if (f32)
    k_mx_quantize<true><<<grid, 256, 0, stream>>>((const u32x4 *)x, items, (uint32_t *)codes, scales);
  else
    k_mx_quantize<false><<<grid, 256, 0, stream>>>((const u32x4 *)x, items, (uint32_t *)codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxView &w, uint16_t *out, hipStream_t stream) {
  const uint64_t items = (uint64_t)w.N * w.K / 8u;
  const uint32_t grid = (uint32_t)((items + 256u * kItems - 1) / (256u * kItems));
  k_mx_dequantize<<<grid, 256, 0, stream>>>((const uint32_t *)w.codes, w.scales, items, (uint4 *)out);
  return hipGetLastError();
}

}  // namespace int8w
