// token_stream.h -- weight rows times one activation row on the vector ALUs, shared by
// the MXFP4 product for one row and the mixture-of-experts layer for one token.
//
// A wave takes pairs of weight rows that share an activation row.  A load covers 1 KiB of
// one row (2048 MXFP4 codes or 1024 8-bit codes), a lane's 16 bytes lie in one scale's
// run, and a ring of segments stays in flight across rows.  The matrix-core form
// (rows_stream.h) would compute 16 columns to use one and change lanes through LDS for
// each 64 bytes; here a code costs a fraction of a conversion and of a two-way dot product:
//  * MXFP4: half a v_cvt_scalef32_pk_bf16_fp4 (scale applied, exact below 2^128) and half a v_dot2.
//  * 8-bit affine: codes to BF16 integers (exact), half a v_dot2; the run's
//    s * sum q x + b * sum x once, sum x from LDS.
// The activations sit in LDS as BF16, their 16-byte pieces in planes so that a wave's
// reads are contiguous; a segment's are read once for both rows of a pair.
#pragma once

#include "mxfp4.h"

namespace int8w {

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}

// Sum over the wave in a fixed order, in every lane.
__device__ __forceinline__ float token_sum(float v) {
#define INT8W_DPP_ADD(ctrl, rows) \
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, rows, 0xF, true))
  INT8W_DPP_ADD(0x111, 0xF);  // row_shr:1
  INT8W_DPP_ADD(0x112, 0xF);
  INT8W_DPP_ADD(0x114, 0xF);
  INT8W_DPP_ADD(0x118, 0xF);
  INT8W_DPP_ADD(0x142, 0xA);  // row_bcast:15
  INT8W_DPP_ADD(0x143, 0xC);  // row_bcast:31
#undef INT8W_DPP_ADD
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

struct MxTok {
  typedef MxView View;
  static constexpr uint32_t kSeg = 2048;  // k of a load
  static constexpr uint32_t kX = 4;       // 16-byte pieces of activations a lane
  struct Row {
    __amdgpu_buffer_rsrc_t codes, scales;
  };
  struct Frag {
    u32x4 q;
    uint32_t s;
  };
  static __device__ __forceinline__ Row row(const MxView &w, uint64_t r, bool have) {
    return Row{make_rsrc(w.codes + r * (w.K / 2u), have ? w.K / 2u : 0u), make_rsrc(w.scales + r * (w.K / 32u), have ? w.K / 32u : 0u)};
  }
  // past the row's end the buffer resource gives zeros
  static __device__ __forceinline__ void load(Frag &f, const Row &r, const MxView &, uint32_t seg, uint32_t lane) {
    f.q = buf_load_b128<kAuxNontemporal>(r.codes, 1024u * seg + 16u * lane);
    f.s = __builtin_amdgcn_raw_buffer_load_b8(r.scales, (int)(64u * seg + lane), 0, 0);
  }
  static __device__ __forceinline__ float dot(float acc, const Frag &f, const u32x4 (&x)[kX], float) {
    const float s = mx_scale_f32(f.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 b = mx_to_bf16x8(f.q[i], s);
      acc = dot2(b.x, x[i].x, acc);
      acc = dot2(b.y, x[i].y, acc);
      acc = dot2(b.z, x[i].z, acc);
      acc = dot2(b.w, x[i].w, acc);
    }
    return acc;
  }
  static constexpr bool kSums = false;
};

struct Int8Tok {
  typedef WeightView View;
  static constexpr uint32_t kSeg = 1024;
  static constexpr uint32_t kX = 2;
  struct Row {
    __amdgpu_buffer_rsrc_t codes, scales, biases;
  };
  struct Frag {
    u32x4 q;
    uint16_t s, b;
  };
  static __device__ __forceinline__ Row row(const WeightView &w, uint64_t r, bool have) {
    const uint32_t G = w.K / w.gs;
    return Row{make_rsrc((const uint8_t *)w.packed + r * w.K, have ? w.K : 0u), make_rsrc(w.scales + r * G, have ? 2u * G : 0u),
               make_rsrc(w.biases + r * G, have ? 2u * G : 0u)};
  }
  static __device__ __forceinline__ void load(Frag &f, const Row &r, const WeightView &w, uint32_t seg, uint32_t lane) {
    f.q = buf_load_b128<kAuxNontemporal>(r.codes, 1024u * seg + 16u * lane);
    const uint32_t o = 2u * ((1024u * seg + 16u * lane) >> (31u - (uint32_t)__builtin_clz(w.gs)));
    f.s = buf_load_b16(r.scales, o);
    f.b = buf_load_b16(r.biases, o);
  }
  static __device__ __forceinline__ float dot(float acc, const Frag &f, const u32x4 (&x)[kX], float sum) {
    float p = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      p = dot2(int8_pair_bf16(f.q[2 * h], 0), x[h].x, p);
      p = dot2(int8_pair_bf16(f.q[2 * h], 1), x[h].y, p);
      p = dot2(int8_pair_bf16(f.q[2 * h + 1], 0), x[h].z, p);
      p = dot2(int8_pair_bf16(f.q[2 * h + 1], 1), x[h].w, p);
    }
    return __builtin_fmaf(bf16_bits_to_f32(f.s), p, __builtin_fmaf(bf16_bits_to_f32(f.b), sum, acc));
  }
  static constexpr bool kSums = true;
};

// Activations of one row of K values in LDS: kX planes of segs * 64 pieces, then the sums
// of the lanes' runs where the format needs them.
template <class F>
__host__ __device__ constexpr uint32_t token_segs(uint32_t K) {
  return (K + F::kSeg - 1u) / F::kSeg;
}
template <class F>
__host__ __device__ constexpr uint32_t token_lds(uint32_t K) {
  return token_segs<F>(K) * (1024u * F::kX + (F::kSums ? 256u : 0u));
}

// n rows of K values, back to back, staged one token_lds() after the other by `threads`
// threads (a multiple of 64); zeros past K.  Four pieces a thread are in flight: with one,
// each was a memory latency of its own.  The first four are loaded by load() and written by
// finish(), with the weight's first loads in between: loads return in order, so the staging
// then waits for the activations alone.
template <class F>
struct TokenStage {
  u32x4 v[4];
  const uint16_t *x;
  uint32_t K, n, row, plane, stride, tid, threads;
  __device__ __forceinline__ TokenStage(const uint16_t *x_, uint32_t K_, uint32_t n_, uint32_t tid_, uint32_t threads_)
      : x(x_), K(K_), n(n_), tid(tid_), threads(threads_) {
    const uint32_t blocks = token_segs<F>(K) * 64u;
    plane = 16u * blocks;
    row = blocks * F::kX;
    stride = token_lds<F>(K);
  }
  __device__ __forceinline__ void load(uint32_t p0) {
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
      const uint32_t p = p0 + i * threads, r = p / row, c = p - r * row;
      v[i] = u32x4{0u, 0u, 0u, 0u};
      if (r < n && 8u * c < K) v[i] = *reinterpret_cast<const u32x4 *>(x + (size_t)r * K + 8u * c);
    }
    keep_order();
  }
  __device__ __forceinline__ void load() { load(tid); }
  __device__ __forceinline__ void write(uint8_t *lds, uint32_t p0) const {
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
      const uint32_t p = p0 + i * threads, r = p / row, c = p - r * row;
      if (r < n) {  // whole waves: a row is a multiple of 64 pieces
        uint8_t *at = lds + r * stride;
        *reinterpret_cast<u32x4 *>(at + (c % F::kX) * plane + 16u * (c / F::kX)) = v[i];
        if constexpr (F::kSums) {  // two neighbouring lanes hold a run of 16
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) s += bf16_lo(v[i][k]) + bf16_hi(v[i][k]);
          s += __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(s), 0xB1, 0xF, 0xF, true));
          if ((c & 1u) == 0) *reinterpret_cast<float *>(at + F::kX * plane + 4u * (c >> 1)) = s;
        }
      }
    }
  }
  __device__ __forceinline__ void finish(uint8_t *lds) {
    write(lds, tid);
    for (uint32_t p0 = tid + 4u * threads; p0 < n * row; p0 += 4u * threads) {
      load(p0);
      write(lds, p0);
    }
  }
};

template <class F>
__device__ __forceinline__ void get_token(u32x4 (&x)[F::kX], float &sum, const uint8_t *lds, uint32_t segs, uint32_t seg,
                                          uint32_t lane) {
  const uint32_t plane = 1024u * segs, at = 1024u * seg + 16u * lane;
#pragma unroll
  for (uint32_t f = 0; f < F::kX; ++f) x[f] = *reinterpret_cast<const u32x4 *>(lds + f * plane + at);
  sum = F::kSums ? *reinterpret_cast<const float *>(lds + F::kX * plane + 4u * (64u * seg + lane)) : 0.f;
}

template <class F>
struct TokenPair {
  typename F::Frag a, b;
};

}  // namespace int8w
