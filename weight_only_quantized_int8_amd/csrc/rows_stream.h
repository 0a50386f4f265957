// rows_stream.h -- weight rows streamed from memory straight into matrix-core
// operands, shared by the MXFP4 product for few rows and the
// mixture-of-experts layer.
//
// Unit: a tile of 16 weight rows times a chunk of 128 k.  v_mfma_f32_16x16x32_bf16
// computes D[i][j] = sum_k A[i][k] B[k][j] with A = activation rows (16 tokens)
// and B = weight rows; lane l holds A[l%16][8 (l/16) + 0..7], B[the same k][l%16]
// and D[4 (l/16) + r][l%16].  Which k stands behind a lane's eight values does not
// matter as long as A and B agree, so a lane loads 16 contiguous code bytes of its
// row and the activations that go with them, with no staging and no barrier:
//  * MXFP4: lane group g = l/16 takes block 4c + g of chunk c (32 codes, 16 bytes,
//    one scale); MFMA f of four takes its codes 8f .. 8f+7, converted to BF16 with
//    the scale applied (exact).
//  * 8-bit affine: sum_k (q s + b) x = s sum q x + b sum x per run of one group:
//    codes enter the MFMA as exact BF16 integers, sum x comes from an MFMA against
//    ones (shared by all tiles of the chunk), and the group's s and b are applied to
//    the fp32 results.  Group size 64 and 128: a lane takes 16 bytes of each 64-code
//    half; 32: 8 bytes of each 32 codes.
// Loads past the end of a row, a weight or a list go to an offset beyond the buffer
// resource: they return zeros and touch no memory.
#pragma once

#include "mxfp4.h"

namespace int8w {

constexpr uint32_t kChunk = 128;  // k per chunk

typedef u32x4 XFrag[4];  // one token tile's A operands of a chunk

__device__ __forceinline__ uint32_t uniform32(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u32x4 bf16_ones() { return u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}; }

// ---- MXFP4 ------------------------------------------------------------------------------------
struct MxFmt {
  typedef MxView View;
  struct Tile {  // 16 weight rows
    __amdgpu_buffer_rsrc_t codes, scales;
    uint32_t oc, os;  // this lane's byte offsets at chunk 0 (kOutOfRange for a row past the end)
  };
  struct Frag {
    u32x4 q;
    uint32_t s;
  };
  static constexpr int kSums = 0;

  // rows [n0, n0 + 16) of the N rows that start at row `base` of the weight
  static __device__ __forceinline__ Tile tile(const MxView &w, uint64_t base, uint32_t n0, uint32_t N, uint32_t lane) {
    Tile t;
    const uint32_t rows = N - n0 < 16u ? N - n0 : 16u, lr = lane & 15u, g = lane >> 4;
    const uint64_t row0 = base + n0;
    t.codes = make_rsrc(w.codes + row0 * (w.K / 2u), rows * (w.K / 2u));
    t.scales = make_rsrc(w.scales + row0 * (w.K / 32u), rows * (w.K / 32u));
    t.oc = lr < rows ? lr * (w.K / 2u) + 16u * g : kOutOfRange;
    t.os = lr < rows ? lr * (w.K / 32u) + g : kOutOfRange;
    return t;
  }
  static __device__ __forceinline__ bool live(uint32_t c, uint32_t K, uint32_t g) { return 4u * c + g < K / 32u; }
  static __device__ __forceinline__ void load(Frag &f, const Tile &t, const MxView &w, uint32_t c, uint32_t lane) {
    const bool in = live(c, w.K, lane >> 4);
    f.q = buf_load_b128<kAuxNontemporal>(t.codes, in ? t.oc + 64u * c : kOutOfRange);
    f.s = __builtin_amdgcn_raw_buffer_load_b8(t.scales, (int)(in ? t.os + 4u * c : kOutOfRange), 0, 0);
  }
  // xo: byte offset of the lane's activation row (kOutOfRange: none)
  static __device__ __forceinline__ void load_x(XFrag &x, __amdgpu_buffer_rsrc_t r, uint32_t xo, uint32_t c, uint32_t K,
                                                uint32_t lane) {
    const uint32_t o = live(c, K, lane >> 4) ? xo + 256u * c + 64u * (lane >> 4) : kOutOfRange;
#pragma unroll
    for (int f = 0; f < 4; ++f) x[f] = buf_load_b128(r, o + 16u * f);
  }
  template <int MT>
  static __device__ __forceinline__ void sums(f32x4 (&)[MT][4], const XFrag (&)[MT]) {}
  template <int MT>
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT], const Frag &f, const XFrag (&x)[MT], const f32x4 (&)[MT][4]) {
    const float s = mx_scale_f32(f.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 b = mx_to_bf16x8(f.q[i], s);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[mt] = mfma16(x[mt][i], u32x4{b.x, b.y, b.z, b.w}, acc[mt]);
    }
  }
};

// ---- 8-bit affine -----------------------------------------------------------------------------
__device__ __forceinline__ u32x4 int8_codes_bf16(uint32_t a, uint32_t b) {  // eight codes as BF16 integers (exact)
  return u32x4{pack_bf16x2(code_f32(a, 0), code_f32(a, 1)), pack_bf16x2(code_f32(a, 2), code_f32(a, 3)),
               pack_bf16x2(code_f32(b, 0), code_f32(b, 1)), pack_bf16x2(code_f32(b, 2), code_f32(b, 3))};
}

template <bool G32>
struct Int8Fmt {
  typedef WeightView View;
  static constexpr int kRuns = G32 ? 4 : 2;  // runs of one group in a chunk
  static constexpr int kSums = kRuns;
  struct Tile {
    __amdgpu_buffer_rsrc_t codes, scales, biases;
    uint32_t oc, os;
  };
  struct Frag {
    u32x4 q[2];
    uint16_t s[kRuns], b[kRuns];
  };

  static __device__ __forceinline__ Tile tile(const WeightView &w, uint64_t base, uint32_t n0, uint32_t N, uint32_t lane) {
    Tile t;
    const uint32_t rows = N - n0 < 16u ? N - n0 : 16u, lr = lane & 15u, g = lane >> 4, G = w.K / w.gs;
    const uint64_t row0 = base + n0;
    t.codes = make_rsrc((const uint8_t *)w.packed + row0 * w.K, rows * w.K);
    t.scales = make_rsrc(w.scales + row0 * G, rows * G * 2u);
    t.biases = make_rsrc(w.biases + row0 * G, rows * G * 2u);
    t.oc = lr < rows ? lr * w.K + (G32 ? 8u : 16u) * g : kOutOfRange;
    t.os = lr < rows ? lr * G * 2u : kOutOfRange;
    return t;
  }
  static __device__ __forceinline__ void load(Frag &f, const Tile &t, const WeightView &w, uint32_t c, uint32_t lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = kChunk * c + 64u * h;
      if constexpr (G32) {
        const u32x2 lo = buf_load_b64<kAuxNontemporal>(t.codes, k < w.K ? t.oc + k : kOutOfRange);
        const u32x2 hi = buf_load_b64<kAuxNontemporal>(t.codes, k + 32u < w.K ? t.oc + k + 32u : kOutOfRange);
        f.q[h] = u32x4{lo.x, lo.y, hi.x, hi.y};
      } else {
        f.q[h] = buf_load_b128<kAuxNontemporal>(t.codes, k < w.K ? t.oc + k : kOutOfRange);
      }
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const uint32_t k = kChunk * c + (kChunk / kRuns) * r;
      const uint32_t o = k < w.K ? t.os + 2u * (k / w.gs) : kOutOfRange;
      f.s[r] = buf_load_b16(t.scales, o);
      f.b[r] = buf_load_b16(t.biases, o);
    }
  }
  static __device__ __forceinline__ void load_x(XFrag &x, __amdgpu_buffer_rsrc_t r, uint32_t xo, uint32_t c, uint32_t K,
                                                uint32_t lane) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const uint32_t k = kChunk * c + (G32 ? 32u * f : 64u * (f >> 1));  // first k of the run
      const uint32_t kl = G32 ? k + 8u * (lane >> 4) : k + 16u * (lane >> 4) + 8u * (f & 1);
      x[f] = buf_load_b128(r, k < K ? xo + 2u * kl : kOutOfRange);
    }
  }
  template <int MT>
  static __device__ __forceinline__ void sums(f32x4 (&S)[MT][4], const XFrag (&x)[MT]) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < kRuns; ++r) {
        if constexpr (G32) {
          S[mt][r] = mfma16(x[mt][r], bf16_ones(), zero);
        } else {
          S[mt][r] = mfma16(x[mt][2 * r], bf16_ones(), zero);
          S[mt][r] = mfma16(x[mt][2 * r + 1], bf16_ones(), S[mt][r]);
        }
      }
  }
  template <int MT>
  static __device__ __forceinline__ void mac(f32x4 (&acc)[MT], const Frag &f, const XFrag (&x)[MT], const f32x4 (&S)[MT][4]) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const float s = bf16_bits_to_f32(f.s[r]), b = bf16_bits_to_f32(f.b[r]);
      u32x4 lo, hi;
      if constexpr (G32) {
        lo = r & 1 ? int8_codes_bf16(f.q[r >> 1].z, f.q[r >> 1].w) : int8_codes_bf16(f.q[r >> 1].x, f.q[r >> 1].y);
      } else {
        lo = int8_codes_bf16(f.q[r].x, f.q[r].y);
        hi = int8_codes_bf16(f.q[r].z, f.q[r].w);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        f32x4 P;
        if constexpr (G32) {
          P = mfma16(x[mt][r], lo, zero);
        } else {
          P = mfma16(x[mt][2 * r], lo, zero);
          P = mfma16(x[mt][2 * r + 1], hi, P);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][i] = __builtin_fmaf(s, P[i], __builtin_fmaf(b, S[mt][r][i], acc[mt][i]));
      }
    }
  }
};

}  // namespace int8w
