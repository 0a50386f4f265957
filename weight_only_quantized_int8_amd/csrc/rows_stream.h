// rows_stream.h -- weight rows streamed through one wave into matrix-core operands,
// shared by the MXFP4 product for few rows and the mixture-of-experts layer.
//
// v_mfma_f32_16x16x32_bf16 computes D[i][j] = sum_k A[i][k] B[k][j]; here A = 16
// activation rows, B = 16 weight rows.  Lane l holds A[l%16][8 (l/16) + 0..7], B[the
// same k][l%16] and D[4 (l/16) + r][l%16].  Which k stands behind a lane's eight
// values does not matter as long as A and B agree.
//
// Unit of work: a piece of 256 code bytes of each of 16 weight rows, in four quarters
// of 64 bytes a row.
//  * In the operand layout neighbouring lanes belong to different rows, and a load in
//    that layout costs the address unit a cycle a lane (measured: 64 a load, 2.4 TB/s
//    over the whole GPU).  So a load takes 128 bytes, a whole cache line, of each of 8
//    rows, eight lanes side by side (with 64 bytes of 16 rows the same stream without its
//    products took 204 us instead of 177), and the two quarters of a line change lanes
//    through 2 KB of LDS that only this wave uses, with no barrier.  16-byte chunks are
//    XOR-swizzled by row against bank conflicts.
//  * Activations of a quarter take the same way (rows of 256 or 128 bytes).
//  * Scales: one load a piece, lane l: row l/4, quarter l%4; a lane fetches its row's by
//    a lane permute.
//  * MXFP4: lane group g = l/16 takes block g of the quarter's four (32 codes, 16
//    bytes, one scale); MFMA f of four takes its codes 8f .. 8f+7, converted to BF16
//    with the scale applied (exact below 2^128).
//  * 8-bit affine: sum_k (q s + b) x = s sum q x + b sum x per run of one group: codes
//    enter the MFMA as exact BF16 integers, sum x comes from an MFMA against ones
//    (shared by the tiles), s and b are applied to the fp32 results.  Group size 64 and
//    128: a quarter is one run; 32: two.
// Loads past the end of a row, a weight or a list go to an offset beyond the buffer
// resource: they return zeros and touch no memory.
#pragma once

#include "mxfp4.h"

namespace int8w {

constexpr uint32_t kPieceBytes = 256;  // code bytes of a row in a piece

__device__ __forceinline__ uint32_t uniform32(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u32x4 bf16_ones() { return u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}; }

typedef int i32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f32x4 mfma_mx(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
  // fp4 operands take the first four registers of eight
  const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// LDS writes of this wave's lanes before reads by its other lanes: LDS instructions of a
// wave execute in order, so only the compiler has to keep it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint32_t lane_get(uint32_t v, uint32_t from) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute((int)(4u * from), (int)v);
}

// Where chunk c (16 bytes) of row r goes in a tile of 16 rows of 16 or of 8 chunks.  A 16-byte
// read goes through LDS in four phases of 16 lanes, 0-3, 12-15 and 20-27 the first of them: rows
// 0-3 and 12-15 of one lane group with rows 4-11 of the next.  So bit 3 of the XOR term (bit 2
// for 8 chunks) tells the two sets of rows apart, and each phase, like 16 lanes in order, takes
// 16 different chunks of the 256 bytes that the banks span.  With c ^ r the tiled BF16 product
// had 3.8 M conflict cycles a launch instead of 0.11 M, and took 1 to 2 % longer.
template <uint32_t P>
__device__ __forceinline__ uint32_t row_swizzle(uint32_t r, uint32_t c) {
  static_assert(P == 16u || P == 8u, "rows of 256 or 128 bytes");
  if constexpr (P == 16u) return c ^ ((r ^ ((r & 4u) << 1)) & 15u);
  const uint32_t t = (r >> 1) & 7u;
  return c ^ (t ^ ((t & 2u) << 1));
}

// A quarter of a tile of 16 rows x 64 bytes in LDS: chunk p of row r at 64 r + 16 (p ^ (r/2 % 4)).
// Of the two quarters of a line the second, i = 1, lies 1024 bytes on with neighbouring rows
// exchanged: writes go eight lanes at a time over 128 bytes of banks, and eight lanes write a
// row of both quarters.  Conflict cycles a piece of 16 rows 8 instead of 40, the expert layer 1
// to 2 % faster (8 experts of 14336x4096, 8 tokens in MXFP4: 132 us without either measure
// against conflicts, 129 with both).
__device__ __forceinline__ uint32_t quarter_at(uint32_t r, uint32_t p) { return 64u * r + 16u * (p ^ ((r >> 1) & 3u)); }
__device__ __forceinline__ u32x4 get_quarter(const uint8_t *lds, uint32_t i, uint32_t lane) {  // chunk l/16 of row l%16
  return *reinterpret_cast<const u32x4 *>(lds + 1024u * i + (quarter_at(lane & 15u, lane >> 4) ^ (64u * i)));
}

// The loads of a tile's piece: load j takes rows 8 (j & 1) + l/8, bytes 128 (j >> 1) + 16 (l % 8).
struct LineOffsets {
  uint32_t o[2];  // this lane's byte offset at piece 0 in the upper and the lower eight rows
  __device__ __forceinline__ LineOffsets() {}
  __device__ __forceinline__ LineOffsets(uint32_t rows, uint32_t row_bytes, uint32_t lane) {
    const uint32_t r = lane >> 3;
    o[0] = r < rows ? r * row_bytes + 16u * (lane & 7u) : kOutOfRange;
    o[1] = r + 8u < rows ? (r + 8u) * row_bytes + 16u * (lane & 7u) : kOutOfRange;
  }
};
template <int AUX>
__device__ __forceinline__ void load_lines(u32x4 (&q)[4], __amdgpu_buffer_rsrc_t rsrc, const LineOffsets &l, uint32_t row_bytes,
                                           uint32_t piece, uint32_t lane) {
  const uint32_t b0 = kPieceBytes * piece, c = 16u * (lane & 7u);
#pragma unroll
  for (uint32_t j = 0; j < 4u; ++j) {
    const uint32_t b = b0 + 128u * (j >> 1);
    q[j] = buf_load_b128<AUX>(rsrc, b + c < row_bytes ? l.o[j & 1u] + b : kOutOfRange);
  }
}
// Quarters 2 hp and 2 hp + 1 of a piece to lds and lds + 1024.
__device__ __forceinline__ void put_lines(uint8_t *lds, const u32x4 (&q)[4], int hp, uint32_t lane) {
  uint8_t *const at = lds + 1024u * ((lane >> 2) & 1u);
  const uint32_t flip = 64u * ((lane >> 2) & 1u);
  *reinterpret_cast<u32x4 *>(at + (quarter_at(lane >> 3, lane & 3u) ^ flip)) = q[2 * hp];
  *reinterpret_cast<u32x4 *>(at + (quarter_at(8u + (lane >> 3), lane & 3u) ^ flip)) = q[2 * hp + 1];
}

// ---- MXFP4 ------------------------------------------------------------------------------------
// DW: scales can be loaded four at a time (K a multiple of 128, scales 4-byte aligned).  A
// choice at run time would cost every wait of the loop: after a branch the compiler counts
// on the path with fewer loads in flight.
__host__ __device__ inline bool mx_dwords(const MxView &w) {
  return w.K % 128u == 0 && (reinterpret_cast<uintptr_t>(w.scales) & 3u) == 0;
}

template <bool DW>
struct MxFmt {
  typedef MxView View;
  static constexpr uint32_t kQuarter = 128;           // k a quarter
  static constexpr uint32_t kPiece = 4 * kQuarter;    // k a piece
  static constexpr uint32_t kXChunks = 16;            // 16-byte chunks of an activation row in a quarter
  static constexpr int kXFrags = 4;                   // A operands of a quarter
  static constexpr int kRuns = 1;
  static constexpr int kBlockWaves = 8;  // of a BlockStream (below): its activations take 32 KiB
  static __host__ __device__ constexpr uint32_t row_bytes(uint32_t K) { return K / 2u; }
  struct Tile {  // 16 weight rows
    __amdgpu_buffer_rsrc_t codes, scales;
    LineOffsets l;
    uint32_t os;  // this lane's byte offset at piece 0 (kOutOfRange for a row past the end)
  };
  struct Piece {
    u32x4 q[4];
    uint32_t s;  // row l/4, the four scales of quarter l%4
  };

  // rows [n0, n0 + 16) of the N rows that start at row `base` of the weight
  static __device__ __forceinline__ Tile tile(const MxView &w, uint64_t base, uint32_t n0, uint32_t N, uint32_t lane) {
    Tile t;
    const uint32_t rows = N - n0 < 16u ? N - n0 : 16u, r = lane >> 2, p = lane & 3u;
    const uint64_t row0 = base + n0;
    const uint8_t *sc = w.scales + row0 * (w.K / 32u);
    t.codes = make_rsrc(w.codes + row0 * (w.K / 2u), rows * (w.K / 2u));
    t.scales = make_rsrc(sc, rows * (w.K / 32u));
    t.l = LineOffsets(rows, w.K / 2u, lane);
    t.os = r < rows ? r * (w.K / 32u) + 4u * p : kOutOfRange;
    return t;
  }
  template <int AUX>
  static __device__ __forceinline__ void load(Piece &f, const Tile &t, const MxView &w, uint32_t piece, uint32_t lane) {
    const uint32_t p = lane & 3u;
    load_lines<AUX>(f.q, t.codes, t.l, w.K / 2u, piece, lane);
    const uint32_t blk = 16u * piece + 4u * p;  // first block of quarter p
    if constexpr (DW) {
      f.s = __builtin_amdgcn_raw_buffer_load_b32(t.scales, (int)(blk < w.K / 32u ? t.os + 16u * piece : kOutOfRange), 0, 0);
    } else {
      f.s = 0;
#pragma unroll
      for (uint32_t i = 0; i < 4u; ++i)
        f.s |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(
                   t.scales, (int)(blk + i < w.K / 32u ? t.os + 16u * piece + i : kOutOfRange), 0, 0) << (8u * i);
    }
  }
  // scale byte of row l%16, block l/16 of quarter h
  static __device__ __forceinline__ uint32_t scale(const Piece &f, int h, uint32_t lane) {
    return (lane_get(f.s, 4u * (lane & 15u) + h) >> (8u * (lane >> 4))) & 0xFFu;
  }
  static __device__ __forceinline__ uint32_t x_chunk(int f, uint32_t g) { return 4u * g + f; }
  struct Sums {};
  static __device__ __forceinline__ void sums(Sums &, const u32x4 (&)[kXFrags]) {}
  static __device__ __forceinline__ void mac(f32x4 &acc, u32x4 q, const Piece &f, int h, const u32x4 (&x)[kXFrags],
                                             const Sums &, uint32_t lane) {
    const float s = mx_scale_f32(scale(f, h, lane));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 b = mx_to_bf16x8(q[i], s);
      acc = mfma16(x[i], u32x4{b.x, b.y, b.z, b.w}, acc);
    }
  }
};

// ---- 8-bit affine -----------------------------------------------------------------------------
__device__ __forceinline__ u32x4 int8_codes_bf16(uint32_t a, uint32_t b) {
  return u32x4{int8_pair_bf16(a, 0), int8_pair_bf16(a, 1), int8_pair_bf16(b, 0), int8_pair_bf16(b, 1)};
}

template <bool G32>
struct Int8Fmt {
  typedef WeightView View;
  static constexpr uint32_t kQuarter = 64;
  static constexpr uint32_t kPiece = 4 * kQuarter;
  static constexpr uint32_t kXChunks = 8;
  static constexpr int kXFrags = 2;
  static constexpr int kRuns = G32 ? 2 : 1;  // runs of one group in a quarter
  static constexpr int kBlockWaves = 4;      // of a BlockStream (below): its activations take 16 KiB
  static __host__ __device__ constexpr uint32_t row_bytes(uint32_t K) { return K; }
  struct Tile {
    __amdgpu_buffer_rsrc_t codes, scales, biases;
    LineOffsets l;
    uint32_t os;
  };
  struct Piece {
    u32x4 q[4];
    uint16_t s[kRuns], b[kRuns];  // row l/4, quarter l%4
  };

  static __device__ __forceinline__ Tile tile(const WeightView &w, uint64_t base, uint32_t n0, uint32_t N, uint32_t lane) {
    Tile t;
    const uint32_t rows = N - n0 < 16u ? N - n0 : 16u, r = lane >> 2, G = w.K / w.gs;
    const uint64_t row0 = base + n0;
    t.codes = make_rsrc((const uint8_t *)w.packed + row0 * w.K, rows * w.K);
    t.scales = make_rsrc(w.scales + row0 * G, rows * G * 2u);
    t.biases = make_rsrc(w.biases + row0 * G, rows * G * 2u);
    t.l = LineOffsets(rows, w.K, lane);
    t.os = r < rows ? r * G * 2u : kOutOfRange;
    return t;
  }
  template <int AUX>
  static __device__ __forceinline__ void load(Piece &f, const Tile &t, const WeightView &w, uint32_t piece, uint32_t lane) {
    const uint32_t p = lane & 3u, b0 = kPieceBytes * piece;
    load_lines<AUX>(f.q, t.codes, t.l, w.K, piece, lane);
    const uint32_t gl = 31u - (uint32_t)__builtin_clz(w.gs);
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const uint32_t k = b0 + 64u * p + 32u * r;  // first k of the run
      const uint32_t o = k < w.K ? t.os + 2u * (k >> gl) : kOutOfRange;
      f.s[r] = buf_load_b16(t.scales, o);
      f.b[r] = buf_load_b16(t.biases, o);
    }
  }
  static __device__ __forceinline__ uint32_t x_chunk(int f, uint32_t g) { return G32 ? 4u * f + g : 2u * g + f; }
  struct Sums {
    f32x4 v[kRuns];
  };
  static __device__ __forceinline__ void sums(Sums &S, const u32x4 (&x)[kXFrags]) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    S.v[0] = mfma16(x[0], bf16_ones(), zero);
    if constexpr (G32)
      S.v[1] = mfma16(x[1], bf16_ones(), zero);
    else
      S.v[0] = mfma16(x[1], bf16_ones(), S.v[0]);
  }
  static __device__ __forceinline__ void mac(f32x4 &acc, u32x4 q, const Piece &f, int h, const u32x4 (&x)[kXFrags],
                                             const Sums &S, uint32_t lane) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const uint32_t sb = lane_get((uint32_t)f.s[r] | (uint32_t)f.b[r] << 16, 4u * (lane & 15u) + h);
      const float s = bf16_lo(sb), b = bf16_hi(sb);
      f32x4 P;
      if constexpr (G32) {
        P = r ? mfma16(x[1], int8_codes_bf16(q.z, q.w), zero) : mfma16(x[0], int8_codes_bf16(q.x, q.y), zero);
      } else {
        P = mfma16(x[0], int8_codes_bf16(q.x, q.y), zero);
        P = mfma16(x[1], int8_codes_bf16(q.z, q.w), P);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(s, P[i], __builtin_fmaf(b, S.v[r][i], acc[i]));
    }
  }
  // G32: a lane's 16 bytes of the quarter are 8 of each run
  static __device__ __forceinline__ u32x4 get(const uint8_t *lds, uint32_t i, uint32_t lane) {
    lds += 1024u * i;
    const uint32_t r = lane & 15u, g = lane >> 4;
    const u32x2 lo = *reinterpret_cast<const u32x2 *>(lds + (quarter_at(r, g >> 1) ^ (64u * i)) + 8u * (g & 1u));
    const u32x2 hi = *reinterpret_cast<const u32x2 *>(lds + (quarter_at(r, 2u + (g >> 1)) ^ (64u * i)) + 8u * (g & 1u));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  }
};

template <class F>
__device__ __forceinline__ u32x4 weight_operand(const uint8_t *lds, uint32_t i, uint32_t lane) {
  return get_quarter(lds, i, lane);
}
template <>
__device__ __forceinline__ u32x4 weight_operand<Int8Fmt<true>>(const uint8_t *lds, uint32_t i, uint32_t lane) {
  return Int8Fmt<true>::get(lds, i, lane);
}

// ---- one wave's stream ------------------------------------------------------------------------

// BF16 activations of up to 4 NX (MXFP4) or 8 NX (8-bit) rows.
template <class F, int NX>
struct XBf16 {
  static constexpr uint32_t kRows = 64u / F::kXChunks;         // rows a load
  static constexpr uint32_t kLds = 1024u * NX;                 // a quarter's
  struct Piece {
    u32x4 v[4][NX];
  };
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t K, xo[NX];  // byte offset of the lane's row of load j, with its chunk
  // row(i): byte offset of activation row i, or kOutOfRange
  template <class Row>
  __device__ __forceinline__ XBf16(const void *x, uint32_t bytes, uint32_t K_, uint32_t lane, Row row) : K(K_) {
    rsrc = make_rsrc(x, bytes);
#pragma unroll
    for (int j = 0; j < NX; ++j) xo[j] = row(kRows * j + lane / F::kXChunks) + 16u * (lane % F::kXChunks);
  }
  __device__ __forceinline__ void load(Piece &f, uint32_t piece, uint32_t lane) const {
    const uint32_t b0 = piece * (2u * F::kPiece), c = 16u * (lane % F::kXChunks);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint32_t b = b0 + 2u * F::kQuarter * h;
#pragma unroll
      for (int j = 0; j < NX; ++j) f.v[h][j] = buf_load_b128(rsrc, b + c < 2u * K ? xo[j] + b : kOutOfRange);
    }
  }
  static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t c) {
    return row * (16u * F::kXChunks) + 16u * row_swizzle<F::kXChunks>(row, c);
  }
  __device__ __forceinline__ void put(uint8_t *lds, const Piece &f, int h, uint32_t lane) const {
#pragma unroll
    for (int j = 0; j < NX; ++j)
      *reinterpret_cast<u32x4 *>(lds + at(kRows * j + lane / F::kXChunks, lane % F::kXChunks)) = f.v[h][j];
  }
  // rows past the ones kept repeat the last: their results are not used
  static __device__ __forceinline__ void get(u32x4 (&x)[F::kXFrags], const uint8_t *lds, uint32_t lane) {
    uint32_t row = lane & 15u;
    if (row >= kRows * NX) row = kRows * NX - 1u;
#pragma unroll
    for (int f = 0; f < F::kXFrags; ++f) x[f] = *reinterpret_cast<const u32x4 *>(lds + at(row, F::x_chunk(f, lane >> 4)));
  }
};

// LDS bytes of one wave: two quarters of its tile and of the activations.
template <class X>
constexpr uint32_t stream_lds() {
  return 2u * (1024u + X::kLds);
}

template <class F, class X>
struct Pieces {
  typename F::Piece w;
  typename X::Piece x;
};

// acc[0] + acc[1] += A B^T of one piece: the two quarters of a line have sums of their own, so
// that neither waits for the other's products.
template <class F, class X>
__device__ __forceinline__ void stream_piece(f32x4 (&acc)[2], const Pieces<F, X> &p, const X &X_, uint8_t *lds,
                                             uint32_t lane) {
  uint8_t *const xl = lds + 2048u;
#pragma unroll
  for (int hp = 0; hp < 2; ++hp) {
    put_lines(lds, p.w.q, hp, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) X_.put(xl + i * X::kLds, p.x, 2 * hp + i, lane);
    wave_fence();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u32x4 x[F::kXFrags];
      X::get(x, xl + i * X::kLds, lane);
      typename F::Sums S;
      F::sums(S, x);
      F::mac(acc[i], weight_operand<F>(lds, i, lane), p.w, 2 * hp + i, x, S, lane);
    }
    wave_fence();
  }
}

// ---- a workgroup's stream ---------------------------------------------------------------------
// KW waves, each with RT tiles of 16 weight rows of its own, walk K together.  The
// activations of a piece are shared in LDS, two buffers, one barrier a piece; weights go as
// above.  A wave requests the next piece's weights as soon as the present one's are used, and
// counts on the other waves of the CU (four a SIMD) to compute meanwhile: a second piece in
// flight a wave cost the registers of the fourth wave (37 tokens, 8 experts in MXFP4: 164 us
// instead of 150, 4 tokens in 8 bits 264 instead of 249).
template <class F, int KW, int RT>
struct BlockStream {
  static constexpr uint32_t kQuarterLds = 256u * F::kXChunks;             // 16 rows of a quarter's activations
  static constexpr uint32_t kXLds = 4u * kQuarterLds;
  static constexpr uint32_t kWaveLds = 2u * 1024u * RT;
  static constexpr uint32_t kLds = 2u * kXLds + KW * kWaveLds;
  static constexpr uint32_t kRowChunks = 4u * F::kXChunks;                // 16-byte chunks of a row in a piece
  static constexpr int NX = (int)(16u * kRowChunks / (64u * KW));         // activation loads a wave
  static_assert(16u * kRowChunks % (64u * KW) == 0, "whole loads");

  typename F::Tile t[RT];
  __amdgpu_buffer_rsrc_t rx;
  uint32_t K, lane, wave, xo[NX], xk[NX], xl[NX];
  uint8_t *lds;
  f32x4 acc[RT][2];  // to be added

  // row(i): byte offset of activation row i (i < 16), or kOutOfRange
  template <class Row>
  __device__ __forceinline__ BlockStream(uint8_t *lds_, const void *x, uint32_t xbytes, uint32_t K_, uint32_t lane_,
                                         uint32_t wave_, Row row)
      : K(K_), lane(lane_), wave(wave_), lds(lds_) {
    rx = make_rsrc(x, xbytes);
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const uint32_t c = (wave * NX + j) * 64u + lane, r = c / kRowChunks, k = c % kRowChunks;
      xk[j] = 16u * k;
      xo[j] = row(r) + 16u * k;
      xl[j] = k / F::kXChunks * kQuarterLds + XBf16<F, 1>::at(r, k % F::kXChunks);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void load_x(u32x4 (&v)[NX], uint32_t piece) const {
    const uint32_t b = piece * (2u * F::kPiece);
#pragma unroll
    for (int j = 0; j < NX; ++j) v[j] = buf_load_b128(rx, b + xk[j] < 2u * K ? xo[j] + b : kOutOfRange);
    keep_order();
  }
  __device__ __forceinline__ void put_x(const u32x4 (&v)[NX], uint32_t buf) const {
#pragma unroll
    for (int j = 0; j < NX; ++j) *reinterpret_cast<u32x4 *>(lds + buf * kXLds + xl[j]) = v[j];
  }
  template <int AUX, class View>
  __device__ __forceinline__ void load_w(typename F::Piece (&w)[RT], const View *const *v, uint32_t piece) const {
#pragma unroll
    for (int i = 0; i < RT; ++i) F::template load<AUX>(w[i], t[i], *v[i], piece, lane);
    keep_order();
  }
  __device__ __forceinline__ void products(const typename F::Piece (&w)[RT], uint32_t buf) {
    uint8_t *const own = lds + 2u * kXLds + wave * kWaveLds;
#pragma unroll
    for (int hp = 0; hp < 2; ++hp) {
#pragma unroll
      for (int t = 0; t < RT; ++t) put_lines(own + 2048u * t, w[t].q, hp, lane);
      wave_fence();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = 2 * hp + i;
        u32x4 x[F::kXFrags];
#pragma unroll
        for (int f = 0; f < F::kXFrags; ++f)
          x[f] = *reinterpret_cast<const u32x4 *>(lds + buf * kXLds + h * kQuarterLds + XBf16<F, 1>::at(lane & 15u, F::x_chunk(f, lane >> 4)));
        typename F::Sums S;
        F::sums(S, x);
#pragma unroll
        for (int t = 0; t < RT; ++t) F::mac(acc[t][i], weight_operand<F>(own + 2048u * t, i, lane), w[t], h, x, S, lane);
      }
      wave_fence();
    }
  }
  // acc += A B^T over all of K, from piece `first` on and round.  Workgroups that start
  // at the same piece walk the rows' same 256 bytes together, a row length apart: with row
  // lengths of whole kilobytes that is one memory channel in sixteen at a time.
  template <int AUX, class View>
  __device__ __forceinline__ void run(const View *const *v, uint32_t first) {
    const uint32_t np = (K + F::kPiece - 1u) / F::kPiece;
    uint32_t next = first % np, left = np;  // the next piece to load
    auto take = [&]() {
      const uint32_t c = left ? next : np;  // past the end: zeros, no traffic
      left -= left ? 1u : 0u;
      next = next + 1u == np ? 0u : next + 1u;
      return c;
    };
    typename F::Piece w[RT];
    u32x4 x[NX];
    uint32_t p = take();
    load_x(x, p);
    load_w<AUX>(w, v, p);
    put_x(x, 0);
    p = take();
    load_x(x, p);
    __syncthreads();
    for (uint32_t c = 0; c < np; ++c) {
      products(w, c & 1u);
      load_w<AUX>(w, v, p);
      put_x(x, (c + 1u) & 1u);
      keep_order();
      p = take();
      load_x(x, p);
      block_barrier();
    }
  }
  // LDS only: the loads in flight go to registers of the wave that waits for them
  static __device__ __forceinline__ void block_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
};

}  // namespace int8w
