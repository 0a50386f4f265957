// mxfp4_gemm.hip -- Y[m, N] = X[m, K] W^T with W in MXFP4 (mxfp4.h) and X in
// BF16 (weight-only) or in MXFP4 too.  fp32 accumulation, one rounding to BF16.
//
// Three kernels, chosen by launch_any() below:
//  k_mx_gemv  one row of BF16: vector ALUs, weight rows streamed along K (token_stream.h).
//  k_mx_rows  few rows, or many on a small weight: a workgroup owns 16 weight rows and up
//             to 16 rows of X, its waves share K piece by piece (rows_stream.h) and meet in
//             LDS in wave order.
//  k_mx_tile  more: LDS-tiled, on bf16 MFMA (X BF16: codes are converted with their scale
//             in registers, exactly below 2^128) or on the scaled fp4 MFMA (both MXFP4: 16 x 16 x 128
//             products with a scale per 32 k in the instruction).
// The first is bound by HBM, once the weight is large enough to hide a launch; the second by the
// re-reading of X through the L2s and by latency; the third, with several hundred rows of X, by
// the matrix cores and by the LDS and conversions that feed them, with fewer again by re-reading.
#include <type_traits>
#include <utility>

#include "rows_stream.h"
#include "token_stream.h"
#include "launch.h"

namespace int8w {

namespace {

// ---- one row ----------------------------------------------------------------------------------

// y[n] = sum_k W[n, k] x[k].  Waves share the pairs of weight rows; KS neighbouring waves
// share a pair's segments where there are few pairs.  LDS: x.  HBM-bound: 8192x28672, 125 MB
// in 21.2 us, 5.9 TB/s; 4096x4096, 8.9 MB, 4.1 us, mostly the start and end of a launch.
template <int KW, int U, int KS>
__global__ __launch_bounds__(64 * KW) void k_mx_gemv(MxView w, const uint16_t *__restrict__ x, uint16_t *__restrict__ y) {
  typedef MxTok F;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_gemv[];
  __shared__ float red[KW][2];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), K = w.K, segs = token_segs<F>(K);
  const uint32_t units = gridDim.x * (KW / KS), unit = blockIdx.x * (KW / KS) + wave / KS, ks = wave % KS;
  const uint32_t pairs = (w.N + 1u) / 2u;
  const uint32_t p0 = (uint32_t)((uint64_t)pairs * unit / units), p1 = (uint32_t)((uint64_t)pairs * (unit + 1u) / units);
  const uint32_t s0 = segs * ks / KS, s1 = segs * (ks + 1u) / KS;  // the wave's segments of a pair
  uint32_t lp = p0, ls = s0;                                       // the next load
  TokenStage<F> stage(x, K, 1u, threadIdx.x, 64u * KW);
  stage.load();
  F::Row ra, rb;
  auto rows = [&]() {
    const bool a = lp < p1, b = a && 2u * lp + 1u < w.N;
    ra = F::row(w, a ? 2u * lp : 0u, a);
    rb = F::row(w, b ? 2u * lp + 1u : 0u, b);
  };
  rows();
  TokenPair<F> ring[U];
  auto load = [&](TokenPair<F> &t) {
    F::load(t.a, ra, w, ls, lane);
    F::load(t.b, rb, w, ls, lane);
    keep_order();
    if (++ls >= s1) {
      ls = s0;
      ++lp;
      rows();
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(ring[u]);
  stage.finish(lds_gemv);
  __syncthreads();
  float a = 0.f, b = 0.f;
  uint32_t cp = p0, cs = s0;
  auto store = [&](uint32_t p, float va, float vb) {
    const uint32_t r = 2u * p + lane;
    if (lane < 2u && r < w.N) y[r] = to_bf16_bits(lane ? vb : va);
  };
  for (uint32_t i = 0, items = (p1 - p0) * (s1 - s0); i < items; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < items) {
        u32x4 xv[F::kX];
        float xsum;
        get_token<F>(xv, xsum, lds_gemv, segs, cs, lane);
        a = F::dot(a, ring[u].a, xv, xsum);
        b = F::dot(b, ring[u].b, xv, xsum);
        if (++cs == s1) {
          cs = s0;
          if constexpr (KS == 1) {
            store(cp, token_sum(a), token_sum(b));
            a = b = 0.f;
          }
          ++cp;
        }
      }
      keep_order();
      load(ring[u]);
    }
  }
  if constexpr (KS > 1) {
    a = token_sum(a);
    b = token_sum(b);
    if (lane == 0) {
      red[wave][0] = a;
      red[wave][1] = b;
    }
    __syncthreads();
    if (ks == 0 && p0 < p1) {
      a = b = 0.f;
#pragma unroll
      for (uint32_t k = 0; k < (uint32_t)KS; ++k) {
        a += red[wave + k][0];
        b += red[wave + k][1];
      }
      store(p0, a, b);
    }
  }
}

template <int KW, int KS>
hipError_t launch_gemv_one(const MxView &w, const uint16_t *x, uint16_t *y, hipStream_t stream) {
  auto kern = k_mx_gemv<KW, 2, KS>;
  const uint32_t lds = token_lds<MxTok>(w.K);
  static LdsAllowance allowance;
  if (needs_lds_allowance(lds, sizeof(float[KW][2]))) {
    const hipError_t e = allow_lds(allowance, kern, 159 << 10);
    if (e != hipSuccess) return e;
  }
  const uint32_t units = KW / KS, want = ((w.N + 1u) / 2u + units - 1u) / units;
  const uint32_t most = (uint32_t)device_cu_count();
  kern<<<KS > 1 || want < most ? want : most, 64 * KW, lds, stream>>>(w, x, y);
  return hipGetLastError();
}

hipError_t launch_gemv(const MxView &w, const uint16_t *x, uint16_t *y, hipStream_t stream) {
  // one workgroup of 8 waves a CU, two segments of a pair in flight: more waves cost more to
  // start, and a longer ring more instructions to fetch, than they bring (us with 8 / 16 waves
  // a CU: 4096x4096 4.9 / 6.5, 4096x14336 8.0 / 9.0, 8192x28672 22.5 / 22.5; with 2 / 4 / 8
  // segments 4.1 / 4.7 / 5.9, 7.8 / 7.9 / 9.5, 22.6 / 22.6 / 23.9)
  const uint32_t pairs = (w.N + 1u) / 2u, waves = 8u * (uint32_t)device_cu_count(), segs = token_segs<MxTok>(w.K);
  if (pairs * 4u <= waves && segs >= 4u) return launch_gemv_one<8, 4>(w, x, y, stream);
  if (pairs * 2u <= waves && segs >= 2u) return launch_gemv_one<8, 2>(w, x, y, stream);
  return launch_gemv_one<8, 1>(w, x, y, stream);
}

// ---- few rows ---------------------------------------------------------------------------------

// Activations in MXFP4: another tile of rows.
template <bool DW>
struct XMx {
  static constexpr uint32_t kLds = 1024u;
  typedef typename MxFmt<DW>::Piece Piece;
  MxView v;
  typename MxFmt<DW>::Tile t;
  __device__ __forceinline__ XMx(const void *x, const uint8_t *scales, uint32_t m0, uint32_t m, uint32_t K, uint32_t lane) {
    v = MxView{(const uint8_t *)x, scales, m, K};
    t = MxFmt<DW>::tile(v, 0, m0, m, lane);
  }
  __device__ __forceinline__ void load(Piece &f, uint32_t piece, uint32_t lane) const { MxFmt<DW>::template load<0>(f, t, v, piece, lane); }
};

template <bool DW>
__device__ __forceinline__ void stream_piece_mx(f32x4 (&acc)[2], const Pieces<MxFmt<DW>, XMx<DW>> &p, uint8_t *lds, uint32_t lane) {
#pragma unroll
  for (int hp = 0; hp < 2; ++hp) {
    put_lines(lds, p.w.q, hp, lane);
    put_lines(lds + 2048u, p.x.q, hp, lane);
    wave_fence();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      acc[i] = mfma_mx(get_quarter(lds + 2048u, i, lane), MxFmt<DW>::scale(p.x, 2 * hp + i, lane),
                       get_quarter(lds, i, lane), MxFmt<DW>::scale(p.w, 2 * hp + i, lane), acc[i]);
    wave_fence();
  }
}

// grid: (16-row weight tiles) x (groups of 16 rows of X), the groups of a tile side by side.
// Every workgroup reads its rows of X itself: in BF16 with m = 16, 32 bytes of X for each 8.5 of
// weight.  And a row of 14336 is 28 pieces, three or four a wave, so the first loads' latency and
// the waves' last sum are a large part of a call.  4096x14336 (31.8 MB at m = 16, floor 4.6 us):
// m = 16 12.4 us with 152 MB requested from the L2s; m = 48, three groups, 27.3 us with 463 MB
// requested and 107 MB from HBM (the groups do not find each other's weights); X in MXFP4 m = 8
// 8.5 us, m = 32 12.6 us with 116 MB requested.
template <bool XMX, bool DW, int KS, int U, int NX, int AUX>
__global__ __launch_bounds__(64 * KS) void k_mx_rows(MxView w, const void *__restrict__ x,
                                                     const uint8_t *__restrict__ xs, uint32_t m, uint32_t groups,
                                                     uint16_t *__restrict__ y) {
  typedef MxFmt<DW> F;
  typedef std::conditional_t<XMX, XMx<DW>, XBf16<F, NX>> X;
  constexpr uint32_t kWaveLds = stream_lds<X>();
  __shared__ __attribute__((aligned(16))) uint8_t lds[KS * kWaveLds];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), K = w.K;
  const uint32_t n0 = 16u * (blockIdx.x / groups), m0 = 16u * (blockIdx.x % groups);
  const uint32_t rows = m - m0 < 16u ? m - m0 : 16u;
  const typename F::Tile t = F::tile(w, 0, n0, w.N, lane);
  auto make = [&]() {
    if constexpr (XMX)
      return X(x, xs, m0, m, K, lane);
    else
      return X((const uint16_t *)x + (size_t)m0 * K, rows * K * 2u, K, lane,
               [&](uint32_t i) { return i < rows ? i * K * 2u : kOutOfRange; });
  };
  const X xr = make();
  Pieces<F, X> r[U];
  const uint32_t np = (K + F::kPiece - 1u) / F::kPiece;
  auto load = [&](Pieces<F, X> &b, uint32_t c) {
    xr.load(b.x, c, lane);
    F::template load<AUX>(b.w, t, w, c, lane);
    keep_order();
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int u = 0; u < U; ++u) load(r[u], wave + KS * u);
  for (uint32_t c = wave; c < np; c += KS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (XMX)
        stream_piece_mx<DW>(acc, r[u], lds + wave * kWaveLds, lane);
      else
        stream_piece<F, X>(acc, r[u], xr, lds + wave * kWaveLds, lane);
      keep_order();
      load(r[u], c + KS * (U + u));  // past the row's end: zeros, no traffic
    }
  }
  __syncthreads();
  float *red = reinterpret_cast<float *>(lds);  // the partial sums reuse the streams' LDS
  reinterpret_cast<f32x4 *>(red)[wave * 64u + lane] = acc[0] + acc[1];
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < 16u * rows; o += 64u * KS) {
    const uint32_t row = o & 15u, tok = o >> 4;
    if (n0 + row < w.N) {
      const uint32_t at = ((tok >> 2) * 16u + row) * 4u + (tok & 3u);
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) v += red[i * 256 + at];
      y[(size_t)(m0 + tok) * w.N + n0 + row] = to_bf16_bits(v);
    }
  }
}

// ---- many rows --------------------------------------------------------------------------------

constexpr uint32_t kChunk = 128;         // k of one fp4 MFMA
constexpr uint32_t kGroup = 4 * kChunk;  // k of one scale load: 16 scale bytes a row

// Tile BM rows of X times BN weight rows, WM x WN waves, steps of CH chunks.  Both
// operands are copied to LDS by DMA, two stages; 16-byte pieces of a row are
// XOR-swizzled so that the rows of an operand read fall into distinct banks.  A =
// weight rows, B = X rows: a lane's four results are neighbours in Y.
// 14336x4096: m = 512 X BF16 51.7 us in calls without a pause, 1.16 PFLOP/s (the bf16 MFMA alone
// reaches 1.66; a call on an idle GPU takes 55 to 61 us, the kernel under the tracer 60); m = 2048
// both MXFP4 83.3 us, 2.9 PFLOP/s (the fp4 MFMA alone 6.1): each product needs its operands
// from LDS once per 16 x 16 x 128, the loads of a step share the address unit, and 448 tiles are
// 1.75 rounds of the CUs.
// The narrow tiles read X once for each 32, 64 or 128 weight rows: m = 128 4096x14336 40.0 us
// (floor 11.6) with 602 MB requested from the L2s for 36, both MXFP4 20.5 us (floor 4.8) with 206.
// Scales: loaded a group ahead, a lane per row and 16 bytes (block g of chunk c at
// byte 4c + g), transposed to bytes 4g + c and put in LDS, so that a lane gets its
// row's scales of block g for all four chunks as one dword whose byte c the scaled
// MFMA selects.  (Loading each lane's own byte took 24 scattered loads a wave and
// step: 236 us instead of 83 at m = 2048 on 14336x4096.)
template <bool XMX, int BM, int BN, int WM, int WN, int CH, int KG>
struct MxTile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;  // of one K part
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16-row tiles a wave
  static constexpr uint32_t XB = (XMX ? 64u : 256u) * CH;     // bytes of an X row in a step
  static constexpr uint32_t WB = 64u * CH;
  static constexpr uint32_t X_BYTES = BM * XB, W_BYTES = BN * WB, STAGE = X_BYTES + W_BYTES;
  static constexpr uint32_t SROWS = BN + (XMX ? BM : 0);  // scale rows: the weight's, then X's
  static constexpr int NS = (int)((SROWS + kThreads - 1) / kThreads);  // scale rows a lane
  static constexpr uint32_t PART = 2u * STAGE + 2u * 16u * SROWS, LDS = KG * PART;  // LDS of a K part, of all
  static constexpr int NX = (int)(X_BYTES / 1024u / kWaves), NW = (int)(W_BYTES / 1024u / kWaves);
  static_assert(X_BYTES % (1024u * kWaves) == 0 && W_BYTES % (1024u * kWaves) == 0, "whole loads a wave");
  static_assert(CH == 1 || CH == 2, "a group is two or four steps");
  static_assert(KG == 1 || KG * (uint32_t)kThreads * 16u <= LDS, "one 16 x 16 result of every wave fits");
};

// piece index -> swizzled piece, rows of P 16-byte pieces
template <uint32_t P>
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t c) {
  if constexpr (P == 16u) return row_swizzle<16>(row, c);
  if constexpr (P == 8u) return c ^ (row & 7u);
  return c ^ ((row >> 1) & 3u);
}

template <int... N, class Body>
__device__ __forceinline__ void for_each(std::integer_sequence<int, N...>, Body &body) {
  (body(std::integral_constant<int, N>{}), ...);
}

template <int C>
__device__ __forceinline__ f32x4 mfma_mx_sel(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
  const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, C, (int)sa, C, (int)sb);
}

// 4 x 4 bytes: byte 4c + g -> 4g + c
__device__ __forceinline__ u32x4 transpose_bytes(u32x4 v) {
  const uint32_t ab02 = __builtin_amdgcn_perm(v.y, v.x, 0x06020400u), ab13 = __builtin_amdgcn_perm(v.y, v.x, 0x07030501u);
  const uint32_t cd02 = __builtin_amdgcn_perm(v.w, v.z, 0x06020400u), cd13 = __builtin_amdgcn_perm(v.w, v.z, 0x07030501u);
  return u32x4{__builtin_amdgcn_perm(cd02, ab02, 0x05040100u), __builtin_amdgcn_perm(cd13, ab13, 0x05040100u),
               __builtin_amdgcn_perm(cd02, ab02, 0x07060302u), __builtin_amdgcn_perm(cd13, ab13, 0x07060302u)};
}

template <bool XMX, int BM, int BN, int WM, int WN, int CH, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG) void k_mx_tile(MxView w, const uint8_t *__restrict__ x,
                                                          const uint8_t *__restrict__ xs, uint32_t m,
                                                          uint16_t *__restrict__ y, uint32_t mt_count) {
  using S = MxTile<XMX, BM, BN, WM, WN, CH, KG>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_all[];
  // the K part's own threads, waves and LDS
  const uint32_t part = KG == 1 ? 0u : uniform32(threadIdx.x / (uint32_t)S::kThreads);
  const uint32_t tid = threadIdx.x - part * (uint32_t)S::kThreads, lane = tid & 63u, wave = uniform32(tid >> 6);
  const uint32_t lr = lane & 15u, g = lane >> 4;
  uint8_t *const lds_mx = lds_all + part * S::PART;
  const uint32_t wm = wave % WM, wn = wave / WM, K = w.K;
  // Workgroups are dealt to the 8 XCDs in turn: give each XCD neighbouring tiles, and of
  // those 8 X tiles by as many weight tiles as run together, so that its L2 serves both
  // (BF16 X, m = 8192 16384x4096: 900 us, 1020 with all X tiles of one weight tile first).
  const uint32_t total = gridDim.x, per = total / 8u, extra = total % 8u, xcd = blockIdx.x % 8u;
  const uint32_t id = xcd * per + (xcd < extra ? xcd : extra) + blockIdx.x / 8u;
  const uint32_t nt_count = total / mt_count, band = id / (8u * nt_count), in = id - band * 8u * nt_count;
  const uint32_t high = mt_count - 8u * band < 8u ? mt_count - 8u * band : 8u;
  const uint32_t m0 = (8u * band + in % high) * BM, n0 = in / high * BN;
  const uint32_t mrows = m - m0 < BM ? m - m0 : BM, nrows = w.N - n0 < BN ? w.N - n0 : BN;
  const uint32_t xrow = XMX ? K / 2u : K * 2u, wrow = K / 2u, srow = K / 32u;  // bytes a row
  const auto rx = make_rsrc(x + (size_t)m0 * xrow, mrows * xrow);
  const auto rw = make_rsrc(w.codes + (size_t)n0 * wrow, nrows * wrow);
  const uint8_t *const wsp = w.scales + (size_t)n0 * srow, *const xsp = XMX ? xs + (size_t)m0 * srow : nullptr;
  const auto rws = make_rsrc(wsp, nrows * srow), rxs = make_rsrc(xsp, XMX ? mrows * srow : 0u);
  // scales sixteen at a time where every row of them is whole dwords
  const bool dwords = K % kChunk == 0 && ((reinterpret_cast<uintptr_t>(wsp) | reinterpret_cast<uintptr_t>(xsp)) & 3u) == 0;

  uint32_t vx[S::NX], vw[S::NW];  // byte offset of this lane's piece at step 0
  uint32_t px[S::NX], pw[S::NW];  // ... and within its row's step
#pragma unroll
  for (int j = 0; j < S::NX; ++j) {
    const uint32_t slot = (wave * S::NX + j) * 64u + lane, row = slot / (S::XB / 16u);
    px[j] = 16u * swz<S::XB / 16u>(row, slot % (S::XB / 16u));
    vx[j] = row < mrows ? row * xrow + px[j] : kOutOfRange;
  }
#pragma unroll
  for (int j = 0; j < S::NW; ++j) {
    const uint32_t slot = (wave * S::NW + j) * 64u + lane, row = slot / (S::WB / 16u);
    pw[j] = 16u * swz<S::WB / 16u>(row, slot % (S::WB / 16u));
    vw[j] = row < nrows ? row * wrow + pw[j] : kOutOfRange;
  }
  // Load j of the wave's NX + NW of a step.
  constexpr int kLoads = S::NX + S::NW;
  auto dma_one = [&](int j, uint32_t step, uint8_t *base) {
    if (j < S::NX) {
      const bool in = step * S::XB + px[j] < xrow;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (__attribute__((address_space(3))) void *)(base + (wave * S::NX + j) * 1024u),
                                               16, (int)(in ? vx[j] + step * S::XB : kOutOfRange), 0, 0, 0);
    } else {
      const int i = j - S::NX;
      const bool in = step * S::WB + pw[i] < wrow;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (__attribute__((address_space(3))) void *)(base + S::X_BYTES + (wave * S::NW + i) * 1024u), 16,
          (int)(in ? vw[i] + step * S::WB : kOutOfRange), 0, 0, 0);
    }
  };
  auto dma = [&](uint32_t step, uint8_t *base) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) dma_one(j, step, base);
  };
  auto load_scales = [&](u32x4 (&v)[S::NS], uint32_t group) {
#pragma unroll
    for (int j = 0; j < S::NS; ++j) {
      const uint32_t row = (uint32_t)S::kThreads * j + tid;
      const bool isw = row < BN;
      const uint32_t r = isw ? row : row - BN;
      const bool have = isw ? r < nrows : XMX && row < S::SROWS && r < mrows;
      const uint32_t at = r * srow + 16u * group;
      auto one = [&](const __amdgpu_buffer_rsrc_t rs, bool mine) {
        u32x4 o = {0u, 0u, 0u, 0u};
        if (dwords && srow % 16u == 0u) {
          o = buf_load_b128(rs, mine && 16u * group < srow ? at : kOutOfRange);
        } else {
#pragma unroll
          for (uint32_t c = 0; c < 4u; ++c)
            if (dwords) {
              o[c] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)(mine && 16u * group + 4u * c < srow ? at + 4u * c : kOutOfRange), 0, 0);
            } else {
#pragma unroll
              for (uint32_t i = 0; i < 4u; ++i)
                o[c] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(
                            rs, (int)(mine && 16u * group + 4u * c + i < srow ? at + 4u * c + i : kOutOfRange), 0, 0) << (8u * i);
            }
        }
        return o;
      };
      const uint32_t first = uniform32(row);  // of the wave's 64
      if (!XMX || first + 63u < BN)
        v[j] = one(rws, have);
      else if (first >= BN)
        v[j] = one(rxs, have);
      else
        v[j] = one(rws, have && isw) | one(rxs, have && !isw);
    }
  };
  uint8_t *const sbase = lds_mx + 2u * S::STAGE;
  auto put_scales = [&](const u32x4 (&v)[S::NS], uint32_t buf) {
#pragma unroll
    for (int j = 0; j < S::NS; ++j) {
      const uint32_t row = (uint32_t)S::kThreads * j + tid;
      if (S::SROWS % S::kThreads == 0 || row < S::SROWS)
        *reinterpret_cast<u32x4 *>(sbase + buf * (16u * S::SROWS) + 16u * row) = transpose_bytes(v[j]);
    }
  };
  uint32_t sw[S::TN], sx[XMX ? S::TM : 1];  // this group's: byte c is chunk c's
  auto get_scales = [&](uint32_t buf) {
    const uint8_t *at = sbase + buf * (16u * S::SROWS) + 4u * g;
#pragma unroll
    for (int t = 0; t < S::TN; ++t) sw[t] = *reinterpret_cast<const uint32_t *>(at + 16u * ((wn * S::TN + t) * 16u + lr));
    if constexpr (XMX)
#pragma unroll
      for (int t = 0; t < S::TM; ++t)
        sx[t] = *reinterpret_cast<const uint32_t *>(at + 16u * (BN + (wm * S::TM + t) * 16u + lr));
  };
  f32x4 acc[S::TN][S::TM];
#pragma unroll
  for (int i = 0; i < S::TN; ++i)
#pragma unroll
    for (int j = 0; j < S::TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The products of a step (chunks C0 .. C0 + CH - 1 of the group).  The weight operands are
  // read kAhead products of a row ahead: with the one that the compiler left by itself, four
  // products did not cover an LDS read.
  // With both operands in MXFP4 the next step's loads go out between the first half of the
  // products: issued together after the barrier, the waves' loads queue for the address unit
  // before any product starts (m = 2048 14336x4096 82 us instead of 86 with both changes).
  // BF16 products take four times as long and the compiler's own order is 3 % faster there.
  auto step_products = [&](auto tag, const uint8_t *base, uint32_t next, uint8_t *next_base) {
    constexpr int C0 = decltype(tag)::value;
    constexpr int kHalf = (CH * S::TN + 1) / 2, kPer = (kLoads + kHalf - 1) / kHalf;
    auto issue = [&](int n) {
#pragma unroll
      for (int j = n * kPer; j < (n + 1) * kPer && j < kLoads; ++j) dma_one(j, next, next_base);
    };
    const uint8_t *xb = base, *wb = base + S::X_BYTES;
    auto wread = [&](int n) {  // weight operand n of the step
      const uint32_t row = (wn * S::TN + (uint32_t)(n % S::TN)) * 16u + lr;
      return *reinterpret_cast<const u32x4 *>(wb + row * S::WB + 16u * swz<S::WB / 16u>(row, 4u * (uint32_t)(n / S::TN) + g));
    };
    constexpr int kAhead = 3, kSteps = CH * S::TN;
    u32x4 wq[kAhead];
    if constexpr (XMX) {
      u32x4 b[2][S::TM];
      auto xread = [&](int c) {
#pragma unroll
        for (int j = 0; j < S::TM; ++j) {
          const uint32_t row = (wm * S::TM + j) * 16u + lr;
          b[c & 1][j] = *reinterpret_cast<const u32x4 *>(xb + row * S::XB + 16u * swz<S::XB / 16u>(row, 4u * c + g));
        }
      };
      xread(0);
#pragma unroll
      for (int n = 0; n < kAhead && n < kSteps; ++n) wq[n] = wread(n);
      keep_order();
      auto row_products = [&](auto ntag) {
        constexpr int n = decltype(ntag)::value, c = n / S::TN, i = n % S::TN;
        const u32x4 q = wq[n % kAhead];
        if (CH > 1 && c + 1 < CH && i == S::TN / 2) xread(c + 1);
        if (n + kAhead < kSteps) wq[n % kAhead] = wread(n + kAhead);
#pragma unroll
        for (int j = 0; j < S::TM; ++j) acc[i][j] = mfma_mx_sel<C0 + c>(q, sw[i], b[c & 1][j], sx[j], acc[i][j]);
        issue(n);
        keep_order();
      };
      for_each(std::make_integer_sequence<int, kSteps>{}, row_products);
    } else {
      static_assert(CH == 1, "one chunk a step");
      dma(next, next_base);
      u32x4 b[S::TM][4];
#pragma unroll
      for (int j = 0; j < S::TM; ++j) {
        const uint32_t row = (wm * S::TM + j) * 16u + lr;
#pragma unroll
        for (int f = 0; f < 4; ++f)
          b[j][f] = *reinterpret_cast<const u32x4 *>(xb + row * S::XB + 16u * swz<S::XB / 16u>(row, 4u * g + f));
      }
#pragma unroll
      for (int i = 0; i < S::TN; ++i) {
        const u32x4 q = wread(i);
        const float sc = mx_scale_f32((sw[i] >> (8 * C0)) & 0xFFu);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const uint4 a = mx_to_bf16x8(q[f], sc);
#pragma unroll
          for (int j = 0; j < S::TM; ++j) acc[i][j] = mfma16(u32x4{a.x, a.y, a.z, a.w}, b[j][f], acc[i][j]);
        }
      }
    }
  };
  // One barrier a step.  Before it every wave has waited for its own loads of the
  // next step (all of them: DMA and register loads are never counted apart) and has
  // read its operands of this one, so after it the next stage is whole and this one
  // may be filled again.
  auto sync = [&]() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  // K part p walks groups p, p + KG, ...; all parts make the same number of steps, and
  // steps past K read zeros
  const uint32_t groups = (K + kGroup - 1u) / kGroup, rounds = (groups + KG - 1u) / KG;
  constexpr uint32_t SPG = 4 / CH;  // steps a group
  u32x4 sv[S::NS];
  load_scales(sv, part);
  dma(part * SPG, lds_mx);
  put_scales(sv, 0);
  sync();
  uint8_t *const st0 = lds_mx, *const st1 = lds_mx + S::STAGE;
  for (uint32_t i = 0; i < rounds; ++i) {
    const uint32_t q = part + KG * i;
    get_scales(i & 1u);
    if constexpr (CH == 2) {
      load_scales(sv, q + KG);
      step_products(std::integral_constant<int, 0>{}, st0, 2u * q + 1u, st1);
      sync();
      step_products(std::integral_constant<int, 2>{}, st1, 2u * (q + KG), st0);
      put_scales(sv, (i + 1u) & 1u);
      sync();
    } else {
      load_scales(sv, q + KG);
      step_products(std::integral_constant<int, 0>{}, st0, 4u * q + 1u, st1);
      sync();
      step_products(std::integral_constant<int, 1>{}, st1, 4u * q + 2u, st0);
      sync();
      step_products(std::integral_constant<int, 2>{}, st0, 4u * q + 3u, st1);
      sync();
      step_products(std::integral_constant<int, 3>{}, st1, 4u * (q + KG), st0);
      put_scales(sv, (i + 1u) & 1u);
      sync();
    }
  }
  if constexpr (KG > 1) {  // the parts' sums, added in order by part 0
    f32x4 *const red = reinterpret_cast<f32x4 *>(lds_all);
#pragma unroll
    for (int i = 0; i < S::TN; ++i)
#pragma unroll
      for (int j = 0; j < S::TM; ++j) {
        red[threadIdx.x] = acc[i][j];
        __syncthreads();
        if (part == 0) {
#pragma unroll
          for (int p = 1; p < KG; ++p) acc[i][j] += red[tid + (uint32_t)(p * S::kThreads)];
        }
        __syncthreads();
      }
    if (part != 0) return;
  }
  // D[4 g + r][lr]: weight row 4 g + r, X row lr
  const bool wide = w.N % 4u == 0u && (reinterpret_cast<uintptr_t>(y) & 7u) == 0u;
#pragma unroll
  for (int j = 0; j < S::TM; ++j) {
    const uint32_t row = (wm * S::TM + j) * 16u + lr;
    if (row >= mrows) continue;
    uint16_t *yr = y + (size_t)(m0 + row) * w.N + n0;
#pragma unroll
    for (int i = 0; i < S::TN; ++i) {
      const uint32_t n = (wn * S::TN + i) * 16u + 4u * g;
      const f32x4 v = acc[i][j];
      if (wide) {
        if (n < nrows) *reinterpret_cast<uint2 *>(yr + n) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      } else {
#pragma unroll
        for (uint32_t r = 0; r < 4u; ++r)
          if (n + r < nrows) yr[n + r] = to_bf16_bits(v[r]);
      }
    }
  }
}

template <bool XMX, bool DW, int NX, int AUX>
hipError_t launch_rows_dw(const MxView &w, const void *x, const uint8_t *xs, uint32_t m, uint16_t *y, hipStream_t stream) {
  const uint32_t groups = (m + 15u) / 16u, grid = (w.N + 15u) / 16u * groups;
  const uint32_t np = (w.K + MxFmt<DW>::kPiece - 1u) / MxFmt<DW>::kPiece;
  // Four waves share a tile's K, eight where there is at most a tile a CU and K is long
  // (us with four / eight, X BF16: m = 16 4096x14336 14.5 / 13.5, 2048x8192 9.3 / 8.3, m = 2
  // 4096x28672 17.5 / 15.4, m = 8 1024x28672 16.1 / 16.6; more tiles: m = 16 8192x8192 15.6 / 16.9,
  // 14336x4096 15.1 / 17.7; X MXFP4: m = 16 4096x14336 11.2 / 9.8, m = 1 1024x28672 15.3 / 10.1; more
  // tiles: m = 8 8192x8192 10.3 / 10.7).  The bound on K was set on long rows: on half as many pieces
  // eight waves are 5 to 10 % faster too (m = 16 2048x4096 6.1 / 5.5, m = 4 4096x4096 5.1 / 4.8).
  constexpr int U4 = !XMX && NX <= 2 ? 2 : 1;
  if (grid <= (uint32_t)device_cu_count() && np >= 16u)
    k_mx_rows<XMX, DW, 8, 1, NX, AUX><<<grid, 512, 0, stream>>>(w, x, xs, m, groups, y);
  else
    k_mx_rows<XMX, DW, 4, U4, NX, AUX><<<grid, 256, 0, stream>>>(w, x, xs, m, groups, y);
  return hipGetLastError();
}

// NX: loads that 4 NX rows of BF16 take.
template <bool XMX, int NX, int AUX>
hipError_t launch_rows(const MxView &w, const void *x, const uint8_t *xs, uint32_t m, uint16_t *y, hipStream_t stream) {
  static_assert(!XMX || NX == 1, "16 rows in MXFP4 are one tile");
  const bool dw = mx_dwords(w) && (!XMX || (reinterpret_cast<uintptr_t>(xs) & 3u) == 0);
  return dw ? launch_rows_dw<XMX, true, NX, AUX>(w, x, xs, m, y, stream) : launch_rows_dw<XMX, false, NX, AUX>(w, x, xs, m, y, stream);
}

template <bool XMX, int BM, int BN, int WM, int WN, int CH, int KG = 1>
hipError_t launch_tile(const MxView &w, const void *x, const uint8_t *xs, uint32_t m, uint16_t *y, hipStream_t stream) {
  using S = MxTile<XMX, BM, BN, WM, WN, CH, KG>;
  const uint32_t mt = (m + BM - 1u) / BM, nt = (w.N + BN - 1u) / BN;
  static LdsAllowance allowance;
  const hipError_t e = allow_lds(allowance, &k_mx_tile<XMX, BM, BN, WM, WN, CH, KG>, (int)S::LDS);
  if (e != hipSuccess) return e;
  k_mx_tile<XMX, BM, BN, WM, WN, CH, KG><<<mt * nt, S::kThreads * KG, S::LDS, stream>>>(w, (const uint8_t *)x, xs, m, y, mt);
  return hipGetLastError();
}

// 256x256 tiles with both operands in MXFP4, 128x256 with X in BF16.
template <bool XMX>
hipError_t launch_large_tile(const MxView &w, const void *x, const uint8_t *xs, uint32_t m, uint16_t *y, hipStream_t stream) {
  if constexpr (XMX)
    return launch_tile<true, 256, 256, 4, 2, 2>(w, x, xs, m, y, stream);
  else
    return launch_tile<false, 128, 256, 2, 4, 1>(w, x, xs, m, y, stream);
}

// A launch counts its threads in 32 bits and wraps without an error: the few-row form, 256 threads
// for 16 weight rows, would leave out the rows of a weight beyond 2^28.
bool rows_form_fits(uint32_t N) { return ((uint64_t)N + 15u) / 16u * 256u <= 0xFFFFFFFFull; }

template <bool XMX>
hipError_t launch_any(const MxView &w, const void *x, const uint8_t *xs, uint32_t m, uint16_t *y, hipStream_t stream) {
  if (!rows_form_fits(w.N)) return launch_large_tile<XMX>(w, x, xs, m, y, stream);
  if constexpr (XMX) {
    if (m <= 16u) return launch_rows<XMX, 1, kAuxNontemporal>(w, x, xs, m, y, stream);
  } else {
    if (m <= 4u) return launch_rows<XMX, 1, kAuxNontemporal>(w, x, xs, m, y, stream);
    if (m <= 8u) return launch_rows<XMX, 2, kAuxNontemporal>(w, x, xs, m, y, stream);
    if (m <= 16u) return launch_rows<XMX, 4, kAuxNontemporal>(w, x, xs, m, y, stream);
  }
  // More rows on small weights: a workgroup per group of 16 rows and tile, as long as that is
  // at most three workgroups a CU (us, here / 64 x 32 tiles below, X BF16 and X MXFP4:
  // two a CU, m = 256 512x14336 18.4 / 35.4 and 10.2 / 17.0; three, m = 48 4096x14336
  // 28.0 / 33.1 and 17.8 / 19.9; four, m = 128 2048x8192 23.2 / 18.4 and 13.1 / 11.6).
  const uint32_t cus = (uint32_t)device_cu_count();
  if ((m + 15u) / 16u * ((w.N + 15u) / 16u) <= 3u * cus) return launch_rows<XMX, XMX ? 1 : 4, 0>(w, x, xs, m, y, stream);
  // Small tiles where the large ones would leave half the GPU idle.  Such a launch is bound by
  // the latency of a step, so K is dealt to parts of the workgroup, and where even 64 x 64
  // tiles are no more than the CUs they are halved to 64 x 32 with four parts (us, 64 x 64 /
  // 64 x 32: X BF16 m = 128 4096x14336 46.2 / 39.6, m = 128 4096x4096 14.1 / 11.9; X MXFP4
  // 25.5 / 20.4 and 9.8 / 8.2; five parts 21.0 and 9.1).
  const uint32_t big = ((m + (XMX ? 255u : 127u)) / (XMX ? 256u : 128u)) * ((w.N + 255u) / 256u);
  const bool few = (m + 63u) / 64u * ((w.N + 63u) / 64u) <= cus;
  if (big >= cus / 2u) return launch_large_tile<XMX>(w, x, xs, m, y, stream);
  if constexpr (XMX) {
    if (few) return launch_tile<true, 64, 32, 2, 1, 2, 4>(w, x, xs, m, y, stream);
    return launch_tile<true, 64, 64, 2, 2, 2, 2>(w, x, xs, m, y, stream);
  } else {
    if (few) return launch_tile<false, 64, 32, 2, 1, 1, 4>(w, x, xs, m, y, stream);
    return launch_tile<false, 64, 128, 2, 2, 1, 2>(w, x, xs, m, y, stream);
  }
}

}  // namespace

hipError_t launch_mx_gemm(const MxView &w, const uint16_t *x, uint16_t *y, uint32_t m, hipStream_t stream) {
  if (m == 1u && token_lds<MxTok>(w.K) <= (159u << 10)) return launch_gemv(w, x, y, stream);
  return launch_any<false>(w, x, nullptr, m, y, stream);
}

hipError_t launch_mx_gemm_mx(const MxView &w, const MxView &x, uint16_t *y, hipStream_t stream) {
  return launch_any<true>(w, x.codes, x.scales, x.N, y, stream);
}

}  // namespace int8w
