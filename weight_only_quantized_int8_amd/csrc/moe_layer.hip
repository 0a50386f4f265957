// moe_layer.hip -- a whole mixture-of-experts layer for a few tokens:
//
//   p = softmax(logits[t]);  the topk experts of largest logit (ties: the lower
//   index first; an expert at -inf is never taken);
//   r_j = p_j / sum of the chosen p (renormalized) or p_j, times routed_scale;
//   y[t] = x_resid[t] + sum_j r_j  Wd_j ( silu(Wg_j x_t) * (Wu_j x_t) ).
//
// Three launches on one stream, up to 64 tokens a pass:
//  k_moe_route   one workgroup: each wave takes tokens.  Its result is a list of
//                segments: an expert and up to C of the slots (t, j) that take it.
//  k_moe_up      workgroup (segment, 16 inner rows): gate and up rows are streamed
//                once for all the segment's tokens (rows_stream.h); the epilogue
//                writes h[slot] = r * silu(g) * u.
//  k_moe_down    workgroup (16 output rows): the segments' down rows one after the
//                other, the waves sharing the list evenly; a wave adds a segment's
//                products to its own fp32 sums by token, so the weighted sum over
//                experts needs no atomics and no further pass.
// Bound: HBM, each chosen expert's three matrices once.  An expert with more than C
// tokens has several segments, whose further reads of its rows come from the caches.
//
// h is kept in BF16 (the matrix cores' operand type): its relative rounding of at
// most 2^-9 a value averages out over the inner sum to about the output's own BF16
// rounding.  All sums, the softmax and the routing weights are fp32.
#include "rows_stream.h"
#include "token_stream.h"
#include "launch.h"

namespace int8w {

namespace {

constexpr uint32_t kTok = kMoePassTokens;  // tokens a pass
constexpr uint32_t kMaxE = INT8W_MAX_MOE_EXPERTS;
constexpr uint32_t kMaxTopk = INT8W_MAX_MOE_TOPK;
constexpr uint32_t kSegTokens = 16;  // most tokens a segment

struct MoeSegment {
  uint32_t expert, n;
  uint16_t slot[kSegTokens];  // t * topk + j, n of them
};

// Head of the workspace; h [slots, I] BF16 follows at kMoeHeadBytes.
struct MoeHead {
  uint32_t segments;
  uint32_t pad[63];
  uint32_t nan[kTok];             // token's logits hold a NaN or +inf: its output is NaN
  float weight[kTok * kMaxTopk];  // of slot t * topk + j
  MoeSegment seg[kTok * kMaxTopk];
};
static_assert(sizeof(MoeHead) <= kMoeHeadBytes, "workspace head");

// Maximum over the wave, in every lane, by data-parallel moves (a shuffle through LDS costs
// over a hundred cycles, and top-k takes six a choice).
__device__ __forceinline__ float wave_max(float v) {
#define INT8W_DPP_MAX(ctrl, rows)                                                                                  \
  v = fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(v), (int)__float_as_uint(v), \
                                                                      ctrl, rows, 0xF, false)))
  INT8W_DPP_MAX(0x111, 0xF);  // row_shr:1
  INT8W_DPP_MAX(0x112, 0xF);
  INT8W_DPP_MAX(0x114, 0xF);
  INT8W_DPP_MAX(0x118, 0xF);
  INT8W_DPP_MAX(0x142, 0xA);  // row_bcast:15
  INT8W_DPP_MAX(0x143, 0xC);  // row_bcast:31
#undef INT8W_DPP_MAX
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// One wave routes one token.  Lane l holds the logits of experts l, l + 64, ...
template <int R>  // ceil(E / 64) at most
struct RouteToken {
  float v[R];
  uint32_t id;  // lane j < topk: choice j's expert (0xFFFF: none)
  float w;      // ... and weight
  __device__ __forceinline__ void load(const void *logits, bool bf16, uint32_t t, uint32_t E, uint32_t lane) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t e = 64u * r + lane;
      v[r] = -__builtin_inff();
      if (e < E)
        v[r] = bf16 ? bf16_bits_to_f32(((const uint16_t *)logits)[(size_t)t * E + e]) : ((const float *)logits)[(size_t)t * E + e];
    }
  }
  // Returns whether the logits hold a NaN or +inf (then nothing is chosen).
  __device__ __forceinline__ bool choose(uint32_t topk, bool renorm, float scale, uint32_t lane) {
    const float ninf = -__builtin_inff();
    float top = ninf;
    bool odd = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      odd |= !(v[r] < __builtin_inff());
      top = fmaxf(top, v[r]);
    }
    id = 0xFFFFu;
    w = 0.f;
    if (__ballot(odd) != 0ull) return true;
    top = wave_max(top);
    if (!(top > ninf)) return false;  // every expert masked out
    float total = 0.f, p = 0.f, best = top;
    if (!renorm) {
#pragma unroll
      for (int r = 0; r < R; ++r) total += v[r] > ninf ? expf(v[r] - top) : 0.f;
      total = token_sum(total);
    }
    for (uint32_t j = 0; j < topk && best > ninf; ++j) {  // the largest left, the lowest index among equals
      uint32_t at = kMaxE;
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        const unsigned long long is = __ballot(v[r] == best);
        if (is) at = 64u * r + (uint32_t)__builtin_ctzll(is);
      }
      float left = ninf;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (64u * r + lane == at) v[r] = ninf;
        left = fmaxf(left, v[r]);
      }
      if (lane == j) {
        id = at;
        p = best;
      }
      if (j + 1u < topk) best = wave_max(left);
    }
    p = id < kMaxE ? expf(p - top) : 0.f;
    if (renorm) total = token_sum(p);
    w = p > 0.f ? p / total * scale : 0.f;
    if (w == 0.f) id = 0xFFFFu;  // underflow, or a scale of 0: the expert adds nothing and is not run
    return false;
  }
};

// 16 waves; wave w routes tokens w, w + 16, ...; segments of up to C tokens.
template <int R>
__global__ __launch_bounds__(1024) void k_moe_route(const void *__restrict__ logits, bool bf16, uint32_t T, uint32_t E,
                                                    uint32_t topk, bool renorm, float scale, uint32_t C,
                                                    MoeHead *__restrict__ head) {
  __shared__ uint16_t ids[kTok * kMaxTopk];
  __shared__ unsigned long long takers[64 * R];  // tokens that take the expert
  __shared__ uint32_t first[64 * R];             // its first segment
  __shared__ uint32_t place[R];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = uniform32(tid >> 6);
  if (tid < 64u * R) takers[tid] = 0ull;
  __syncthreads();
  for (uint32_t t = wave; t < T; t += 16u) {
    RouteToken<R> route;
    route.load(logits, bf16, t, E, lane);
    const bool is_nan = route.choose(topk, renorm, scale, lane);
    if (lane < topk) {
      ids[t * topk + lane] = (uint16_t)route.id;
      head->weight[t * topk + lane] = route.w;
      if (route.id < kMaxE) atomicOr(&takers[route.id], 1ull << t);  // order-free
    }
    if (lane == 0) head->nan[t] = is_nan ? 1u : 0u;
  }
  __syncthreads();
  // segments in ascending order of experts: waves 0 .. R-1 take 64 experts each
  uint32_t n = 0, segs = 0, before = 0;
  if (wave < (uint32_t)R) {
    n = (uint32_t)__popcll(takers[64u * wave + lane]);
    segs = (n + C - 1u) / C;
    uint32_t sum = segs;  // inclusive prefix over the lanes
#pragma unroll
    for (uint32_t off = 1; off < 64u; off <<= 1) {
      const uint32_t up = (uint32_t)__shfl_up((int)sum, off, kWave);
      if (lane >= off) sum += up;
    }
    before = sum - segs;
    if (lane == 63u) place[wave] = sum;
  }
  __syncthreads();
  if (wave < (uint32_t)R) {
    for (uint32_t i = 0; i < wave; ++i) before += place[i];
    first[64u * wave + lane] = before;
    for (uint32_t i = 0; i < segs; ++i) {
      head->seg[before + i].expert = 64u * wave + lane;
      head->seg[before + i].n = n - i * C < C ? n - i * C : C;
    }
    if (wave == (uint32_t)R - 1u && lane == 63u) head->segments = before + segs;
  }
  __syncthreads();
  if (tid < T * topk && ids[tid] < kMaxE) {
    const uint32_t e = ids[tid], t = tid / topk;
    const uint32_t at = (uint32_t)__popcll(takers[e] & ((1ull << t) - 1ull));
    head->seg[first[e] + at / C].slot[at % C] = (uint16_t)tid;
  }
}

// Sum of the waves' accumulators, in wave order: red[wave][tile][lane] f32x4.
template <int KS>
__device__ __forceinline__ float red_sum(const float *red, uint32_t tiles, uint32_t tile, uint32_t row, uint32_t tok) {
  const uint32_t at = (tile * 64u + (tok >> 2) * 16u + row) * 4u + (tok & 3u);
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < KS; ++w) v += red[(uint32_t)w * tiles * 256u + at];
  return v;
}

// grid (16-row tiles of I, segments at most).  NX: loads that a quarter's activations take.
template <class F, int KS, int U, int NX, int AUX>
__global__ __launch_bounds__(64 * KS) void k_moe_up(typename F::View wg, typename F::View wu, uint32_t I,
                                                    const uint16_t *__restrict__ x, uint32_t T, uint32_t topk,
                                                    const MoeHead *__restrict__ head, uint16_t *__restrict__ h) {
  typedef XBf16<F, NX> X;
  constexpr uint32_t kWaveLds = stream_lds<X, 2>();
  static_assert(KS * kWaveLds >= KS * 2048u, "the partial sums reuse the stream's LDS");
  __shared__ __attribute__((aligned(16))) uint8_t lds[KS * kWaveLds];
  const MoeSegment *seg = &head->seg[blockIdx.y];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), K = wg.K, i0 = 16u * blockIdx.x;
  const uint32_t n = uniform32(seg->n), e = uniform32(seg->expert);  // meaningless, and unused, past the last segment
  if (blockIdx.y >= uniform32(head->segments)) return;
  const typename F::Tile tg = F::tile(wg, (uint64_t)e * I, i0, I, lane), tu = F::tile(wu, (uint64_t)e * I, i0, I, lane);
  const X xs(x, T * K * 2u, K, lane, [&](uint32_t i) { return i < n ? seg->slot[i] / topk * (K * 2u) : kOutOfRange; });
  const uint32_t np = (K + F::kPiece - 1u) / F::kPiece;
  Pieces<F, X, 2> r[U];
  auto load = [&](Pieces<F, X, 2> &b, uint32_t c) {
    xs.load(b.x, c, lane);
    F::template load<AUX>(b.w[0], tg, wg, c, lane);
    F::template load<AUX>(b.w[1], tu, wu, c, lane);
    keep_order();
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int u = 0; u < U; ++u) load(r[u], wave + KS * u);
  for (uint32_t c = wave; c < np; c += KS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      stream_piece<F, X, 2>(acc, r[u], xs, lds + wave * kWaveLds, lane);
      keep_order();
      load(r[u], c + KS * (U + u));  // past the row's end: zeros, no traffic
    }
  }
  __syncthreads();
  float *red = reinterpret_cast<float *>(lds);
  reinterpret_cast<f32x4 *>(red)[(wave * 2u) * 64u + lane] = acc[0];
  reinterpret_cast<f32x4 *>(red)[(wave * 2u + 1u) * 64u + lane] = acc[1];
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < 16u * n; o += 64u * KS) {
    const uint32_t row = o & 15u, tok = o >> 4;
    if (i0 + row < I) {
      const float g = red_sum<KS>(red, 2u, 0, row, tok), u = red_sum<KS>(red, 2u, 1, row, tok);
      const uint32_t p = seg->slot[tok];
      h[(size_t)p * I + i0 + row] = to_bf16_bits(head->weight[p] * silu_mul(g, u));
    }
  }
}

// grid: 16-row tiles of H.  Dynamic LDS: the streams', then the waves' sums
// [KS][tokens][16], then the segments.  ONE: a single token, whose sums stay in registers.
template <class F, int KS, int U, int NX, bool ONE, int AUX>
__global__ __launch_bounds__(64 * KS) void k_moe_down(typename F::View wd, uint32_t H, const uint16_t *__restrict__ h,
                                                      uint32_t T, uint32_t topk, const MoeHead *__restrict__ head,
                                                      const uint16_t *__restrict__ resid, uint16_t *__restrict__ y) {
  typedef XBf16<F, NX> X;
  constexpr uint32_t kWaveLds = stream_lds<X, 1>();
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  float *sums = reinterpret_cast<float *>(lds + KS * kWaveLds);  // [KS][T][16]
  MoeSegment *segs = reinterpret_cast<MoeSegment *>(sums + KS * T * 16u);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), n0 = 16u * blockIdx.x, K = wd.K;
  const uint32_t count = uniform32(head->segments);
  for (uint32_t i = threadIdx.x; i < count * (sizeof(MoeSegment) / 4u); i += 64u * KS)
    reinterpret_cast<uint32_t *>(segs)[i] = reinterpret_cast<const uint32_t *>(head->seg)[i];
  for (uint32_t i = threadIdx.x; i < KS * T * 16u; i += 64u * KS) sums[i] = 0.f;
  __syncthreads();
  const uint32_t np = (K + F::kPiece - 1u) / F::kPiece, items = count * np;
  // this wave's items: neighbouring pieces of one segment after the other
  const uint32_t i0 = (uint32_t)((uint64_t)items * wave / KS), i1 = (uint32_t)((uint64_t)items * (wave + 1u) / KS);
  uint32_t ls = 0, lp = 0;  // segment and piece of the next load
  typename F::Tile tile = {};
  X xs(h, T * topk * K * 2u, K, lane, [&](uint32_t) { return kOutOfRange; });
  auto segment = [&](uint32_t s) {
    const MoeSegment &g = segs[s];
    tile = F::tile(wd, (uint64_t)uniform32(g.expert) * H, n0, H, lane);
    const uint32_t n = g.n;
    xs = X(h, T * topk * K * 2u, K, lane, [&](uint32_t i) { return i < n ? g.slot[i] * (K * 2u) : kOutOfRange; });
  };
  if (i0 < i1) {
    ls = i0 / np;
    lp = i0 - ls * np;
    segment(ls);
  }
  uint32_t cs = ls, cp = lp;  // ... of the next products
  Pieces<F, X, 1> r[U];
  uint32_t next = i0;
  auto load = [&](Pieces<F, X, 1> &b) {
    if (lp == np) {
      lp = 0;
      if (++ls < count) segment(ls);
    }
    const uint32_t p = next < i1 ? lp : np;  // piece np: past the row's end, zeros
    xs.load(b.x, p, lane);
    F::template load<AUX>(b.w[0], tile, wd, p, lane);
    ++lp;
    ++next;
    keep_order();
  };
  f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
  auto flush = [&](uint32_t s) {  // D[4 g + i][row]: token i of the segment, output row
    const uint32_t n = segs[s].n;
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
      const uint32_t k = 4u * (lane >> 4) + i;
      if (k < n) sums[(wave * T + segs[s].slot[k] / topk) * 16u + (lane & 15u)] += acc[0][i];
    }
    acc[0] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(r[u]);
  for (uint32_t i = i0; i < i1;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      stream_piece<F, X, 1>(acc, r[u], xs, lds + wave * kWaveLds, lane);
      keep_order();
      load(r[u]);
      ++i;
      if (!ONE && i <= i1 && (++cp == np || i == i1)) {
        flush(cs);
        cp = 0;
        ++cs;
      }
    }
  }
  if (ONE && lane < 16u) sums[wave * 16u + lane] = acc[0][0];
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < 16u * T; o += 64u * KS) {
    const uint32_t row = o & 15u, tok = o >> 4, n = n0 + row;
    if (n < H) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < KS; ++w) v += sums[((uint32_t)w * T + tok) * 16u + row];
      if (head->nan[tok]) v = __builtin_nanf("");
      if (resid) v += bf16_bits_to_f32(resid[(size_t)tok * H + n]);
      y[(size_t)tok * H + n] = to_bf16_bits(v);
    }
  }
}

// ---- one token --------------------------------------------------------------------------------
// Two launches: each wave of the first routes the token itself (a few hundred cycles, against
// a launch of its own), so that no kernel has to come before the first weight load.

// Waves share the gate/up row pairs of the chosen experts evenly.  LDS: x.
template <class F, int KW, int U, int R>
__global__ __launch_bounds__(64 * KW) void k_moe1_up(typename F::View wg, typename F::View wu, uint32_t I,
                                                     const uint16_t *__restrict__ x, const void *__restrict__ logits,
                                                     bool bf16, uint32_t E, uint32_t topk, bool renorm, float scale,
                                                     MoeHead *__restrict__ head, uint16_t *__restrict__ h) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), K = wg.K, segs = token_segs<F>(K);
  RouteToken<R> route;
  route.load(logits, bf16, 0, E, lane);
  TokenStage<F> stage(x, K, 1u, threadIdx.x, 64u * KW);
  stage.load();
  const bool is_nan = route.choose(topk, renorm, scale, lane);
  const uint32_t id = route.id;
  const float w = route.w;
  const uint32_t n = (uint32_t)__popcll(__ballot(id < kMaxE));  // choices 0 .. n-1: their weights fall
  if (blockIdx.x == 0 && wave == 0) {
    if (lane < topk) {
      head->seg[lane].expert = id;
      head->seg[lane].n = 1u;
    }
    if (lane == 0) {
      head->segments = n;
      head->nan[0] = is_nan ? 1u : 0u;
    }
  }
  const uint32_t units = gridDim.x * KW, unit = blockIdx.x * KW + wave, pairs = n * I;
  const uint32_t p0 = (uint32_t)((uint64_t)pairs * unit / units), p1 = (uint32_t)((uint64_t)pairs * (unit + 1u) / units);
  uint32_t lj = p0 / I, li = p0 - lj * I, ls = 0, left = (p1 - p0) * segs;  // the next load
  typename F::Row rg, ru;
  auto rows = [&]() {
    const bool have = lj < n;
    const uint64_t r = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)id, (int)(have ? lj : 0u)) * I + li;
    rg = F::row(wg, have ? r : 0u, have);
    ru = F::row(wu, have ? r : 0u, have);
  };
  rows();
  TokenPair<F> ring[U];
  auto load = [&](TokenPair<F> &t) {
    const uint32_t s = left ? ls : segs;  // segment segs: past the row's end, zeros
    F::load(t.a, rg, wg, s, lane);
    F::load(t.b, ru, wu, s, lane);
    token_order();
    if (left) {
      --left;
      if (++ls == segs) {
        ls = 0;
        if (++li == I) {
          li = 0;
          ++lj;
        }
        rows();
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(ring[u]);
  stage.finish(lds);
  __syncthreads();
  uint32_t cp = p0, cs = 0;
  float g = 0.f, up = 0.f;
  for (uint32_t i = 0, items = (p1 - p0) * segs; i < items; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < items) {
        u32x4 xv[F::kX];
        float xsum;
        get_token<F>(xv, xsum, lds, segs, cs, lane);
        g = F::dot(g, ring[u].a, xv, xsum);
        up = F::dot(up, ring[u].b, xv, xsum);
        if (++cs == segs) {
          cs = 0;
          const float gs = token_sum(g), us = token_sum(up);
          const uint32_t j = cp / I;
          const float r = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(w), (int)j));
          if (lane == 0) h[cp] = to_bf16_bits(r * silu_mul(gs, us));
          g = up = 0.f;
          ++cp;
        }
      }
      token_order();
      load(ring[u]);
    }
  }
}

// Waves share the pairs of output rows; KS neighbouring waves share a pair's experts and
// segments where there are few pairs.  LDS: h of the chosen experts.
template <class F, int KW, int U, int KS>
__global__ __launch_bounds__(64 * KW) void k_moe1_down(typename F::View wd, uint32_t H, const uint16_t *__restrict__ h,
                                                       uint32_t topk, const MoeHead *__restrict__ head,
                                                       const uint16_t *__restrict__ resid, uint16_t *__restrict__ y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ float red[KW][2];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), K = wd.K, segs = token_segs<F>(K);
  // the rows of h past the last chosen expert's hold nothing, and are not used
  TokenStage<F> stage(h, K, topk, threadIdx.x, 64u * KW);
  const uint32_t n = uniform32(head->segments), ids = head->seg[lane < kMaxTopk ? lane : 0u].expert;
  stage.load();
  const uint32_t units = gridDim.x * (KW / KS), unit = blockIdx.x * (KW / KS) + wave / KS, ks = wave % KS;
  const uint32_t pairs = (H + 1u) / 2u;
  const uint32_t p0 = (uint32_t)((uint64_t)pairs * unit / units), p1 = (uint32_t)((uint64_t)pairs * (unit + 1u) / units);
  const uint32_t q0 = n * segs * ks / KS, q1 = n * segs * (ks + 1u) / KS;  // the wave's share of a pair
  const uint32_t j0 = q0 / segs, s0 = q0 - j0 * segs;
  uint32_t lp = p0, lq = q0, lj = j0, ls = s0;  // the next load
  typename F::Row ra, rb;
  auto rows = [&]() {
    const bool have = lp < p1 && lj < n;
    const uint64_t r = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)ids, (int)(have ? lj : 0u)) * H + 2u * lp;
    ra = F::row(wd, have ? r : 0u, have);
    rb = F::row(wd, have && 2u * lp + 1u < H ? r + 1u : 0u, have && 2u * lp + 1u < H);
  };
  rows();
  TokenPair<F> ring[U];
  auto load = [&](TokenPair<F> &t) {
    F::load(t.a, ra, wd, ls, lane);
    F::load(t.b, rb, wd, ls, lane);
    token_order();
    ++lq;
    if (++ls == segs || lq == q1) {
      ls = 0;
      ++lj;
      if (lq >= q1) {
        ++lp;
        lq = q0;
        lj = j0;
        ls = s0;
      }
      rows();
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(ring[u]);
  const uint32_t stride = token_lds<F>(K);
  stage.finish(lds);
  __syncthreads();
  float a = 0.f, b = 0.f;
  uint32_t cp = p0, cq = q0, cj = j0, cs = s0;
  auto store = [&](uint32_t p, float va, float vb) {
    const uint32_t r = 2u * p + lane;
    if (lane < 2u && r < H) {
      float v = lane ? vb : va;
      if (head->nan[0]) v = __builtin_nanf("");
      if (resid) v += bf16_bits_to_f32(resid[r]);
      y[r] = to_bf16_bits(v);
    }
  };
  for (uint32_t i = 0, items = (p1 - p0) * (q1 - q0); i < items; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < items) {
        u32x4 xv[F::kX];
        float xsum;
        get_token<F>(xv, xsum, lds + cj * stride, segs, cs, lane);
        a = F::dot(a, ring[u].a, xv, xsum);
        b = F::dot(b, ring[u].b, xv, xsum);
        if (++cs == segs) {
          cs = 0;
          ++cj;
        }
        if (++cq == q1) {
          cq = q0;
          cj = j0;
          cs = s0;
          if constexpr (KS == 1) {
            store(cp, token_sum(a), token_sum(b));
            a = b = 0.f;
          }
          ++cp;
        }
      }
      token_order();
      load(ring[u]);
    }
  }
  if (KS == 1 && n == 0u)  // no expert taken
    for (uint32_t p = p0; p < p1; ++p) store(p, 0.f, 0.f);
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

constexpr uint32_t kLdsBytes = 160u << 10;

// Whether the one-token kernels' activations fit the LDS.
template <class F>
bool one_token_fits(uint32_t H, uint32_t I, uint32_t topk) {
  return token_lds<F>(H) <= kLdsBytes - 1024u && (uint64_t)topk * token_lds<F>(I) <= kLdsBytes - 1024u;
}

template <class K>
hipError_t allow_lds(K kernel, uint32_t lds) {
  if (lds <= 64u << 10) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
}

template <class F, int KW, int R>
hipError_t launch_one_up(const typename F::View &g, const typename F::View &u, const MoeArgs &m, MoeHead *head, uint16_t *h,
                         uint32_t I, uint32_t lds, hipStream_t stream) {
  auto kern = k_moe1_up<F, KW, 4, R>;
  hipError_t e = allow_lds(kern, lds);
  if (e != hipSuccess) return e;
  const uint32_t cus = (uint32_t)device_cu_count(), want = (m.topk * I + KW - 1u) / KW, most = cus * 16u / KW;
  kern<<<want < most ? want : most, 64 * KW, lds, stream>>>(g, u, I, m.x, m.logits, m.logits_bf16, m.E, m.topk, m.renorm,
                                                           m.scale, head, h);
  return hipGetLastError();
}

template <class F, int KW, int KS>
hipError_t launch_one_down(const typename F::View &d, const MoeArgs &m, MoeHead *head, const uint16_t *h, uint32_t H,
                           uint32_t lds, hipStream_t stream) {
  auto kern = k_moe1_down<F, KW, 4, KS>;
  hipError_t e = allow_lds(kern, lds);
  if (e != hipSuccess) return e;
  const uint32_t cus = (uint32_t)device_cu_count(), units = KW / KS, want = ((H + 1u) / 2u + units - 1u) / units;
  const uint32_t most = cus * 16u / KW;
  kern<<<KS > 1 || want < most ? want : most, 64 * KW, lds, stream>>>(d, H, h, m.topk, head, m.resid, m.y);
  return hipGetLastError();
}

template <class F, int KW>
hipError_t launch_one_up_r(const typename F::View &g, const typename F::View &u, const MoeArgs &m, MoeHead *head,
                           uint16_t *h, uint32_t I, uint32_t lds, hipStream_t stream) {
  return m.E <= 64u ? launch_one_up<F, KW, 1>(g, u, m, head, h, I, lds, stream)
                    : m.E <= 128u ? launch_one_up<F, KW, 2>(g, u, m, head, h, I, lds, stream)
                                  : launch_one_up<F, KW, 8>(g, u, m, head, h, I, lds, stream);
}

template <class F>
hipError_t launch_one(const typename F::View &g, const typename F::View &u, const typename F::View &d, const MoeArgs &m,
                      MoeHead *head, uint16_t *h, hipStream_t stream) {
  const uint32_t I = g.N / m.E, H = d.N / m.E;
  // two workgroups of 8 waves a CU where their LDS allows, else one of 16
  const uint32_t lu = token_lds<F>(H), ld = m.topk * token_lds<F>(I), half = kLdsBytes / 2u - 1024u;
  const hipError_t e = lu <= half ? launch_one_up_r<F, 8>(g, u, m, head, h, I, lu, stream)
                                  : launch_one_up_r<F, 16>(g, u, m, head, h, I, lu, stream);
  if (e != hipSuccess) return e;
  const uint32_t pairs = (H + 1u) / 2u, waves = 16u * (uint32_t)device_cu_count();
  if (ld > half) return launch_one_down<F, 16, 1>(d, m, head, h, H, ld, stream);
  if (pairs * 4u <= waves) return launch_one_down<F, 8, 4>(d, m, head, h, H, ld, stream);
  if (pairs * 2u <= waves) return launch_one_down<F, 8, 2>(d, m, head, h, H, ld, stream);
  return launch_one_down<F, 8, 1>(d, m, head, h, H, ld, stream);
}

template <class F, int NX, bool ONE>
hipError_t launch_pass(const typename F::View &g, const typename F::View &u, const typename F::View &d, const MoeArgs &m,
                       MoeHead *head, uint16_t *h, uint32_t T, uint32_t most, const uint16_t *x, const uint16_t *resid,
                       uint16_t *y, hipStream_t stream) {
  const uint32_t I = g.N / m.E, H = d.N / m.E;
  constexpr int KU = 4, KD = NX == 1 ? 16 : 8, U = NX == 1 ? 2 : 1, AUX = ONE ? kAuxNontemporal : 0;
  k_moe_up<F, KU, U, NX, AUX><<<dim3((I + 15u) / 16u, most), 64 * KU, 0, stream>>>(g, u, I, x, T, m.topk, head, h);
  const uint32_t lds = KD * (stream_lds<XBf16<F, NX>, 1>() + T * 64u) + most * (uint32_t)sizeof(MoeSegment);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&k_moe_down<F, KD, U, NX, ONE, AUX>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  k_moe_down<F, KD, U, NX, ONE, AUX><<<(H + 15u) / 16u, 64 * KD, lds, stream>>>(d, H, h, T, m.topk, head, resid, y);
  return hipGetLastError();
}

template <class F, class One>
hipError_t launch_layer(const typename F::View &g, const typename F::View &u, const typename F::View &d, const MoeArgs &m,
                        hipStream_t stream) {
  MoeHead *head = reinterpret_cast<MoeHead *>(m.ws);
  uint16_t *h = reinterpret_cast<uint16_t *>((uint8_t *)m.ws + kMoeHeadBytes);
  const size_t H = d.N / m.E;
  if (m.tokens == 1u && one_token_fits<One>((uint32_t)H, g.N / m.E, m.topk)) return launch_one<One>(g, u, d, m, head, h, stream);
  for (uint32_t t0 = 0; t0 < m.tokens; t0 += kTok) {
    const uint32_t T = m.tokens - t0 < kTok ? m.tokens - t0 : kTok, slots = T * m.topk;
    const uint8_t *logits = (const uint8_t *)m.logits + (size_t)t0 * m.E * (m.logits_bf16 ? 2u : 4u);
    // tokens a segment: the rows of one activation load where experts have few tokens
    constexpr uint32_t kOne = 64u / F::kXChunks;
    const bool few = T <= kOne || slots <= m.E * (kOne / 2u);
    const uint32_t C = few ? kOne : kSegTokens;
    // segments at most: one an expert taken, one more for each C further tokens
    const uint32_t taken = slots < m.E ? slots : m.E, most = taken + (slots - taken) / C;
    auto route = m.E <= 64u ? k_moe_route<1> : m.E <= 128u ? k_moe_route<2> : m.E <= 256u ? k_moe_route<4> : k_moe_route<8>;
    route<<<1, 1024, 0, stream>>>(logits, m.logits_bf16, T, m.E, m.topk, m.renorm, m.scale, C, head);
    const uint16_t *x = m.x + t0 * H, *resid = m.resid ? m.resid + t0 * H : nullptr;
    uint16_t *y = m.y + t0 * H;
    const hipError_t e = T == 1u ? launch_pass<F, 1, true>(g, u, d, m, head, h, T, most, x, resid, y, stream)
                         : few   ? launch_pass<F, 1, false>(g, u, d, m, head, h, T, most, x, resid, y, stream)
                                 : launch_pass<F, kSegTokens / kOne, false>(g, u, d, m, head, h, T, most, x, resid, y, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_moe_int8(const WeightView &g, const WeightView &u, const WeightView &d, const MoeArgs &m,
                           hipStream_t stream) {
  return g.gs == 32u ? launch_layer<Int8Fmt<true>, Int8Tok>(g, u, d, m, stream) : launch_layer<Int8Fmt<false>, Int8Tok>(g, u, d, m, stream);
}

hipError_t launch_moe_mx(const MxView &g, const MxView &u, const MxView &d, const MoeArgs &m, hipStream_t stream) {
  return launch_layer<MxFmt, MxTok>(g, u, d, m, stream);
}

}  // namespace int8w
