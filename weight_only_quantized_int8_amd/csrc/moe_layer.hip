// moe_layer.hip -- a whole mixture-of-experts layer for a few tokens:
//
//   p = softmax(logits[t]);  the topk experts of largest logit (ties: the lower
//   index first; an expert at -inf is never taken);
//   r_j = p_j / sum of the chosen p (renormalized) or p_j, times routed_scale;
//   y[t] = x_resid[t] + sum_j r_j  Wd_j ( silu(Wg_j x_t) * (Wu_j x_t) ).
//
// Three launches on one stream, up to 64 tokens a pass:
//  k_moe_route   one workgroup: each wave takes tokens, and the result is written
//                as one list of the experts that any token takes, with a table
//                slot[a][t] (1 + the slot t*topk + j that takes active expert a,
//                0: none) and the slots' weights.
//  k_moe_up      workgroup (active expert, 16 inner rows): gate and up rows are
//                streamed once for all the expert's tokens (rows_stream.h); the
//                epilogue writes h[slot] = r * silu(g) * u.
//  k_moe_down    workgroup (16 output rows): the chosen experts' down rows one
//                after the other into the same fp32 accumulators, so the weighted
//                sum over experts needs no second pass and no atomics; the rows
//                of A are the tokens, and a token that does not take the expert
//                at hand has zeros there.
// Bound: HBM, each chosen expert's three matrices once.
//
// h is kept in BF16 (the matrix cores' operand type): its relative rounding of
// 2^-9 per value averages out over the inner sum to less than the output's own
// BF16 rounding.  All sums, the softmax and the routing weights are fp32.
#include "rows_stream.h"
#include "launch.h"

namespace int8w {

namespace {

constexpr uint32_t kTok = kMoePassTokens;  // tokens a pass
constexpr uint32_t kMaxE = INT8W_MAX_MOE_EXPERTS;
constexpr uint32_t kMaxTopk = INT8W_MAX_MOE_TOPK;

// Head of the workspace; h [slots, I] BF16 follows at kMoeHeadBytes.
struct MoeHead {
  uint32_t active;              // experts taken by any token
  uint32_t pad[63];
  uint32_t expert[kMaxE];       // their indices, ascending
  uint32_t nan[kTok];           // token's logits hold a NaN or +inf: its output is NaN
  float weight[kTok * kMaxTopk];  // of slot t * topk + j
  uint16_t slot[kMaxE][kTok];   // 1 + slot, by active expert and token; 0: none
};
static_assert(sizeof(MoeHead) <= kMoeHeadBytes, "workspace head");

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  return v;
}

// 16 waves; wave w routes tokens w, w + 16, ...
__global__ __launch_bounds__(1024) void k_moe_route(const void *__restrict__ logits, bool bf16, uint32_t T, uint32_t E,
                                                    uint32_t topk, bool renorm, float scale, MoeHead *__restrict__ head) {
  constexpr int R = kMaxE / 64;
  __shared__ uint16_t ids[kTok][kMaxTopk];
  __shared__ unsigned long long takers[kMaxE];  // tokens that take the expert
  __shared__ uint32_t place[kMaxE / 64 + 1];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = uniform32(tid >> 6);
  for (uint32_t e = tid; e < kMaxE; e += 1024u) takers[e] = 0ull;
  __syncthreads();
  const float ninf = -__builtin_inff();
  for (uint32_t t = wave; t < T; t += 16u) {
    float v[R];
    bool odd = false;  // NaN or +inf
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t e = 64u * r + lane;
      v[r] = ninf;
      if (e < E) {
        v[r] = bf16 ? bf16_bits_to_f32(((const uint16_t *)logits)[(size_t)t * E + e])
                    : ((const float *)logits)[(size_t)t * E + e];
        odd |= !(v[r] < __builtin_inff());
      }
    }
    const bool is_nan = __ballot(odd) != 0ull;
    float top = ninf;
#pragma unroll
    for (int r = 0; r < R; ++r) top = fmaxf(top, v[r]);
    top = wave_max(top);
    const bool none = !(top > ninf);  // every expert masked out
    float total = 0.f;
    if (!renorm) {
#pragma unroll
      for (int r = 0; r < R; ++r) total += v[r] > ninf ? expf(v[r] - top) : 0.f;
      total = wave_sum(total);
    }
    // the topk largest: one at a time, the lowest index among equals
    uint32_t my_id = 0xFFFFu;  // lane j: expert of choice j
    float my_p = 0.f;
    if (!is_nan && !none) {
      for (uint32_t j = 0; j < topk; ++j) {
        float best = ninf;
#pragma unroll
        for (int r = 0; r < R; ++r) best = fmaxf(best, v[r]);
        best = wave_max(best);
        if (!(best > ninf)) break;
        uint32_t id = kMaxE;
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
          const unsigned long long at = __ballot(v[r] == best);
          if (at) id = 64u * r + (uint32_t)__builtin_ctzll(at);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (64u * r + lane == id) v[r] = ninf;
        if (lane == j) {
          my_id = id;
          my_p = expf(best - top);
        }
      }
    }
    if (renorm) total = wave_sum(my_p);
    const float w = my_p > 0.f ? my_p / total * scale : 0.f;
    if (w == 0.f) my_id = 0xFFFFu;  // a weight of zero (underflow, scale 0): the expert adds nothing and is not run
    if (lane < topk) {
      ids[t][lane] = (uint16_t)my_id;
      head->weight[t * topk + lane] = w;
      if (my_id < kMaxE) atomicOr(&takers[my_id], 1ull << t);  // order-free
    }
    if (lane == 0) head->nan[t] = is_nan ? 1u : 0u;
  }
  __syncthreads();
  // active experts in ascending order: waves 0 .. R-1 take 64 experts each
  unsigned long long mine = 0ull, any = 0ull;
  if (wave < (uint32_t)R) {
    mine = takers[64u * wave + lane];
    any = __ballot(mine != 0ull);
    if (lane == 0) place[wave] = (uint32_t)__popcll(any);
  }
  __syncthreads();
  if (wave < (uint32_t)R) {
    uint32_t a = 0;
    for (uint32_t i = 0; i < wave; ++i) a += place[i];
    if (wave == (uint32_t)R - 1u && lane == 0) head->active = a + place[wave];
    a += (uint32_t)__popcll(any & ((1ull << lane) - 1ull));
    const uint32_t e = 64u * wave + lane;
    if (mine) {
      head->expert[a] = e;
      for (uint32_t t = 0; t < kTok; ++t) {
        uint32_t s = 0;
        if (mine >> t & 1ull)
          for (uint32_t j = 0; j < topk; ++j)
            if (ids[t][j] == e) s = t * topk + j + 1u;
        head->slot[a][t] = (uint16_t)s;
      }
    }
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

// Gate and up of 16 inner rows for the expert's n tokens, MT tiles of 16.
template <class F, int KS, int U, int MT>
__device__ __forceinline__ void up_tile(const typename F::View &wg, const typename F::View &wu, uint64_t base, uint32_t i0,
                                        uint32_t I, const uint16_t *__restrict__ x, uint32_t T, const uint16_t *list,
                                        const uint16_t *slots, uint32_t n, uint32_t topk, const float *__restrict__ weight,
                                        uint16_t *__restrict__ h, float *red, uint32_t wave, uint32_t lane) {
  const uint32_t K = wg.K;
  const typename F::Tile tg = F::tile(wg, base, i0, I, lane), tu = F::tile(wu, base, i0, I, lane);
  const auto rx = make_rsrc(x, T * K * 2u);
  uint32_t xo[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const uint32_t i = 16u * mt + (lane & 15u);
    xo[mt] = i < n ? (uint32_t)list[i] * K * 2u : kOutOfRange;
  }
  const uint32_t nc = (K + kChunk - 1u) / kChunk;
  struct Ring {
    typename F::Frag g, u;
    XFrag x[MT];
  } r[U];
  auto load = [&](Ring &b, uint32_t c) {
    F::load(b.g, tg, wg, c, lane);
    F::load(b.u, tu, wu, c, lane);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) F::load_x(b.x[mt], rx, xo[mt], c, K, lane);
  };
  f32x4 ag[MT], au[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) ag[mt] = au[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < U; ++u) load(r[u], wave + KS * u);
  for (uint32_t c = wave; c < nc; c += KS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f32x4 S[MT][4];
      F::template sums<MT>(S, r[u].x);
      F::template mac<MT>(ag, r[u].g, r[u].x, S);
      F::template mac<MT>(au, r[u].u, r[u].x, S);
      load(r[u], c + KS * (U + u));  // past the row's end: zeros, no traffic
    }
  }
  // red [wave][2 MT tiles]
  f32x4 *out = reinterpret_cast<f32x4 *>(red) + (wave * 2u * MT) * 64u + lane;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    out[(2 * mt) * 64] = ag[mt];
    out[(2 * mt + 1) * 64] = au[mt];
  }
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < 256u * MT; o += 64u * KS) {
    const uint32_t row = o & 15u, tok = (o >> 4) & 15u, mt = o >> 8, i = 16u * mt + tok;
    if (i < n && i0 + row < I) {
      const float g = red_sum<KS>(red, 2u * MT, 2u * mt, row, tok), u = red_sum<KS>(red, 2u * MT, 2u * mt + 1u, row, tok);
      const uint32_t p = slots[i] - 1u;
      h[(size_t)p * I + i0 + row] = to_bf16_bits(weight[p] * silu_mul(g, u));
    }
  }
}

// grid (16-row tiles of I, active experts at most)
template <class F, int KS, int U, int MT>
__global__ __launch_bounds__(64 * KS) void k_moe_up(typename F::View wg, typename F::View wu, uint32_t I,
                                                    const uint16_t *__restrict__ x, uint32_t T, uint32_t topk,
                                                    const MoeHead *__restrict__ head, uint16_t *__restrict__ h) {
  extern __shared__ __attribute__((aligned(16))) float moe_red[];
  __shared__ uint16_t list[kTok], slots[kTok];
  const uint32_t a = blockIdx.y, lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6);
  const uint32_t s = head->slot[a][lane];  // meaningless, and unused, for a past the active ones
  if (a >= uniform32(head->active)) return;
  const uint64_t base = (uint64_t)uniform32(head->expert[a]) * I;
  const unsigned long long on = __ballot(lane < T && s != 0u);
  const uint32_t n = (uint32_t)__popcll(on);
  if (wave == 0 && (on >> lane & 1ull)) {
    const uint32_t at = (uint32_t)__popcll(on & ((1ull << lane) - 1ull));
    list[at] = (uint16_t)lane;
    slots[at] = (uint16_t)s;
  }
  __syncthreads();
  const uint32_t i0 = 16u * blockIdx.x;
  if (MT == 1 || n <= 16u)
    up_tile<F, KS, U, 1>(wg, wu, base, i0, I, x, T, list, slots, n, topk, head->weight, h, moe_red, wave, lane);
  else if (MT == 2 || n <= 32u)
    up_tile<F, KS, U, 2>(wg, wu, base, i0, I, x, T, list, slots, n, topk, head->weight, h, moe_red, wave, lane);
  else
    up_tile<F, KS, U, 4>(wg, wu, base, i0, I, x, T, list, slots, n, topk, head->weight, h, moe_red, wave, lane);
}

// grid: 16-row tiles of H.  LDS: red, then expert[active], then slot[active][16 MT].
template <class F, int KS, int U, int MT>
__global__ __launch_bounds__(64 * KS) void k_moe_down(typename F::View wd, uint32_t H, const uint16_t *__restrict__ h,
                                                      uint32_t T, uint32_t topk, const MoeHead *__restrict__ head,
                                                      const uint16_t *__restrict__ resid, uint16_t *__restrict__ y) {
  extern __shared__ __attribute__((aligned(16))) float moe_red[];
  uint32_t *experts = reinterpret_cast<uint32_t *>(moe_red + KS * MT * 256);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), n0 = 16u * blockIdx.x, K = wd.K;
  const uint32_t active = uniform32(head->active);
  uint16_t *slot = reinterpret_cast<uint16_t *>(experts + active);
  for (uint32_t i = threadIdx.x; i < active; i += 64u * KS) experts[i] = head->expert[i];
  for (uint32_t i = threadIdx.x; i < active * 16u * MT; i += 64u * KS) {
    const uint32_t t = i % (16u * MT);
    slot[i] = t < T ? head->slot[i / (16u * MT)][t] : (uint16_t)0;
  }
  __syncthreads();
  const auto rh = make_rsrc(h, T * topk * K * 2u);
  const uint32_t nc = (K + kChunk - 1u) / kChunk;
  struct Ring {
    typename F::Frag w;
    XFrag x[MT];
  } r[U];
  // this wave's items: chunk c of active expert a, KS apart in the flat order
  uint32_t la = 0, lc = wave;
  auto load = [&](Ring &b) {
    while (lc >= nc && la < active) {
      lc -= nc;
      ++la;
    }
    const bool in = la < active;
    const uint32_t a = in ? la : 0u, c = in ? lc : nc;
    const uint32_t e = uniform32(active ? experts[a] : 0u);
    const typename F::Tile t = F::tile(wd, (uint64_t)e * H, n0, H, lane);
    F::load(b.w, t, wd, c, lane);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint32_t s = in ? slot[(a * MT + mt) * 16u + (lane & 15u)] : 0u;
      F::load_x(b.x[mt], rh, s ? (s - 1u) * K * 2u : kOutOfRange, c, K, lane);
    }
    lc += KS;
  };
  f32x4 acc[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < U; ++u) load(r[u]);
  for (uint32_t i = wave; i < active * nc; i += KS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f32x4 S[MT][4];
      F::template sums<MT>(S, r[u].x);
      F::template mac<MT>(acc, r[u].w, r[u].x, S);
      load(r[u]);
    }
  }
  f32x4 *out = reinterpret_cast<f32x4 *>(moe_red) + (wave * MT) * 64u + lane;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) out[mt * 64] = acc[mt];
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < 256u * MT; o += 64u * KS) {
    const uint32_t row = o & 15u, tok = o >> 4, n = n0 + row;
    if (tok < T && n < H) {
      float v = red_sum<KS>(moe_red, MT, tok >> 4, row, tok & 15u);
      if (head->nan[tok]) v = __builtin_nanf("");
      if (resid) v += bf16_bits_to_f32(resid[(size_t)tok * H + n]);
      y[(size_t)tok * H + n] = to_bf16_bits(v);
    }
  }
}

template <class F, int MT>
hipError_t launch_pass(const typename F::View &g, const typename F::View &u, const typename F::View &d, const MoeArgs &m,
                       MoeHead *head, uint16_t *h, uint32_t T, const uint16_t *x, const uint16_t *resid, uint16_t *y,
                       hipStream_t stream) {
  const uint32_t I = g.N / m.E, H = d.N / m.E, most = T * m.topk < m.E ? T * m.topk : m.E;
  constexpr int KU = 4, KD = 16, U = MT == 1 ? 3 : 2;
  k_moe_up<F, KU, U, MT><<<dim3((I + 15u) / 16u, most), 64 * KU, KU * 2 * MT * 1024, stream>>>(g, u, I, x, T, m.topk, head, h);
  const uint32_t lds = KD * MT * 1024 + most * (4u + 32u * MT);
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&k_moe_down<F, KD, U, MT>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  k_moe_down<F, KD, U, MT><<<(H + 15u) / 16u, 64 * KD, lds, stream>>>(d, H, h, T, m.topk, head, resid, y);
  return hipGetLastError();
}

template <class F>
hipError_t launch_layer(const typename F::View &g, const typename F::View &u, const typename F::View &d, const MoeArgs &m,
                        hipStream_t stream) {
  MoeHead *head = reinterpret_cast<MoeHead *>(m.ws);
  uint16_t *h = reinterpret_cast<uint16_t *>((uint8_t *)m.ws + kMoeHeadBytes);
  const size_t H = d.N / m.E;
  for (uint32_t t0 = 0; t0 < m.tokens; t0 += kTok) {
    const uint32_t T = m.tokens - t0 < kTok ? m.tokens - t0 : kTok;
    const uint8_t *logits = (const uint8_t *)m.logits + (size_t)t0 * m.E * (m.logits_bf16 ? 2u : 4u);
    k_moe_route<<<1, 1024, 0, stream>>>(logits, m.logits_bf16, T, m.E, m.topk, m.renorm, m.scale, head);
    const uint16_t *x = m.x + t0 * H, *resid = m.resid ? m.resid + t0 * H : nullptr;
    uint16_t *y = m.y + t0 * H;
    const hipError_t e = T <= 16u   ? launch_pass<F, 1>(g, u, d, m, head, h, T, x, resid, y, stream)
                         : T <= 32u ? launch_pass<F, 2>(g, u, d, m, head, h, T, x, resid, y, stream)
                                    : launch_pass<F, 4>(g, u, d, m, head, h, T, x, resid, y, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_moe_int8(const WeightView &g, const WeightView &u, const WeightView &d, const MoeArgs &m,
                           hipStream_t stream) {
  return g.gs == 32u ? launch_layer<Int8Fmt<true>>(g, u, d, m, stream) : launch_layer<Int8Fmt<false>>(g, u, d, m, stream);
}

hipError_t launch_moe_mx(const MxView &g, const MxView &u, const MxView &d, const MoeArgs &m, hipStream_t stream) {
  return launch_layer<MxFmt>(g, u, d, m, stream);
}

}  // namespace int8w
