// moe_layer.hip -- a whole mixture-of-experts layer for a few tokens:
//
//   p = softmax(logits[t]);  the topk experts of largest logit (ties: the lower
//   index first; an expert at -inf is never taken);
//   r_j = p_j / sum of the chosen p (renormalized) or p_j, times routed_scale;
//   y[t] = x_resid[t] + sum_j r_j  Wd_j ( silu(Wg_j x_t) * (Wu_j x_t) ).
//
// One token: two launches (k_moe1_up, k_moe1_down, token_stream.h).  More: four launches on
// one stream, up to 64 tokens a pass:
//  k_moe_route   one workgroup: each wave takes tokens.  Its result is a list of
//                segments: an expert and up to 16 of the slots (t, j) that take it.
//  k_moe_up      workgroup (segment, rows): gate and up rows are streamed once for all
//                the segment's tokens (rows_stream.h); the epilogue writes
//                h[slot] = r * silu(g) * u.
//  k_moe_down    workgroup (segment, rows): the slot's share of its token's sum, fp32.
//  k_moe_sum     the shares of a token in the order of its choices, and the residual:
//                no atomics, so the same bits each time.
// Bound: HBM, each chosen expert's three matrices once.  An expert with more than
// 16 tokens has several segments, whose further reads of its rows come from the caches
// where they run together.  Measured, up / down: 13 tokens, 64 experts of 1024x2048 in 8 bits,
// 6 each: 38.2 us (191 MB fetched, 5.0 TB/s) / 21.9 us (96 MB, 4.4 TB/s), in groups of 32 52.7 / 23.6;
// 37 tokens, 8 experts of 14336x4096 in MXFP4, 2 each: 102 us (503 MB, 4.9 TB/s) / 50 us (276 MB,
// 5.5 TB/s); one token, 8 experts of 14336x4096 in 8 bits, 2 taken: 40.0 us (250 MB, 6.2 TB/s) /
// 22.4 us (125 MB, 5.6 TB/s).  Route and sum take 4.6 to 6.3 us each, mostly the start and end of a
// launch.  Each pass of 64 tokens streams its experts again: on a prompt the weights are read
// tokens/64 times (512 tokens, 8 experts of 14336x4096 in MXFP4: 1.69 ms).
//
// h is kept in BF16 (the matrix cores' operand type): its relative rounding of at
// most 2^-8 a value, 2^-9 rms, averages out over the inner sum to about the output's own BF16
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

// grid (row blocks of I) x (segments at most): a wave has 16 gate and the same 16 up rows.
template <class F, int KW, int AUX>
__global__ __launch_bounds__(64 * KW, 4) void k_moe_up(typename F::View wg, typename F::View wu, uint32_t I, uint32_t blocks,
                                                    const uint16_t *__restrict__ x, uint32_t T, uint32_t topk,
                                                    const MoeHead *__restrict__ head, uint16_t *__restrict__ h) {
  typedef BlockStream<F, KW, 2> S;
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::kLds];
  const MoeSegment *seg = &head->seg[blockIdx.x / blocks];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), K = wg.K;
  const uint32_t n = uniform32(seg->n), e = uniform32(seg->expert);  // meaningless, and unused, past the last segment
  if (blockIdx.x / blocks >= uniform32(head->segments)) return;
  const uint32_t i0 = 16u * (blockIdx.x % blocks * KW + wave);
  S s(lds, x, T * K * 2u, K, lane, wave, [&](uint32_t i) { return i < n ? seg->slot[i] / topk * (K * 2u) : kOutOfRange; });
  s.t[0] = F::tile(wg, (uint64_t)e * I, i0 < I ? i0 : I - 1u, I, lane);  // a wave past the last row repeats it
  s.t[1] = F::tile(wu, (uint64_t)e * I, i0 < I ? i0 : I - 1u, I, lane);
  const typename F::View *const v[2] = {&wg, &wu};
  s.template run<AUX>(v, blockIdx.x);
  // D[4 g + i][row]: token i of the segment, inner row
  const uint32_t row = i0 + (lane & 15u);
  if (row >= I) return;
#pragma unroll
  for (uint32_t i = 0; i < 4u; ++i) {
    const uint32_t k = 4u * (lane >> 4) + i;
    if (k < n) {
      const uint32_t p = seg->slot[k];
      h[(size_t)p * I + row] = to_bf16_bits(head->weight[p] * silu_mul(s.acc[0][0][i] + s.acc[0][1][i], s.acc[1][0][i] + s.acc[1][1][i]));
    }
  }
}

// grid (row blocks of H) x (segments at most); out [slots, H]: the slot's share of its token's sum.
template <class F, int KW, int AUX>
__global__ __launch_bounds__(64 * KW, 4) void k_moe_down(typename F::View wd, uint32_t H, uint32_t blocks,
                                                      const uint16_t *__restrict__ h, uint32_t slots,
                                                      const MoeHead *__restrict__ head, float *__restrict__ out) {
  typedef BlockStream<F, KW, 1> S;
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::kLds];
  const MoeSegment *seg = &head->seg[blockIdx.x / blocks];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), K = wd.K;
  const uint32_t n = uniform32(seg->n), e = uniform32(seg->expert);
  if (blockIdx.x / blocks >= uniform32(head->segments)) return;
  const uint32_t n0 = 16u * (blockIdx.x % blocks * KW + wave);
  S s(lds, h, slots * K * 2u, K, lane, wave, [&](uint32_t i) { return i < n ? seg->slot[i] * (K * 2u) : kOutOfRange; });
  s.t[0] = F::tile(wd, (uint64_t)e * H, n0 < H ? n0 : H - 1u, H, lane);
  const typename F::View *const v[1] = {&wd};
  s.template run<AUX>(v, blockIdx.x);
  const uint32_t row = n0 + (lane & 15u);
  if (row >= H) return;
#pragma unroll
  for (uint32_t i = 0; i < 4u; ++i) {
    const uint32_t k = 4u * (lane >> 4) + i;
    if (k < n) out[(size_t)seg->slot[k] * H + row] = s.acc[0][0][i] + s.acc[0][1][i];
  }
}

// y[t] = x_resid[t] + the sum of the token's slots in order (a slot of weight 0 was not run).
__global__ __launch_bounds__(256) void k_moe_sum(const float *__restrict__ out, uint32_t H, uint32_t topk,
                                                 const MoeHead *__restrict__ head, const uint16_t *__restrict__ resid,
                                                 uint16_t *__restrict__ y) {
  const uint32_t t = blockIdx.y, n = blockIdx.x * 256u + threadIdx.x;
  if (n >= H) return;
  float v = 0.f;
  for (uint32_t j = 0; j < topk; ++j)
    if (head->weight[t * topk + j] != 0.f) v += out[(size_t)(t * topk + j) * H + n];
  if (head->nan[t]) v = __builtin_nanf("");
  if (resid) v += bf16_bits_to_f32(resid[(size_t)t * H + n]);
  y[(size_t)t * H + n] = to_bf16_bits(v);
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
    keep_order();
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
      keep_order();
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
  const uint32_t count = head->segments, ids = head->seg[lane < kMaxTopk ? lane : 0u].expert;
  stage.load();
  const uint32_t n = uniform32(count);
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
    keep_order();
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
      keep_order();
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

// Whether the one-token kernels' activations fit the LDS.  Beyond it a token takes the form for
// several, with one of 16 rows of the matrix products in use: 8 of 16 experts of 8192x4096 take
// 81 us in MXFP4 and 151 in 8 bits, of 8224x4096 151 and 246.
template <class F>
bool one_token_fits(uint32_t H, uint32_t I, uint32_t topk) {
  return token_lds<F>(H) <= kLdsBytes - 1024u && (uint64_t)topk * token_lds<F>(I) <= kLdsBytes - 1024u;
}

template <class F, int KW, int R>
hipError_t launch_one_up(const typename F::View &g, const typename F::View &u, const MoeArgs &m, MoeHead *head, uint16_t *h,
                         uint32_t I, uint32_t lds, hipStream_t stream) {
  auto kern = k_moe1_up<F, KW, 2, R>;
  static LdsAllowance allowance;
  if (needs_lds_allowance(lds, 0)) {
    const hipError_t e = allow_lds(allowance, kern, (int)kLdsBytes - 1024);
    if (e != hipSuccess) return e;
  }
  const uint32_t most = (uint32_t)device_cu_count(), want = (m.topk * I + KW - 1u) / KW;
  kern<<<want < most ? want : most, 64 * KW, lds, stream>>>(g, u, I, m.x, m.logits, m.logits_bf16, m.E, m.topk, m.renorm,
                                                           m.scale, head, h);
  return hipGetLastError();
}

template <class F, int KW, int KS>
hipError_t launch_one_down(const typename F::View &d, const MoeArgs &m, MoeHead *head, const uint16_t *h, uint32_t H,
                           uint32_t lds, hipStream_t stream) {
  auto kern = k_moe1_down<F, KW, 2, KS>;
  static LdsAllowance allowance;
  if (needs_lds_allowance(lds, sizeof(float[KW][2]))) {
    const hipError_t e = allow_lds(allowance, kern, (int)kLdsBytes - 1024);
    if (e != hipSuccess) return e;
  }
  const uint32_t most = (uint32_t)device_cu_count(), units = KW / KS, want = ((H + 1u) / 2u + units - 1u) / units;
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
  // One workgroup of 8 waves a CU with two segments of a pair in flight each: more waves cost
  // more to start, and a longer ring more instructions to fetch, than they bring (us with
  // 8 / 16 waves a CU: the smallest layers 15 / 18.5 and 13 / 17.6, 8x14336x4096 64 / 64; with
  // 2 / 4 / 8 segments 14.8 / 14.7 / 18.2, 12.4 / 13.0 / 15.9, 64 / 66 / 68).
  constexpr int KW = 8;
  const uint32_t lu = token_lds<F>(H), ld = m.topk * token_lds<F>(I);
  const hipError_t e = launch_one_up_r<F, KW>(g, u, m, head, h, I, lu, stream);
  if (e != hipSuccess) return e;
  const uint32_t pairs = (H + 1u) / 2u, waves = KW * (uint32_t)device_cu_count();
  if (pairs * 4u <= waves) return launch_one_down<F, KW, 4>(d, m, head, h, H, ld, stream);
  if (pairs * 2u <= waves) return launch_one_down<F, KW, 2>(d, m, head, h, H, ld, stream);
  return launch_one_down<F, KW, 1>(d, m, head, h, H, ld, stream);
}

template <class F, class One>
hipError_t launch_layer(const typename F::View &g, const typename F::View &u, const typename F::View &d, const MoeArgs &m,
                        hipStream_t stream) {
  MoeHead *head = reinterpret_cast<MoeHead *>(m.ws);
  uint16_t *h = reinterpret_cast<uint16_t *>((uint8_t *)m.ws + kMoeHeadBytes);
  const uint32_t I = g.N / m.E, H = d.N / m.E;
  if (m.tokens == 1u && one_token_fits<One>(H, I, m.topk)) return launch_one<One>(g, u, d, m, head, h, stream);
  float *out = reinterpret_cast<float *>(h + (size_t)(m.tokens < kTok ? m.tokens : kTok) * m.topk * I);
  // us with 4 / 8 waves a workgroup: 37 tokens in MXFP4 163 / 150, 4 tokens in 8 bits 249 / 303
  constexpr int KW = F::kBlockWaves;
  for (uint32_t t0 = 0; t0 < m.tokens; t0 += kTok) {
    const uint32_t T = m.tokens - t0 < kTok ? m.tokens - t0 : kTok, slots = T * m.topk;
    const uint8_t *logits = (const uint8_t *)m.logits + (size_t)t0 * m.E * (m.logits_bf16 ? 2u : 4u);
    // segments at most: one an expert taken, one more for each kSegTokens further tokens
    const uint32_t taken = slots < m.E ? slots : m.E, most = taken + (slots - taken) / kSegTokens;
    auto route = m.E <= 64u ? k_moe_route<1> : m.E <= 128u ? k_moe_route<2> : m.E <= 256u ? k_moe_route<4> : k_moe_route<8>;
    route<<<1, 1024, 0, stream>>>(logits, m.logits_bf16, T, m.E, m.topk, m.renorm, m.scale, kSegTokens, head);
    const size_t at = (size_t)t0 * H;
    const uint32_t ub = (I + 16u * KW - 1u) / (16u * KW), db = (H + 16u * KW - 1u) / (16u * KW);
    // streamed past the caches where a row is whole cache lines (else neighbouring pieces share
    // one) and experts hardly have a second segment (us past the caches / through them, in MXFP4,
    // 2 experts a token: 8 experts of 14336x4096, 16 tokens 141 / 157, 37 149 / 164, 48 163 / 175, 64
    // 218 / 215; of 4096x4096, 64 tokens, 16 experts 96 / 106, 4 73 / 66; 16 tokens, 8 of 992x1984 35 / 30;
    // in 8 bits: 8 of 14336x4096, 16 tokens 298 / 348, 48 354 / 390, 64 441 / 448)
    const bool nt = F::row_bytes(g.K) % 128u == 0 && F::row_bytes(d.K) % 128u == 0 && (T <= kSegTokens || slots <= 12u * m.E);
    if (nt) {
      k_moe_up<F, KW, kAuxNontemporal><<<ub * most, 64 * KW, 0, stream>>>(g, u, I, ub, m.x + at, T, m.topk, head, h);
      k_moe_down<F, KW, kAuxNontemporal><<<db * most, 64 * KW, 0, stream>>>(d, H, db, h, slots, head, out);
    } else {
      k_moe_up<F, KW, 0><<<ub * most, 64 * KW, 0, stream>>>(g, u, I, ub, m.x + at, T, m.topk, head, h);
      k_moe_down<F, KW, 0><<<db * most, 64 * KW, 0, stream>>>(d, H, db, h, slots, head, out);
    }
    k_moe_sum<<<dim3((H + 255u) / 256u, T), 256, 0, stream>>>(out, H, m.topk, head, m.resid ? m.resid + at : nullptr, m.y + at);
    const hipError_t e = hipGetLastError();
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
  return mx_dwords(g) && mx_dwords(u) && mx_dwords(d) ? launch_layer<MxFmt<true>, MxTok>(g, u, d, m, stream)
                                                      : launch_layer<MxFmt<false>, MxTok>(g, u, d, m, stream);
}

}  // namespace int8w
