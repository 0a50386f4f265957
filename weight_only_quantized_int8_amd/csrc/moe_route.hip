// moe_route.hip -- the routing to experts by itself: scores, choice, weights.
//
//   s = softmax(l) or 1 / (1 + e^-l);  c = s + bias, or l without a bias;  of the groups of experts
//   the best topk_groups by their largest c or the sum of the two largest s + bias;  in them the
//   topk largest c, the lower index first among equals;  weight = scale s [/ sum of the taken s].
//
// A wave routes a token: lane l holds experts l R .. l R + R - 1.  A candidate is one 32-bit integer:
// the upper bits of c in an order that integers have, the expert in the lower bits (the lower index as
// the larger value), so that the lanes sort theirs by minima and maxima and top-k is topk times a maximum over
// the lanes' first ones and a step in the lane that had it.
// Which experts are taken must not hang on how a score was rounded or cut off: scores are formed within
// a known error (below), and a token with two values too near to tell is done again in fp64.
//
// Bound: a launch up to some thousand tokens, then the vector ALUs' issue.  us, under a tracer: 1 token of 64
// experts 3.1, 131 of 60 3.6, 64 of 256 in 8 groups 5.6, 16384 of those 22 (17.8 MB, which a copy moves in 3.6; about
// 590 vector instructions a token, most of them in the groups' and the choices' maxima over the lanes).
// All in fp64 16384 tokens took 35.
#include "rows_stream.h"
#include "wave_ops.h"

namespace int8w {

namespace {

constexpr uint32_t kRouteWaves = 4;

// Errors of the fp32 scores, with the hardware's 2^x and reciprocal (a unit of 2^-23 each):
//  sigmoid  e^-l is within (1 + |l|) 2^-23 of itself, s within s (1 - s) times that and 1.5 units more: since
//           s (1 - s) |l| < 1/4, within 2^-22;
//  softmax  e^(l - top) within (1 + |l - top|) 2^-22, and the sum of up to 512 of them, whose mean of
//           |l - top| so weighted is below 2 ln 512, within 2^-18.5: s within 2^-18 of the largest s.
// c adds 2^-24 of itself, a sum of two adds up theirs.  Two values further apart than twice that and a margin
// are in their true order.
__device__ __forceinline__ float score_margin(bool sigmoid, float top_score) { return sigmoid ? 0x1p-20f : 0x1p-16f * top_score; }
constexpr float kMarginOf = 0x1p-21f;  // ... and this part of the values' magnitudes

// Integers in the order of floats (no NaN), and back.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int)~k >> 31) | 0x80000000u));
}
// Maximum over the wave: over rows of 16 lanes by data-parallel moves, which are part of the maximum's own
// instruction where lanes without a source give 0, over the four rows on the scalar unit.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max<0x111>(v);  // row_shr:1
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 15), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 31);
  const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 47), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  uint32_t x = a > b ? a : b, y = c > d ? c : d;
  x = x > y ? x : y;
  return uniform32(x);
}

__device__ __forceinline__ double score64(float l, bool sigmoid, float top, double total) {
  if (!(l > -__builtin_inff())) return 0.0;
  return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / total;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}
__device__ __forceinline__ float lane_value(float v, uint32_t lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), (int)lane));
}

// The two largest of the group: merged with another lane's by a data-parallel move.
template <int CTRL>
__device__ __forceinline__ void merge_top2(float &one, float &two) {
  const float o1 = dpp_or_self<CTRL, 0xF>(one), o2 = dpp_or_self<CTRL, 0xF>(two);
  two = fmaxf(fmaxf(two, o2), fminf(one, o1));
  one = fmaxf(one, o1);
}

// LDS of a wave.
template <int R>
struct RouteLds {
  float logit[64 * R];
  float c[64 * R];  // for groups that are not a power of two lanes
  double wide[64 * R];
  uint32_t order[64];
};

// In fp64 throughout.  id: lane j < topk its expert; returns how many are taken.
template <int R>
__device__ __forceinline__ uint32_t choose64(const RouteArgs &a, const float (&v)[R], const float (&b)[R], bool biased, float top,
                                          double total, uint32_t lane, RouteLds<R> &lds, uint32_t &id) {
  const double ninf = -__builtin_inf();
  double c[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const double s = score64(v[r], a.sigmoid, top, total) + (double)b[r];  // what groups of two are scored by
    lds.wide[R * lane + r] = v[r] > -__builtin_inff() ? (biased || a.top2 ? s : (double)v[r]) : ninf;
    c[r] = v[r] > -__builtin_inff() ? (biased ? s : (double)v[r]) : ninf;
  }
  wave_fence();
  if (a.groups > 1u) {
    const uint32_t size = a.group_size;
    double one = ninf, two = ninf;  // lane g: of group g
    if (lane < a.groups)
      for (uint32_t i = 0, e = lane % size; i < size; ++i) {  // each lane from its own start: banks
        const double x = lds.wide[lane * size + e];
        two = fmax(two, fmin(one, x));
        one = fmax(one, x);
        if (++e == size) e = 0;
      }
    double of = a.top2 && two > ninf ? one + two : one;
    unsigned long long stay = 0ull;
    for (uint32_t j = 0; j < a.topk_groups; ++j) {
      const double best = wave_max(of);
      if (!(best > ninf)) break;
      const uint32_t g = (uint32_t)__builtin_ctzll(__ballot(of == best));
      stay |= 1ull << g;
      if (lane == g) of = ninf;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t g = (R * lane + r) * a.group_magic >> 20;  // e / size
      if (g >= a.groups || !(stay >> g & 1ull)) c[r] = ninf;
    }
  }
  id = INT8W_NO_EXPERT;
  uint32_t n = 0;
  for (; n < a.topk; ++n) {
    double left = ninf;
#pragma unroll
    for (int r = 0; r < R; ++r) left = fmax(left, c[r]);
    const double best = wave_max(left);
    if (!(best > ninf)) break;
    const uint32_t from = (uint32_t)__builtin_ctzll(__ballot(left == best));
    uint32_t at = 0;
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
      if (c[r] == best) at = r;
    if (lane == from) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if ((uint32_t)r == at) c[r] = ninf;
    }
    at = R * from + (uint32_t)__builtin_amdgcn_readlane((int)at, (int)from);
    if (lane == n) id = at;
  }
  return n;
}

template <int R>
__device__ __forceinline__ void load_values(float (&v)[R], const void *from, bool bf16, size_t at, uint32_t n, bool whole) {
  // n of the R values exist; whole: n is R or 0, and the values are aligned for one access
  if (bf16) {
    const uint16_t *const p = (const uint16_t *)from + at;
    if constexpr (R > 1) {
      if (whole) {
        typedef uint16_t Vec __attribute__((ext_vector_type(R)));
        const Vec w = n ? *reinterpret_cast<const Vec *>(p) : (Vec)0xFF80;
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = bf16_bits_to_f32(w[r]);
        return;
      }
    }
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) v[r] = r < n ? bf16_bits_to_f32(p[r]) : -__builtin_inff();
  } else {
    const float *const p = (const float *)from + at;
    if constexpr (R > 1) {
      if (whole) {
        typedef float Vec __attribute__((ext_vector_type(R)));
        const Vec w = n ? *reinterpret_cast<const Vec *>(p) : (Vec)(-__builtin_inff());
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = w[r];
        return;
      }
    }
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) v[r] = r < n ? p[r] : -__builtin_inff();
  }
}

// R: ceil(E / 64) at most.
template <int R, bool BIASED>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(const RouteArgs a) {
  __shared__ RouteLds<R> all[kRouteWaves];
  const float ninf = -__builtin_inff();
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), E = a.E;
  const uint32_t t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.tokens) return;
  RouteLds<R> &lds = all[wave];
  const uint32_t e0 = R * lane, have = e0 >= E ? 0u : E - e0 < R ? E - e0 : R;
  float v[R], b[R] = {}, top = ninf;
  load_values<R>(v, a.logits, a.logits_bf16, (size_t)t * E + (have ? e0 : 0u), have, a.whole);
  if constexpr (BIASED) load_values<R>(b, a.bias, false, have ? e0 : 0u, have, a.whole_bias);
  bool odd = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if ((uint32_t)r >= have) b[r] = 0.f;
    odd |= (a.sigmoid ? v[r] != v[r] : !(v[r] < __builtin_inff())) || b[r] != b[r];
    top = fmaxf(top, v[r]);
    lds.logit[e0 + r] = v[r];
  }
  odd = __ballot(odd) != 0ull;
  const bool sums = a.groups > 1u && a.top2;
  if (!a.sigmoid) top = wave_max(top);
  // fp32 scores, where anything goes by them
  float s[R], top_score = 1.f;
  if (BIASED || sums) {
    if (a.sigmoid) {
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = __builtin_amdgcn_rcpf(1.f + __expf(-v[r]));
    } else {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = v[r] > ninf ? __expf(v[r] - top) : 0.f;
        sum += s[r];
      }
      top_score = __builtin_amdgcn_rcpf(wave_add(sum));
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] *= top_score;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = v[r] > ninf ? s[r] + b[r] : ninf;
  }
  float c[R];
#pragma unroll
  for (int r = 0; r < R; ++r) c[r] = BIASED ? s[r] : v[r] + 0.f;  // -0 is 0: equal as floats, and not as the integers below
  const float margin = score_margin(a.sigmoid, top_score);
  bool near = false;  // two values that cannot be told apart
  if (a.groups > 1u) {
    float one = ninf, two = ninf;
    if (a.group_lanes) {  // a group is a power of two lanes
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float x = BIASED || sums ? s[r] : c[r];
        two = fmaxf(two, fminf(one, x));
        one = fmaxf(one, x);
      }
      if (a.group_lanes > 1u) merge_top2<0xB1>(one, two);   // lane ^ 1
      if (a.group_lanes > 2u) merge_top2<0x4E>(one, two);   // lane ^ 2
      if (a.group_lanes > 4u) merge_top2<0x141>(one, two);  // lane ^ 7, quads being alike
      if (a.group_lanes > 8u) merge_top2<0x140>(one, two);  // lane ^ 15
      if (a.group_lanes > 16u) {
        const float o1 = __shfl_xor(one, 16, kWave), o2 = __shfl_xor(two, 16, kWave);
        two = fmaxf(fmaxf(two, o2), fminf(one, o1));
        one = fmaxf(one, o1);
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) lds.c[e0 + r] = BIASED || sums ? s[r] : c[r];
      wave_fence();
      const uint32_t size = a.group_size;
      if (lane < a.groups)
        for (uint32_t i = 0, e = lane % size; i < size; ++i) {  // each lane from its own start: banks
          const float x = lds.c[lane * size + e];
          two = fmaxf(two, fminf(one, x));
          one = fmaxf(one, x);
          if (++e == size) e = 0;
        }
    }
    const float of = sums && two > ninf ? one + two : one;
    near |= sums && two > ninf && one < __builtin_inff() && fabsf(of) == __builtin_inff();  // a sum past fp32's range, not fp64's
    const float size_of = of > ninf ? fabsf(one) + (sums && two > ninf ? fabsf(two) : 0.f) : 0.f;
    const uint32_t lanes = a.group_lanes ? a.group_lanes : 1u, own = lane / lanes;
    const float apart = 2.f * margin;
    unsigned long long stay = 0ull;  // groups
    if (a.groups <= 8u) {            // lane 8 g + h compares groups g and h
      const uint32_t g = lane >> 3, h = lane & 7u;
      const float x = __shfl(of, (int)(g * lanes), kWave), y = __shfl(of, (int)(h * lanes), kWave);
      const bool both = g < a.groups && h < a.groups;
      const unsigned long long before = __ballot(both && (y > x || (y == x && h < g)));  // byte g: the groups before g
      if (BIASED || sums) {
        const float m = __shfl(size_of, (int)(g * lanes), kWave) + __shfl(size_of, (int)(h * lanes), kWave);
        near |= both && g != h && y > ninf && fabsf(y - x) <= apart + kMarginOf * m;
      }
      const bool keep = lane < a.groups && (uint32_t)__popcll(before >> (8u * (lane & 7u)) & 0xFFull) < a.topk_groups;
      stay = __ballot(keep);
    } else {
      uint32_t before = 0;  // groups before this lane's
      for (uint32_t g = 0; g < a.groups; ++g) {
        const float other = lane_value(of, g * lanes);
        before += other > of || (other == of && g < own) ? 1u : 0u;
        if (BIASED || sums)
          near |= g != own && own < a.groups && other > ninf && fabsf(other - of) <= apart + kMarginOf * (size_of + lane_value(size_of, g * lanes));
      }
      const unsigned long long keep = __ballot(own < a.groups && before < a.topk_groups);  // by lanes
      for (uint32_t g = 0; g < a.groups; ++g) stay |= (keep >> (g * lanes) & 1ull) << g;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t g = a.group_lanes ? own : (e0 + r) * a.group_magic >> 20;  // e / size
      if (g >= a.groups || !(stay >> g & 1ull)) c[r] = ninf;
    }
  }
  // The lower bits of a candidate; 0: none.  BF16 logits themselves have nothing in their lower 16 bits: the whole
  // index fits, and nothing is lost.  Otherwise the index in the lane alone, and two more candidates than are
  // taken, so that it shows which of them are surely in their order, and before all others.
  const bool cut = BIASED || !a.logits_bf16;
  const uint32_t low = cut ? R - 1u : 64u * R - 1u;
  uint32_t k[R];
#pragma unroll
  for (int r = 0; r < R; ++r) k[r] = c[r] > ninf ? (ordered(c[r]) & ~low) | (low - (cut ? 0u : e0) - r) : 0u;
#pragma unroll
  for (int i = 1; i < R; ++i)
#pragma unroll
    for (int j = i; j > 0; --j) {
      const uint32_t x = k[j], y = k[j - 1];
      k[j - 1] = x > y ? x : y;
      k[j] = x > y ? y : x;
    }
  const uint32_t rounds = a.topk + (cut ? 2u : 0u);
  uint32_t mine = 0, id = INT8W_NO_EXPERT, n = 0;  // lane j: choice j
  for (; n < rounds; ++n) {
    const uint32_t best = wave_max_u32(k[0]);
    if (best == 0u) break;
    const uint32_t from = (uint32_t)__builtin_ctzll(__ballot(k[0] == best));
    const uint32_t e = low - (best & low) + (cut ? R * from : 0u);
    mine = lane == n ? best : mine;
    id = lane == n ? e : id;
    if (lane == from) {
#pragma unroll
      for (int r = 0; r + 1 < R; ++r) k[r] = k[r + 1];
      k[R - 1] = 0u;
    }
  }
  bool again = __ballot(near) != 0ull && !odd;
  double total = 1.0;
  const auto sum64 = [&]() {
    double x = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r) x += v[r] > ninf ? exp((double)v[r] - (double)top) : 0.0;
    return wave_sum(x);
  };
  if (cut && !again) {
    const uint32_t next = (uint32_t)__shfl_down((int)mine, 1, kWave);
    const float x = unordered(mine & ~low), y = unordered(next & ~low);
    // what the index took the place of: less than R units of 2^-23
    const float reach = BIASED ? margin + (kMarginOf + R * 0x1p-23f) * (fabsf(x) + fabsf(y)) : R * 0x1p-23f * (fabsf(x) + fabsf(y));
    // two infinities differ by a NaN: not surely in their order either
    if (__ballot(lane + 1u < n && lane < a.topk && !(x - y > reach)) != 0ull && !odd) {
      // the candidates themselves in fp64; one that is not among them is at most `most_out`
      wave_fence();
      if (BIASED && !a.sigmoid) total = sum64();
      double c64 = -__builtin_inf();
      if (lane < n) c64 = BIASED ? score64(lds.logit[id], a.sigmoid, top, total) + (double)a.bias[id] : (double)lds.logit[id];
      uint32_t place = 0;
      for (uint32_t j = 0; j < n; ++j) {
        const double other = __shfl(c64, (int)j, kWave);
        const uint32_t other_id = (uint32_t)__builtin_amdgcn_readlane((int)id, (int)j);
        place += other > c64 || (other == c64 && other_id < id) ? 1u : 0u;
      }
      const float last = lane_value(x, n - 1u);
      const double most_out = n < rounds ? -__builtin_inf() : (double)last + (double)(margin + (kMarginOf + R * 0x1p-22f) * fabsf(last));
      again = __ballot(lane < n && place < a.topk && !(c64 > most_out)) != 0ull;
      lds.order[lane < n ? place : 63u] = id;
      wave_fence();
      if (lane < n) id = lds.order[lane];
    }
  }
  if (n > a.topk) n = a.topk;
  if (again) {
    if (!a.sigmoid) total = sum64();
    n = choose64<R>(a, v, b, BIASED, top, total, lane, lds, id);
  }
  if (odd) n = 0;
  // weights, in fp32 unless what is to be divided by its sum is all far down; with the hardware's reciprocal, a unit of 2^-23
  // off (an IEEE division is about ten instructions): off by 7e-8 on the mean, where one rounding of 64 bits is by 2.7e-8
  wave_fence();
  const float l = lane < n ? lds.logit[id] : ninf, d = a.sigmoid ? l : l - top;
  float w;
  if (a.renorm && __ballot(d >= -40.f) == 0ull) {
    double x = score64(l, a.sigmoid, top, 1.0), sum = 0.0;
    for (uint32_t j = 0; j < n; ++j) sum += __shfl(x, (int)j, kWave);
    w = sum > 0.0 ? (float)(x / sum * (double)a.scale) : 0.f;
  } else {
    const float e = lane < n ? expf(a.sigmoid ? -d : d) : 0.f;
    float sum = 1.f;
    w = a.sigmoid ? (lane < n ? __builtin_amdgcn_rcpf(1.f + e) : 0.f) : e;
    if (a.renorm) {
      sum = wave_add(w);
    } else if (!a.sigmoid) {
      sum = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) sum += v[r] > ninf ? expf(v[r] - top) : 0.f;
      sum = wave_add(sum);
    }
    w = sum > 0.f ? w * __builtin_amdgcn_rcpf(sum) * a.scale : 0.f;
  }
  if (lane >= a.topk) return;
  a.ids[(size_t)t * a.topk + lane] = lane < n ? id : INT8W_NO_EXPERT;
  a.weights[(size_t)t * a.topk + lane] = odd ? __builtin_nanf("") : lane < n ? w : 0.f;  // 0 whatever the factor
}

template <int R>
void launch_route_r(RouteArgs a, hipStream_t stream) {
  // whole vectors of a lane's values: logits of every row, and the bias
  const uint32_t el = a.logits_bf16 ? 2u : 4u;
  a.whole = a.E % R == 0u && reinterpret_cast<uintptr_t>(a.logits) % (R * el) == 0u;
  a.whole_bias = a.E % R == 0u && reinterpret_cast<uintptr_t>(a.bias) % (R * 4u) == 0u;
  const uint32_t lanes = a.group_size % R == 0u ? a.group_size / R : 0u;
  a.group_lanes = lanes <= 32u && (lanes & (lanes - 1u)) == 0u ? lanes : 0u;
  constexpr uint32_t kMost = 1u << 25;  // tokens a launch, which has fewer than 2^32 threads
  for (uint32_t left = a.tokens; left; left -= a.tokens) {
    a.tokens = left < kMost ? left : kMost;
    const dim3 grid((a.tokens + kRouteWaves - 1u) / kRouteWaves);
    if (a.bias)
      k_route<R, true><<<grid, 64 * kRouteWaves, 0, stream>>>(a);
    else
      k_route<R, false><<<grid, 64 * kRouteWaves, 0, stream>>>(a);
    a.logits = (const uint8_t *)a.logits + (size_t)a.tokens * a.E * el;
    a.ids += (size_t)a.tokens * a.topk;
    a.weights += (size_t)a.tokens * a.topk;
  }
}

}  // namespace

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
  a.group_size = a.E / a.groups;
  // e * group_magic >> 20 is e / group_size: e * (group_magic * group_size - 2^20) <= 512 * 512 < 2^20
  a.group_magic = (1u << 20) / a.group_size + 1u;
  if (a.E <= 64u)
    launch_route_r<1>(a, stream);
  else if (a.E <= 128u)
    launch_route_r<2>(a, stream);
  else if (a.E <= 256u)
    launch_route_r<4>(a, stream);
  else
    launch_route_r<8>(a, stream);
  return hipGetLastError();
}

}  // namespace int8w
