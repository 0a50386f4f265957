// moe_route.hip -- the routing to experts by itself: scores, choice, weights.
//
//   s = softmax(l) or 1 / (1 + e^-l);  c = s + bias, or l without a bias;  of the groups of experts
//   the best topk_groups by their largest c or the sum of the two largest s + bias;  in them the
//   topk largest c, the lower index first among equals;  weight = scale s [/ sum of the taken s].
//
// A wave routes a token: lane l holds experts l R .. l R + R - 1, sorted, so that top-k is a
// maximum over the lanes' heads, a ballot for its place (the lowest lane: the lowest index among
// equals) and one step of that lane's list, topk times.
// Which experts are taken must not hang on how a score was rounded.  Logits are compared
// themselves; scores are formed in fp32 within a known error (below), and a token with two of them
// too near to tell is done again in fp64.  The weights of the few taken experts are formed in
// fp64 as well and rounded once.
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

// Sorts a lane's values, the earlier first among equals; at: where they came from.
template <int R>
__device__ __forceinline__ void sort_lane(float (&c)[R], uint32_t (&at)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i) at[i] = i;
#pragma unroll
  for (int i = 1; i < R; ++i)  // insertion: compares neighbours only, so equal values keep their order
#pragma unroll
    for (int j = i; j > 0; --j) {
      const bool swap = c[j] > c[j - 1];
      const float x = c[j], y = c[j - 1];
      const uint32_t p = at[j], q = at[j - 1];
      c[j - 1] = swap ? x : y;
      c[j] = swap ? y : x;
      at[j - 1] = swap ? p : q;
      at[j] = swap ? q : p;
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
  top = wave_max(top);
  uint32_t id = INT8W_NO_EXPERT, n = 0;
  double total = 1.0;
  // fp32 scores, where anything goes by them
  const bool sums = a.groups > 1u && a.top2;
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
  for (int r = 0; r < R; ++r) c[r] = BIASED ? s[r] : v[r];
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
    const float size_of = of > ninf ? fabsf(one) + (sums && two > ninf ? fabsf(two) : 0.f) : 0.f;
    const uint32_t lanes = a.group_lanes ? a.group_lanes : 1u, own = lane / lanes;
    uint32_t before = 0;  // groups before this lane's
    for (uint32_t g = 0; g < a.groups; ++g) {
      const float other = lane_value(of, g * lanes);
      before += other > of || (other == of && g < own) ? 1u : 0u;
      if (BIASED || sums)
        near |= g != own && own < a.groups && other > ninf && fabsf(other - of) <= 2.f * margin + kMarginOf * (size_of + lane_value(size_of, g * lanes));
    }
    const unsigned long long stay = __ballot(own < a.groups && before < a.topk_groups && of > ninf);  // by lanes
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t g = a.group_lanes ? own : (e0 + r) * a.group_magic >> 20;  // e / size
      if (g >= a.groups || !(stay >> (g * lanes) & 1ull)) c[r] = ninf;
    }
  }
  uint32_t at[R];
  sort_lane<R>(c, at);
  float last = 0.f;
  const uint32_t rounds = BIASED ? a.topk + 1u : a.topk;  // the first one that is not taken tells whether the last one is surely before it
  for (uint32_t j = 0; j < rounds; ++j) {
    const float best = wave_max(c[0]);
    if (!(best > ninf)) break;
    if (BIASED && j) near |= last - best <= margin + kMarginOf * (fabsf(last) + fabsf(best));
    last = best;
    if (j == a.topk) break;
    const uint32_t from = (uint32_t)__builtin_ctzll(__ballot(c[0] == best));
    const uint32_t e = R * from + (uint32_t)__builtin_amdgcn_readlane((int)at[0], (int)from);
    if (lane == j) id = e;
    ++n;
    if (lane == from) {
#pragma unroll
      for (int r = 0; r + 1 < R; ++r) {
        c[r] = c[r + 1];
        at[r] = at[r + 1];
      }
      c[R - 1] = ninf;
    }
  }
  near = (BIASED || sums) && __ballot(near) != 0ull && !odd;
  if (!a.sigmoid && (near || !a.renorm)) {
    total = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r) total += v[r] > ninf ? exp((double)v[r] - (double)top) : 0.0;
    total = wave_sum(total);
  }
  if (near) n = choose64<R>(a, v, b, BIASED, top, total, lane, lds, id);
  if (odd) n = 0;
  if (lane >= a.topk) return;
  wave_fence();
  double w = lane < n ? score64(lds.logit[id], a.sigmoid, top, total) : 0.0;
  if (a.renorm) {
    double sum = 0.0;
    for (uint32_t j = 0; j < n; ++j) sum += __shfl(w, (int)j, kWave);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  a.ids[(size_t)t * a.topk + lane] = lane < n ? id : INT8W_NO_EXPERT;
  a.weights[(size_t)t * a.topk + lane] = odd ? __builtin_nanf("") : (float)(w * (double)a.scale);
}

template <int R>
void launch_route_r(RouteArgs a, hipStream_t stream) {
  // whole vectors of a lane's values: logits of every row, and the bias
  const uint32_t el = a.logits_bf16 ? 2u : 4u;
  a.whole = a.E % R == 0u && reinterpret_cast<uintptr_t>(a.logits) % (R * el) == 0u;
  a.whole_bias = a.E % R == 0u && reinterpret_cast<uintptr_t>(a.bias) % (R * 4u) == 0u;
  const uint32_t lanes = a.group_size % R == 0u ? a.group_size / R : 0u;
  a.group_lanes = lanes <= 32u && (lanes & (lanes - 1u)) == 0u ? lanes : 0u;
  const dim3 grid((a.tokens + kRouteWaves - 1u) / kRouteWaves);
  if (a.bias)
    k_route<R, true><<<grid, 64 * kRouteWaves, 0, stream>>>(a);
  else
    k_route<R, false><<<grid, 64 * kRouteWaves, 0, stream>>>(a);
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
