// moe_route.hip -- the routing to experts by itself: scores, choice, weights.
//
//   s = softmax(l) or 1 / (1 + e^-l);  c = s + bias;  of the groups of experts the best
//   topk_groups by their largest c or the sum of their two largest;  in them the topk
//   largest c, the lower index first among equals;  weight = scale s [/ sum of the taken s].
//
// A wave routes a token: lane l holds experts l, l + 64, ...; top-k is a maximum over the wave
// and a ballot for its place, topk times.  Which experts are taken must not hang on how a
// score was rounded: without a bias and groups c orders as the logit, which is compared itself;
// otherwise scores and sums are fp64.  The weights of the few taken experts are formed in
// fp64 as well and rounded once.
#include "launch.h"
#include "wave_ops.h"

namespace int8w {

namespace {

constexpr uint32_t kRouteWaves = 4;

// Score of a logit: top and total for softmax.
__device__ __forceinline__ double route_score(float l, bool sigmoid, float top, double total) {
  if (!(l > -__builtin_inff())) return 0.0;
  return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / total;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// R: ceil(E / 64) at most.  WIDE: c = s + bias in fp64 (and groups); else c is the logit.
template <int R, bool WIDE>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(const RouteArgs a) {
  typedef typename std::conditional<WIDE, double, float>::type C;
  __shared__ C all[WIDE ? kRouteWaves : 1][WIDE ? 64 * R : 1];
  __shared__ float taken[kRouteWaves][INT8W_MAX_MOE_TOPK];  // logits
  const float ninf = -__builtin_inff();
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, E = a.E;
  const uint32_t at_t = blockIdx.x * kRouteWaves + wave;
  const bool live = at_t < a.tokens;
  const uint32_t t = live ? at_t : a.tokens - 1u;  // a wave past the last token repeats it
  float v[R], top = ninf;
  C c[R];
  bool odd = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t e = 64u * r + lane;
    v[r] = ninf;
    if (e < E)
      v[r] = a.logits_bf16 ? bf16_bits_to_f32(((const uint16_t *)a.logits)[(size_t)t * E + e]) : ((const float *)a.logits)[(size_t)t * E + e];
    odd |= a.sigmoid ? v[r] != v[r] : !(v[r] < __builtin_inff());
    top = fmaxf(top, v[r]);
  }
  top = wave_max(top);
  double total = 1.0;
  if (!a.sigmoid && (WIDE || !a.renorm)) {
    total = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r) total += v[r] > ninf ? exp((double)v[r] - (double)top) : 0.0;
    total = wave_sum(total);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    c[r] = v[r];
    if constexpr (WIDE) {
      const uint32_t e = 64u * r + lane;
      const double with = route_score(v[r], a.sigmoid, top, total) + (a.bias && e < E ? (double)a.bias[e] : 0.0);
      odd |= with != with;
      c[r] = v[r] > ninf ? with : (double)ninf;
    }
  }
  odd = __ballot(odd) != 0ull;
  if constexpr (WIDE) {
    if (a.groups > 1u) {
#pragma unroll
      for (int r = 0; r < R; ++r) all[wave][64u * r + lane] = c[r];
      __syncthreads();
      const uint32_t size = a.group_size;
      double one = ninf, two = ninf;  // lane g: the group's two largest
      if (lane < a.groups)
        for (uint32_t i = 0, e = lane % size; i < size; ++i) {  // each lane from its own start: banks
          const double x = all[wave][lane * size + e];
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
        const uint32_t g = ((64u * r + lane) * a.group_magic) >> 20;  // e / size
        if (g >= a.groups || !(stay >> g & 1ull)) c[r] = ninf;
      }
    }
  }
  uint32_t id = INT8W_NO_EXPERT, n = 0;
  for (uint32_t j = 0; j < a.topk && !odd; ++j) {
    C left = ninf;
#pragma unroll
    for (int r = 0; r < R; ++r) left = fmax(left, c[r]);
    const C best = wave_max(left);
    if (!(best > ninf)) break;
    uint32_t at = 0;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const unsigned long long is = __ballot(c[r] == best);
      if (is) at = 64u * r + (uint32_t)__builtin_ctzll(is);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (64u * r + lane == at) {
        c[r] = ninf;
        taken[wave][j] = v[r];
      }
    if (lane == j) id = at;
    ++n;
  }
  __syncthreads();
  if (lane >= a.topk || !live) return;
  double w = lane < n ? route_score(taken[wave][lane], a.sigmoid, top, total) : 0.0;
  if (a.renorm) {
    double sum = 0.0;
    for (uint32_t j = 0; j < n; ++j) sum += __shfl(w, (int)j, kWave);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  a.ids[(size_t)t * a.topk + lane] = id;
  a.weights[(size_t)t * a.topk + lane] = odd ? __builtin_nanf("") : (float)(w * (double)a.scale);
}

template <int R>
void launch_route_r(const RouteArgs &a, hipStream_t stream) {
  const dim3 grid((a.tokens + kRouteWaves - 1u) / kRouteWaves);
  if (a.bias || a.groups > 1u)
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
