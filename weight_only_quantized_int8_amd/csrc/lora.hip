// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//   u[t] = A_e x[t],  y[t] = base[t] + scale_e B_e u[t],  e = ids[t];
//   A_e [R, K], B_e [N, R], R far below K and N; id INT8W_NO_ADAPTER: y[t] = base[t].
//
// Two launches, on the matrix cores (16x16x32 products):
//  shrink  u in fp32, K cut into `parts` (the sum over K is the long one, and a single token's
//          A has to come through many CUs): u [parts, m, R] in the workspace.
//  expand  sums the parts in their order, scales, multiplies by B_e, adds base, rounds once.
//          u enters the matrix cores as the sum of two BF16 values (u's own rounding to one
//          would be as large as the output's); the products are exact and summed in fp32.
// No atomics: the same bits each time.
//
// Both have two forms.  Few rows (rows form): a decode batch, rows in any order, mostly each with an
// adapter of its own.  A workgroup stands for a row; of the rows that share an adapter each 16th
// leads and its workgroup takes it and the next 15 (found by ballots over ids, read by every
// wave), the others end at once: an adapter is streamed once for up to 16 rows wherever they are.
// Many rows (tile form): windows of 64 neighbouring rows; a workgroup goes over the adapters
// that occur in its window, for a prompt one or two.
// A row is a column of the product, and columns do not mix: what another row or its adapter
// holds (infinities, NaN) does not reach it.
#include "common.h"
#include "launch.h"

namespace int8w {

namespace {

constexpr uint32_t kRowsGroup = 16;   // rows of a workgroup in the rows form
constexpr uint32_t kTileRows = 64;    // in the tile form
constexpr uint32_t kStepK = 64;       // K of a wave's step: whole cache lines of A and x
constexpr uint32_t kTileN = 256;      // output columns of a workgroup of four waves
constexpr uint32_t kRowsMax = 256;    // most rows that the rows form takes

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The adapter's own rank, rounded up to whole 16-byte pieces of a row of B.
__device__ __forceinline__ uint32_t own_rank(const LoraStack &s, uint32_t e) {
  if (!s.ranks) return s.R;
  const uint32_t r = (s.ranks[e] + 7u) & ~7u;
  return r < s.R ? r : s.R;
}

// Rows form: whether row i leads, and then list[0 .. n-1] = the rows of its group.  Every wave
// finds the same and writes the same list.
__device__ __forceinline__ bool gather_rows(const uint32_t *ids, uint32_t m, uint32_t i, uint32_t id, uint32_t lane,
                                            uint32_t *list, uint32_t &n) {
  uint32_t before = 0;
  n = 0;
  for (uint32_t j0 = 0; j0 < m && n < kRowsGroup; j0 += 64u) {
    const uint32_t j = j0 + lane;
    const unsigned long long same = __ballot(j < m && ids[j < m ? j : 0u] == id);
    const unsigned long long mine = j0 + 64u <= i ? 0ull : j0 >= i ? ~0ull : ~0ull << (i - j0);  // rows from i on
    before += (uint32_t)__popcll(same & ~mine);
    const unsigned long long next = same & mine;
    const uint32_t at = n + (uint32_t)__popcll(next & ((1ull << lane) - 1ull));
    if ((next >> lane & 1ull) && at < kRowsGroup) list[at] = j;
    n += (uint32_t)__popcll(next);
  }
  if (n > kRowsGroup) n = kRowsGroup;
  return before % kRowsGroup == 0u;
}

// acc[t] += A rows 16 t .. 16 t + 15 of the step times x.  Lane (c, q) holds of a row 32 bytes
// from k0 + 16 q: both operands alike, and a row's four lanes cover a cache line.
template <int RT>
struct ShrinkStep {
  u32x4 x[2], a[RT][2];
  __device__ __forceinline__ void load(const uint16_t *xrow, __amdgpu_buffer_rsrc_t ra, uint32_t K, uint32_t rank,
                                       uint32_t k0, uint32_t lane) {
    const uint32_t c = lane & 15u, k = k0 + 16u * (lane >> 4);
#pragma unroll
    for (uint32_t h = 0; h < 2u; ++h) {
      const bool in = k + 8u * h < K;
      x[h] = *reinterpret_cast<const u32x4 *>(xrow + (in ? k + 8u * h : 0u));
      if (!in) x[h] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (uint32_t t = 0; t < RT; ++t) {
        const uint32_t r = 16u * t + c;
        a[t][h] = buf_load_b128(ra, in && r < rank ? (r * K + k + 8u * h) * 2u : kOutOfRange);
      }
    }
  }
  __device__ __forceinline__ void multiply(f32x4 (&acc)[RT]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = mfma(a[t][h], x[h], acc[t]);
  }
};

// grid (parts, rows, stacks).  The four waves of a workgroup take steps of the part in turn.
template <int RT>
__global__ __launch_bounds__(256) void k_shrink_rows(const LoraArgs g) {
  __shared__ uint32_t list[kRowsGroup];
  constexpr int kTiles = RT < 4 ? RT : 4;  // added up at a time
  __shared__ f32x4 sums[4][kTiles * 64];
  const LoraStack &s = g.s[blockIdx.z];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6), part = blockIdx.x, i = blockIdx.y;
  const uint32_t id = uniform(g.ids[i]);
  if (id >= g.num) return;
  uint32_t n;
  if (!gather_rows(g.ids, g.m, i, id, lane, list, n)) return;
  __syncthreads();
  const uint32_t c = lane & 15u, rank = own_rank(s, id);
  const uint16_t *xrow = g.x + list[c < n ? c : 0u] * g.x_stride;  // columns from n on repeat a row, unused
  const auto ra = make_rsrc(s.a + (size_t)id * s.R * g.K, s.R * g.K * 2u);
  f32x4 acc[RT] = {};
  const uint32_t k1 = (part + 1u) * g.part_k < g.K ? (part + 1u) * g.part_k : g.K;
  for (uint32_t k0 = part * g.part_k + wave * kStepK; k0 < k1; k0 += 4u * kStepK) {
    ShrinkStep<RT> step;
    step.load(xrow, ra, g.K, rank, k0, lane);
    step.multiply(acc);
  }
#pragma unroll
  for (int t0 = 0; t0 < RT; t0 += kTiles) {
    if (t0) __syncthreads();
#pragma unroll
    for (int t = 0; t < kTiles; ++t) sums[wave][64 * t + lane] = acc[t0 + t];
    __syncthreads();
    const uint32_t p = threadIdx.x, r = 16u * (t0 + (p >> 6)) + 4u * (p >> 4 & 3u), col = p & 15u;
    if (p < kTiles * 64u && col < n && r < s.R) {
      const f32x4 v = (sums[0][p] + sums[1][p]) + (sums[2][p] + sums[3][p]);
      *reinterpret_cast<f32x4 *>(s.u + ((size_t)part * g.m + list[col]) * s.R + r) = v;
    }
  }
}

// grid (parts, windows, stacks).  A wave has 16 of the window's rows.
template <int RT>
__global__ __launch_bounds__(256) void k_shrink_tile(const LoraArgs g) {
  const LoraStack &s = g.s[blockIdx.z];
  const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6), part = blockIdx.x;
  const uint32_t row = blockIdx.y * kTileRows + 16u * wave + (lane & 15u);
  uint32_t id = row < g.m ? g.ids[row] : INT8W_NO_ADAPTER;
  if (id >= g.num) id = INT8W_NO_ADAPTER;
  const uint16_t *xrow = g.x + (row < g.m ? row : g.m - 1u) * g.x_stride;
  const uint32_t k1 = (part + 1u) * g.part_k < g.K ? (part + 1u) * g.part_k : g.K;
  unsigned long long left = __ballot(id != INT8W_NO_ADAPTER);
  while (left) {
    const uint32_t e = (uint32_t)__builtin_amdgcn_readlane((int)id, __builtin_ctzll(left));
    left &= ~__ballot(id == e);
    const uint32_t rank = own_rank(s, e);
    const auto ra = make_rsrc(s.a + (size_t)e * s.R * g.K, s.R * g.K * 2u);
    f32x4 acc[RT] = {};
    for (uint32_t k0 = part * g.part_k; k0 < k1; k0 += kStepK) {
      ShrinkStep<RT> step;
      step.load(xrow, ra, g.K, rank, k0, lane);
      step.multiply(acc);
    }
    if (id == e) {
#pragma unroll
      for (uint32_t t = 0; t < RT; ++t) {
        const uint32_t r = 16u * t + 4u * (lane >> 4);
        if (r < s.R) *reinterpret_cast<f32x4 *>(s.u + ((size_t)part * g.m + row) * s.R + r) = acc[t];
      }
    }
  }
}

// u of up to ROWS rows in LDS: summed over the parts, scaled, as two BF16 values.  A row is
// padded by 16 bytes so that the sixteen rows of an operand lie in different banks.
template <int KS>  // steps of 32 of the rank
struct ExpandU {
  static constexpr uint32_t kRow = 64u * KS + 16u;
  // Thread's share of rows x rank; row(c) >= m: zeros.
  template <class Row, class Scale>
  static __device__ __forceinline__ void stage(uint8_t *hi, uint8_t *lo, const LoraArgs &g, const LoraStack &s, uint32_t rows,
                                               Row row, Scale scale) {
    for (uint32_t p = threadIdx.x; p < rows * 8u * KS; p += blockDim.x) {
      const uint32_t c = p / (8u * KS), r = 4u * (p % (8u * KS)), t = row(c);
      f32x4 v = {};
      if (t < g.m && r < s.R) {
        const float *from = s.u + (size_t)t * s.R + r;
        for (uint32_t i = 0; i < g.parts; ++i) v += *reinterpret_cast<const f32x4 *>(from + (size_t)i * g.m * s.R);
        v *= scale(c);
      }
      uint2 h = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      // a value beyond BF16's range has an infinity for its upper part and NaN for the difference
      float d[4] = {v[0] - bf16_lo(h.x), v[1] - bf16_hi(h.x), v[2] - bf16_lo(h.y), v[3] - bf16_hi(h.y)};
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = fabsf(d[i]) < __builtin_inff() ? d[i] : 0.f;
      *reinterpret_cast<uint2 *>(hi + c * kRow + 2u * r) = h;
      *reinterpret_cast<uint2 *>(lo + c * kRow + 2u * r) = make_uint2(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]));
    }
  }
  static __device__ __forceinline__ u32x4 get(const uint8_t *lds, uint32_t c, uint32_t step, uint32_t lane) {
    return *reinterpret_cast<const u32x4 *>(lds + c * kRow + 64u * step + 16u * (lane >> 4));
  }
};

// 64 columns from n0 in four tiles: as a row of the product's first operand lane (c, q) loads
// column n0 + 16 (c / 4) + 4 t + c % 4 of tile t, so that as a result it holds n0 + 16 q + 4 t + i:
// sixteen neighbouring outputs of its row.
template <int KS>
__device__ __forceinline__ void load_b(u32x4 (&b)[4][KS], __amdgpu_buffer_rsrc_t rb, uint32_t R, uint32_t rank, uint32_t n0,
                                       uint32_t lane) {
  const uint32_t c = lane & 15u;
#pragma unroll
  for (uint32_t t = 0; t < 4u; ++t) {
    const uint32_t n = n0 + 16u * (c >> 2) + 4u * t + (c & 3u);  // past the last one: zeros by the resource
#pragma unroll
    for (uint32_t k = 0; k < KS; ++k) {
      const uint32_t r = 32u * k + 8u * (lane >> 4);
      b[t][k] = buf_load_b128(rb, r < rank ? (n * R + r) * 2u : kOutOfRange);
    }
  }
}

// Sixteen neighbouring values of a row: y = base + v, columns from n on.
struct OutRow {
  const uint16_t *base;
  uint16_t *y;
  uint32_t left;  // columns to the row's end
  bool wide;      // 16-byte pieces
  __device__ __forceinline__ OutRow(const LoraStack &s, size_t row, uint32_t n, bool wide_) {
    left = n < s.N ? s.N - n : 0u;
    base = s.base ? s.base + row * s.base_stride + n : nullptr;
    y = s.y + row * s.y_stride + n;
    wide = wide_ && left >= 16u;
  }
  __device__ __forceinline__ void add(const f32x4 (&v)[4]) const {
    if (wide) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 o = base ? *reinterpret_cast<const u32x4 *>(base + 8 * h) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 &w = v[2 * h + i / 2];
          o[i] = pack_bf16x2(bf16_lo(o[i]) + w[2 * (i & 1)], bf16_hi(o[i]) + w[2 * (i & 1) + 1]);
        }
        *reinterpret_cast<u32x4 *>(y + 8 * h) = o;
      }
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 16u; ++i)
        if (i < left) y[i] = to_bf16_bits((base ? bf16_bits_to_f32(base[i]) : 0.f) + v[i / 4][i % 4]);
    }
  }
  // no adapter: base itself; an id outside the pool: NaN
  __device__ __forceinline__ void pass(bool nan) const {
    if (!nan && base == y) return;
#pragma unroll
    for (uint32_t i = 0; i < 16u; ++i)
      if (i < left) y[i] = nan ? 0x7FC0u : base ? base[i] : 0u;
  }
};

__device__ __forceinline__ bool wide_rows(const LoraStack &s) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(s.y) | (s.y_stride * 2u) | reinterpret_cast<uintptr_t>(s.base) |
                       (s.base ? s.base_stride * 2u : 0u);
  return (at & 15u) == 0u;
}

// The stack and column tile of a block: the stacks' tiles one after the other.
__device__ __forceinline__ const LoraStack &stack_of(const LoraArgs &g, uint32_t &tile, uint32_t tile_n) {
  uint32_t i = 0;
  for (; i + 1u < g.count; ++i) {
    const uint32_t tiles = (g.s[i].N + tile_n - 1u) / tile_n;
    if (tile < tiles) break;
    tile -= tiles;
  }
  return g.s[i];
}

// grid (column tiles of all stacks, rows).  A wave has 64 columns.
template <int KS>
__global__ __launch_bounds__(256) void k_expand_rows(const LoraArgs g) {
  typedef ExpandU<KS> U;
  __shared__ uint32_t list[kRowsGroup];
  __shared__ __attribute__((aligned(16))) uint8_t hi[kRowsGroup * U::kRow], lo[kRowsGroup * U::kRow];
  uint32_t tile = blockIdx.x;
  const LoraStack &s = stack_of(g, tile, kTileN);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6), i = blockIdx.y, c = lane & 15u;
  const uint32_t n0 = tile * kTileN + 64u * wave, id = uniform(g.ids[i]);
  if (id >= g.num) {
    if (threadIdx.x < kTileN / 16u)
      OutRow(s, i, tile * kTileN + 16u * threadIdx.x, false).pass(id != INT8W_NO_ADAPTER);
    return;
  }
  uint32_t n;
  if (!gather_rows(g.ids, g.m, i, id, lane, list, n)) return;
  const uint32_t rank = own_rank(s, id);
  const auto rb = make_rsrc(s.b + (size_t)id * s.N * s.R, s.N * s.R * 2u);
  u32x4 b[4][KS];
  load_b<KS>(b, rb, s.R, rank, n0, lane);
  const float scale = s.scales ? s.scales[id] : 1.f;
  __syncthreads();
  U::stage(hi, lo, g, s, kRowsGroup, [&](uint32_t r) { return r < n ? list[r] : g.m; }, [&](uint32_t) { return scale; });
  __syncthreads();
  f32x4 acc[4] = {};
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const u32x4 uh = U::get(hi, c, k, lane), ul = U::get(lo, c, k, lane);
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = mfma(b[t][k], ul, mfma(b[t][k], uh, acc[t]));
  }
  if (c < n) OutRow(s, list[c], n0 + 16u * (lane >> 4), wide_rows(s)).add(acc);
}

// grid (chunks of chunk_n columns of all stacks, windows).  The waves take blocks of 64 columns in turn.
template <int KS>
__global__ __launch_bounds__(256) void k_expand_tile(const LoraArgs g, uint32_t chunk_n) {
  typedef ExpandU<KS> U;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint8_t *const hi = lds, *const lo = lds + kTileRows * U::kRow;
  uint32_t tile = blockIdx.x;
  const LoraStack &s = stack_of(g, tile, chunk_n);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6), c = lane & 15u;
  const uint32_t row0 = blockIdx.y * kTileRows;
  const uint32_t own = row0 + lane < g.m ? g.ids[row0 + lane] : INT8W_NO_ADAPTER;
  const bool here = row0 + lane < g.m;
  U::stage(hi, lo, g, s, kTileRows,
           [&](uint32_t r) {
             const uint32_t t = row0 + r;
             return t < g.m && g.ids[t] < g.num ? t : g.m;
           },
           [&](uint32_t r) { return s.scales ? s.scales[g.ids[row0 + r]] : 1.f; });
  __syncthreads();
  const bool wide = wide_rows(s);
  const unsigned long long some = __ballot(here && own < g.num), bad = __ballot(here && own >= g.num && own != INT8W_NO_ADAPTER);
  const unsigned long long none = __ballot(here && own == INT8W_NO_ADAPTER);
  const uint32_t end = (tile + 1u) * chunk_n < s.N ? (tile + 1u) * chunk_n : s.N;
  for (uint32_t n0 = tile * chunk_n + 64u * wave; n0 < end; n0 += 256u) {
    for (unsigned long long left = some; left;) {
      const uint32_t e = (uint32_t)__builtin_amdgcn_readlane((int)own, __builtin_ctzll(left));
      const unsigned long long rows = __ballot(own == e) & some;
      left &= ~rows;
      const uint32_t rank = own_rank(s, e);
      u32x4 b[4][KS];
      load_b<KS>(b, make_rsrc(s.b + (size_t)e * s.N * s.R, s.N * s.R * 2u), s.R, rank, n0, lane);
#pragma unroll
      for (uint32_t tt = 0; tt < kTileRows / 16u; ++tt) {
        if ((rows >> (16u * tt) & 0xFFFFull) == 0ull) continue;
        f32x4 acc[4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const u32x4 uh = U::get(hi, 16u * tt + c, k, lane), ul = U::get(lo, 16u * tt + c, k, lane);
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[t] = mfma(b[t][k], ul, mfma(b[t][k], uh, acc[t]));
        }
        if (rows >> (16u * tt + c) & 1ull) OutRow(s, row0 + 16u * tt + c, n0 + 16u * (lane >> 4), wide).add(acc);
      }
    }
    if ((none | bad) != 0ull)
      for (uint32_t tt = 0; tt < kTileRows / 16u; ++tt) {
        const uint32_t r = 16u * tt + c;
        if ((none | bad) >> r & 1ull) OutRow(s, row0 + r, n0 + 16u * (lane >> 4), wide).pass(bad >> r & 1ull);
      }
  }
}

bool rows_form(uint32_t m) { return m <= kRowsMax; }

uint32_t max_rank(const LoraArgs &a) {
  uint32_t r = 0;
  for (uint32_t i = 0; i < a.count; ++i) r = a.s[i].R > r ? a.s[i].R : r;
  return r;
}

// How K is cut: enough workgroups to load from every CU, each with a step for every wave.
void cut_k(LoraArgs &a) {
  const uint32_t steps = (a.K + kStepK - 1u) / kStepK;
  const uint32_t blocks = a.count * (rows_form(a.m) ? a.m : (a.m + kTileRows - 1u) / kTileRows);
  uint32_t parts = 1024u / blocks, most = rows_form(a.m) ? 32u : 8u;
  if (rows_form(a.m) && parts < 8u) parts = 8u;
  if (parts > most) parts = most;
  if (parts > (steps + 3u) / 4u) parts = (steps + 3u) / 4u;
  if (parts < 1u) parts = 1u;
  const uint32_t each = (steps + parts - 1u) / parts;
  a.part_k = each * kStepK;
  a.parts = (steps + each - 1u) / each;
}

template <int RT>
void launch_shrink(const LoraArgs &a, hipStream_t stream) {
  if (rows_form(a.m))
    k_shrink_rows<RT><<<dim3(a.parts, a.m, a.count), 256, 0, stream>>>(a);
  else
    k_shrink_tile<RT><<<dim3(a.parts, (a.m + kTileRows - 1u) / kTileRows, a.count), 256, 0, stream>>>(a);
}

template <int KS>
hipError_t launch_expand(const LoraArgs &a, hipStream_t stream) {
  uint32_t tiles = 0;
  if (rows_form(a.m)) {
    for (uint32_t i = 0; i < a.count; ++i) tiles += (a.s[i].N + kTileN - 1u) / kTileN;
    k_expand_rows<KS><<<dim3(tiles, a.m), 256, 0, stream>>>(a);
    return hipGetLastError();
  }
  const uint32_t lds = 2u * kTileRows * ExpandU<KS>::kRow, windows = (a.m + kTileRows - 1u) / kTileRows;
  static LdsAllowance allowance;
  if (needs_lds_allowance(lds, 0)) {
    const hipError_t e = allow_lds(allowance, k_expand_tile<KS>, (int)lds);
    if (e != hipSuccess) return e;
  }
  uint32_t all = 0;
  for (uint32_t i = 0; i < a.count; ++i) all += (a.s[i].N + kTileN - 1u) / kTileN;
  const uint32_t chunks = 2048u / windows < 1u ? 1u : 2048u / windows;  // per window
  const uint32_t chunk_n = (all + chunks - 1u) / chunks * kTileN;
  for (uint32_t i = 0; i < a.count; ++i) tiles += (a.s[i].N + chunk_n - 1u) / chunk_n;
  k_expand_tile<KS><<<dim3(tiles, windows), 256, lds, stream>>>(a, chunk_n);
  return hipGetLastError();
}

}  // namespace

uint64_t lora_workspace(const LoraArgs &given, uint64_t *offsets) {
  LoraArgs a = given;
  cut_k(a);
  uint64_t bytes = 0;
  for (uint32_t i = 0; i < a.count; ++i) {
    offsets[i] = bytes;
    bytes += ((uint64_t)a.parts * a.m * a.s[i].R * 4u + 255u) & ~255ull;
  }
  return bytes;
}

hipError_t launch_lora(LoraArgs a, void *ws, hipStream_t stream) {
  cut_k(a);
  uint64_t offsets[INT8W_MAX_MULTI];
  lora_workspace(a, offsets);
  for (uint32_t i = 0; i < a.count; ++i) a.s[i].u = reinterpret_cast<float *>((uint8_t *)ws + offsets[i]);
  const uint32_t R = max_rank(a);
  if (R <= 16u)
    launch_shrink<1>(a, stream);
  else if (R <= 32u)
    launch_shrink<2>(a, stream);
  else if (R <= 64u)
    launch_shrink<4>(a, stream);
  else if (R <= 128u)
    launch_shrink<8>(a, stream);
  else
    launch_shrink<16>(a, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (R <= 32u) return launch_expand<1>(a, stream);
  if (R <= 64u) return launch_expand<2>(a, stream);
  if (R <= 128u) return launch_expand<4>(a, stream);
  return launch_expand<8>(a, stream);
}

}  // namespace int8w
