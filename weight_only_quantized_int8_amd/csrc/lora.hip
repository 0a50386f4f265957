// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//   u[t] = A_e x[t],  y[t] = base[t] + scale_e B_e u[t],  e = ids[t];
//   A_e [R, K], B_e [N, R], R far below K and N; id INT8W_NO_ADAPTER: y[t] = base[t].
//
// Bound: memory.  A product of rank R has 2 R operations for the 4 or 6 bytes of each x, base
// and y, and where rows have an adapter each, one for each byte of it; the matrix cores are there to keep
// the vector ALUs free.  Two launches:
//  shrink  u in fp32, K cut into `parts` (the sum over K is the long one, and a single token's
//          A has to come through many CUs): u [parts, m, R] in the workspace.
//  expand  sums the parts in their order, multiplies by B_e, scales, adds base, rounds once.
//          u enters the matrix cores as the sum of two BF16 values (u's own rounding to one
//          would be as large as the output's); the products are exact and summed in fp32.
// One launch (k_solo) for a few rows of small matrices: there the second launch costs more than
// reading A again for each 512 columns.
// No atomics in any sum: the same bits each time.
//
// A workgroup works on a group: rows with one adapter, wherever they are in the batch, so that its
// matrices are read once for all of them; up to 16 rows with K or N shared out among its waves
// ("few"), or up to 64 with the rows shared out ("many").
//  Up to 64 rows in the batch: a workgroup stands for a row; of the rows that share an adapter each
//   16th leads and takes the next 15 along, found by one ballot; the others end at once.
//  More: a launch before the others (k_plan, 3 to 5 us) sorts the rows of each 1024 into groups, which
//   a fixed number of workgroups shares: with a workgroup for each group that there might be, those
//   without one took longer than the work (200 rows: shrink 32 instead of 23 us).
// A row is a row or column of the products, which do not mix: what another row or its adapter
// holds (infinities, NaN) does not reach it.
//
// Measured, plan + shrink + expand, us (bytes that shrink and expand fetch and write):
//  8192 rows in 5 runs, 14336x4096, rank 64:   5 + 24 + 113  (71 and 437 MB in, 235 out: 6.0 TB/s in expand)
//  2109 rows, 24 adapters, 4096x14336, 8..64:  4 + 22 + 18   (84 and 44 MB in, 5 and 17 out: 4.0 TB/s in shrink)
//  549 rows, 16 adapters, gate and up, 16:     4 + 8 + 18    (8 and 15 MB in, 31 out: starts and ends of workgroups)
//  200 rows, 57 adapters, 4096x14336, rank 64: 4 + 24 + 15   (114 and 33 MB in: 4.8 TB/s in shrink)
//  33 rows, 25 adapters, q, k and v, 32:       - + 6.6 + 6.0 (9 and 8 MB in)
//  one row, 4096x4096, rank 16, one launch:    4.7 (3.9 in a graph)
// Of a rank above 64 shrink goes over x again for each 64 of it: 2109 rows, 24 adapters, 4096x14336, whole calls of rank
// 64 / 128 / 256 46 / 86 / 154, where the bytes alone take 31 / 42 / 65.
#include "rows_stream.h"
#include "token_stream.h"

namespace int8w {

namespace {

constexpr uint32_t kFew = 16;         // rows of a group, with K or N shared out among the waves
constexpr uint32_t kMany = 64;        // ... with the rows shared out
constexpr uint32_t kBallotRows = 64;  // largest batch without a plan
constexpr uint32_t kStepK = 64;       // K of a step: a cache line of a row
constexpr uint32_t kBlockN = 128;     // output columns of a step
constexpr uint32_t kShrinkBlocks = 512;  // workgroups over a plan's groups: what fits the CUs
constexpr uint32_t kExpandBlocks = 1024;
constexpr uint32_t kXcdGroups = 24;      // where an XCD of expand has groups of its own: three each,
constexpr uint32_t kXcdColumns = 4096;   // few columns
constexpr uint32_t kXcdValues = 2048;    // or much of u in a group

#define INT8W_VMCNT(n) __builtin_amdgcn_s_waitcnt((((n) >> 4) << 14) | 0x0F70 | ((n) & 15))
#define INT8W_LGKMCNT0() __builtin_amdgcn_s_waitcnt(0xC07F)

// Pointers out of the stacks' table, whose memory the compiler does not know: with plain ones it
// emits flat accesses, which wait for LDS and its DMA as well.
typedef __attribute__((address_space(1))) uint16_t g_u16;
typedef __attribute__((address_space(1))) float g_f32;
typedef __attribute__((address_space(1))) u32x4 g_u32x4;
typedef __attribute__((address_space(1))) f32x4 g_f32x4;

// ---- DMA of 16 bytes a lane into LDS: lane l of the wave writes `to` + 16 l
__device__ __align__(16) uint32_t g_zeros[4];  // what lanes beyond the end of K load

template <int AUX = 0>
__device__ __forceinline__ void dma(const uint16_t *from, uint8_t *to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from, (__attribute__((address_space(3))) void *)to, 16, 0, AUX);
}
__device__ __forceinline__ void dma(__amdgpu_buffer_rsrc_t from, uint32_t off, uint8_t *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, (int)off, 0, 0, 0);
}

// The adapter's own rank.  Rows of A from it on are not read, and their u is 0 whatever x holds: infinities and NaN
// meet no padding.
__device__ __forceinline__ uint32_t own_rank(const LoraStack &s, uint32_t e) {
  if (!s.ranks) return s.R;
  const uint32_t r = s.ranks[e];
  return uniform32(r < s.R ? r : s.R);
}
// u of four rows from `row`.
__device__ __forceinline__ f32x4 within_rank(f32x4 v, uint32_t row, uint32_t rank) {
#pragma unroll
  for (uint32_t i = 0; i < 4u; ++i) v[i] = row + i < rank ? v[i] : 0.f;
  return v;
}

// ---- groups --------------------------------------------------------------------------------

// A batch of up to 64 rows: whether row i, with id, leads, and then list[0 .. n-1] = the rows of its
// group.  Every wave finds the same and writes the same list.
__device__ __forceinline__ bool gather_rows(uint32_t own, uint32_t i, uint32_t id, uint32_t lane, uint32_t *list, uint32_t &n) {
  const unsigned long long same = __ballot(own == id), next = same >> i << i;
  const uint32_t at = (uint32_t)__popcll(next & ((1ull << lane) - 1ull));
  if ((next >> lane & 1ull) && at < kFew) list[at] = lane;
  n = (uint32_t)__popcll(next);
  if (n > kFew) n = kFew;
  return (uint32_t)__popcll(same ^ next) % kFew == 0u;
}

struct PlanItem {
  uint32_t e;  // adapter; num: rows without one; num + 1: rows with an id outside the pool
  uint32_t n;  // 1 .. kMany
  uint32_t pad[2];
  uint32_t rows[kMany];  // of the batch
};
struct LoraPlan {  // of kLoraPlanRows rows
  uint32_t items;
  uint32_t pad[15];
  PlanItem item[kLoraPlanRows];
};
static_assert(sizeof(LoraPlan) <= kLoraPlanBytes && kLoraPlanBytes % 256u == 0, "workspace");

// Sorts the rows of a piece of the batch into groups; a thread has a row.  Rows with the same id
// find each other in their wave by ballots over the id's bits, then across the waves by a
// hash table in LDS with a count of each wave.  A row's place among the rows with its id goes by
// their order in the batch, and so does the cut into groups; only where a group lies in the
// plan depends on the atomics' order, and no result does.
__global__ __launch_bounds__(kLoraPlanRows) void k_plan(const uint32_t *__restrict__ ids, uint32_t m, uint32_t num, uint32_t bits,
                                                        LoraPlan *__restrict__ plans) {
  constexpr uint32_t kSlots = 2u * kLoraPlanRows, kWaves = kLoraPlanRows / 64u, kEmpty = 0xFFFFFFFFu;
  static_assert(kWaves == 16u, "a slot's counts are 16 bytes");
  __shared__ uint32_t key[kSlots];
  __shared__ __attribute__((aligned(16))) uint8_t count[kSlots][kWaves];
  __shared__ uint32_t item0[kSlots];
  __shared__ uint32_t items;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6, t = blockIdx.x * kLoraPlanRows + tid;
  LoraPlan &plan = plans[blockIdx.x];
  const bool live = t < m;
  const uint32_t id = live ? ids[t] : 0u, e = id < num ? id : id == INT8W_NO_ADAPTER ? num : num + 1u;
  for (uint32_t i = tid; i < kSlots; i += kLoraPlanRows) {
    key[i] = kEmpty;
    *reinterpret_cast<uint4 *>(count[i]) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (tid == 0u) items = 0u;
  __syncthreads();
  unsigned long long same = __ballot(live);
  for (uint32_t b = 0; b < bits; ++b) {
    const unsigned long long set = __ballot(e >> b & 1u);
    same &= e >> b & 1u ? set : ~set;
  }
  const uint32_t leader = live ? (uint32_t)__builtin_ctzll(same) : lane;
  uint32_t slot = 0;
  if (live && lane == leader) {
    slot = e * 2654435761u >> 21;  // of 2048; at most 1024 are taken, so a free one is found
    while (true) {
      const uint32_t was = atomicCAS(&key[slot], kEmpty, e);
      if (was == kEmpty || was == e) break;
      slot = (slot + 1u) % kSlots;
    }
    count[slot][wave] = (uint8_t)__popcll(same);
  }
  slot = (uint32_t)__shfl((int)slot, (int)leader, 64);
  __syncthreads();
  uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1ull)), total = 0;
  const u32x4 c = *reinterpret_cast<const u32x4 *>(count[slot]);
#pragma unroll
  for (uint32_t w = 0; w < kWaves; ++w) {
    const uint32_t n = c[w / 4u] >> 8u * (w % 4u) & 0xFFu;
    total += n;
    if (w < wave) rank += n;
  }
  if (live && rank == 0u) item0[slot] = atomicAdd(&items, (total + kMany - 1u) / kMany);
  __syncthreads();
  if (live) {
    PlanItem &it = plan.item[item0[slot] + rank / kMany];
    it.rows[rank % kMany] = t;
    if (rank % kMany == 0u) {
      it.e = e;
      it.n = total - rank < kMany ? total - rank : kMany;
    }
  }
  if (tid == 0u) plan.items = items;
}

// The groups of up to 64 plans, one after the other, as every workgroup that works on them sees them.
struct Groups {
  const LoraPlan *plans;
  uint32_t until;  // lane p: groups of plans 0 .. p
  uint32_t total;
  __device__ __forceinline__ Groups(const LoraArgs &g, uint32_t plan0, uint32_t lane) {
    plans = reinterpret_cast<const LoraPlan *>(g.plans) + plan0;
    const uint32_t have = (g.m + kLoraPlanRows - 1u) / kLoraPlanRows - plan0;
    until = lane < have ? plans[lane].items : 0u;
#pragma unroll
    for (uint32_t off = 1; off < 64u; off <<= 1) {
      const uint32_t up = (uint32_t)__shfl_up((int)until, off, 64);
      if (lane >= off) until += up;
    }
    total = (uint32_t)__builtin_amdgcn_readlane((int)until, 63);
  }
  // Parts of K, one workgroup of shrink to each where there are that many: shrink and expand find the same.
  __device__ __forceinline__ uint32_t parts(const LoraArgs &g, uint32_t &steps) const {
    uint32_t n = kShrinkBlocks / total;
    n = n < 1u ? 1u : n > g.parts ? g.parts : n;
    const uint32_t all = (g.K + kStepK - 1u) / kStepK;
    steps = (all + n - 1u) / n;
    return (all + steps - 1u) / steps;
  }
  // Group i: f(adapter, n) with its rows in `list`.
  template <class F>
  __device__ __forceinline__ void with(uint32_t i, uint32_t *list, F f) const {
    const uint32_t p = (uint32_t)__popcll(__ballot(until <= i));
    const uint32_t before = p ? (uint32_t)__builtin_amdgcn_readlane((int)until, (int)(p - 1u)) : 0u;
    const PlanItem &it = plans[p].item[i - before];
    const uint32_t row = threadIdx.x < kMany ? it.rows[threadIdx.x] : 0u;  // beyond n: no row, unused
    const uint32_t e = uniform32(it.e), n = uniform32(it.n);
    __syncthreads();  // the last group is done with
    if (threadIdx.x < kMany) list[threadIdx.x] = row;
    __syncthreads();
    f(e, n);
  }
};

// f(i) for this workgroup's share of 0 .. end - 1: an eighth in a row to the workgroups of each XCD (the grid
// is a multiple of 8).  With a part of K or a run of columns of all groups after the other, an XCD's L2 sees an eighth
// of the adapters' matrices, and groups of many rows and of few are spread evenly.
template <class F>
__device__ __forceinline__ void each_share(uint32_t end, F f) {
  const uint32_t per = (end + 7u) / 8u, from = blockIdx.x % 8u * per, until = from + per < end ? from + per : end;
  for (uint32_t i = from + blockIdx.x / 8u; i < until; i += gridDim.x / 8u) f(i);
}

// ---- shrink --------------------------------------------------------------------------------
// A load in the layout of a matrix operand, neighbouring lanes in different rows, costs the
// address unit a cycle a lane.  So rows come by DMA, eight lanes side by side on a row's cache
// line (64 values, a step of K), and are read from LDS as operands.  Chunk p (16 bytes) of
// row r lies at chunk row_swizzle<8>(r, p) of its row: no bank conflicts.

// Operand `half` (32 of the 64 values) of 16 rows: row l%16, chunk 4 half + l/16.
__device__ __forceinline__ u32x4 get_rows(const uint8_t *lds, uint32_t half, uint32_t lane) {
  const uint32_t r = lane & 15u;
  return *reinterpret_cast<const u32x4 *>(lds + 128u * r + 16u * row_swizzle<8>(r, 4u * half + (lane >> 4)));
}
// Byte offset of chunk p of row r of A at K 0 (from which K's, below 2^22, stays out of range).
__device__ __forceinline__ uint32_t a_offset(uint32_t r, uint32_t rank, uint32_t K, uint32_t p) {
  const uint32_t at = (r * K + 8u * p) * 2u;
  return r < rank ? at : kOutOfRange;
}

// A part of K.
struct PartK {
  uint32_t part, first, end, steps;
  __device__ __forceinline__ PartK(const LoraArgs &g, uint32_t part_, uint32_t part_steps) {
    part = part_;
    first = part * part_steps * kStepK;
    end = first + part_steps * kStepK < g.K ? first + part_steps * kStepK : g.K;
    steps = (end - first + kStepK - 1u) / kStepK;
  }
  __device__ __forceinline__ uint32_t at(uint32_t step) const { return step < steps ? first + step * kStepK : end; }
};

// u of the n <= 16 rows in `list` (LDS, may lie where lds does), this part of K.  The four waves
// take steps in turn, each with two stages of its own in LDS; their sums are added up there.
template <int RT>  // 16-row tiles of A at a time
struct ShrinkFew {
  static constexpr uint32_t kStage = (RT + 1) * 2048u;  // A, then x
  static constexpr uint32_t kLds = 4u * 2u * kStage;
  static __device__ __forceinline__ void run(const LoraArgs &g, const LoraStack &s, uint32_t e, const uint32_t *list, uint32_t n,
                                             const PartK &part_k, uint8_t *lds, uint32_t lane, uint32_t wave) {
    const uint32_t r = lane >> 3, rank = own_rank(s, e);
    uint8_t *const mine = lds + wave * 2u * kStage;
    // load j: rows 8 j + l/8; chunk l%8 in LDS is this one of the row
    const uint32_t p0 = 8u * row_swizzle<8>(r, lane & 7u), p1 = 8u * row_swizzle<8>(8u + r, lane & 7u);
    const uint16_t *const x0 = g.x + list[r < n ? r : 0u] * g.x_stride + p0;  // rows from n on: any, unused
    const uint16_t *const x1 = g.x + list[8u + r < n ? 8u + r : 0u] * g.x_stride + p1;
    const uint32_t out_row = list[(threadIdx.x & 15u) < n ? threadIdx.x & 15u : 0u];
    __syncthreads();
    const auto ra = make_rsrc(s.a + (size_t)e * s.R * g.K, s.R * g.K * 2u);
    const bool more = n > 8u;
    for (uint32_t r0 = 0; r0 < s.R; r0 += 16u * RT) {
      f32x4 acc[RT] = {};
      uint32_t oa[2 * RT];
#pragma unroll
      for (uint32_t j = 0; j < 2u * RT; ++j) oa[j] = a_offset(r0 + 8u * j + r, rank, g.K, (j & 1u ? p1 : p0) / 8u);
      auto load = [&](uint32_t step, uint8_t *to) {  // beyond the part: zeros, without touching A or x
        const uint32_t at = part_k.at(step);
        const bool in0 = at + p0 < part_k.end, in1 = at + p1 < part_k.end;
#pragma unroll
        for (uint32_t j = 0; j < 2u * RT; ++j) dma(ra, (j & 1u ? in1 : in0) ? oa[j] + 2u * at : kOutOfRange, to + 1024u * j);
        dma(in0 ? x0 + at : (const uint16_t *)g_zeros, to + 2048u * RT);
        if (more) dma(in1 ? x1 + at : (const uint16_t *)g_zeros, to + 2048u * RT + 1024u);
      };
      auto step = [&](uint8_t *at, uint32_t next) {  // one stage: await, read, refill, multiply
        if (more)
          INT8W_VMCNT(2 * RT + 2);
        else
          INT8W_VMCNT(2 * RT + 1);
        keep_order();
        u32x4 a[RT][2], x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h] = get_rows(at + 2048u * RT, h, lane);
#pragma unroll
          for (int t = 0; t < RT; ++t) a[t][h] = get_rows(at + 2048u * t, h, lane);
        }
        INT8W_LGKMCNT0();  // read before it is written again
        keep_order();
        load(next, at);
        keep_order();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[t] = mfma16(a[t][h], x[h], acc[t]);
      };
      uint32_t b = wave;
      if (r0 < rank && b < part_k.steps) {
        load(b, mine);
        load(b + 4u, mine + kStage);
        while (true) {
          step(mine, b + 8u);
          if ((b += 4u) >= part_k.steps) break;
          step(mine + kStage, b + 8u);
          if ((b += 4u) >= part_k.steps) break;
        }
        INT8W_VMCNT(0);  // the look-ahead has landed
      }
      __syncthreads();
      // acc[t]: row 16 t + 4 (l / 16) + i of the tile for row l%16 of the group
      f32x4 *const sums = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
      for (int t = 0; t < RT; ++t) sums[(wave * RT + t) * 64u + lane] = acc[t];
      __syncthreads();
      const uint32_t p = threadIdx.x, row = r0 + 16u * (p >> 6) + 4u * (p >> 4 & 3u);
      if (p < RT * 64u && (p & 15u) < n && row < s.R) {
        f32x4 v = sums[p];
#pragma unroll
        for (uint32_t w = 1; w < 4u; ++w) v += sums[w * RT * 64u + p];
        *(g_f32x4 *)((g_f32 *)s.u + ((size_t)part_k.part * g.m + out_row) * s.R + row) = within_rank(v, row, rank);
      }
      __syncthreads();
    }
  }
};

// The same for up to 64 rows: a wave has 16 of them, A is shared.  NS stages in LDS, one barrier a step.
template <int RT>
struct ShrinkMany {
  static constexpr uint32_t kStage = (RT + 4) * 2048u;  // A, then x
  static constexpr int NS = 4;
  static constexpr uint32_t kLds = NS * kStage;
  static constexpr int kA = RT >= 2 ? RT / 2 : 1;  // loads of A a wave (of one tile: waves 2 and 3 repeat them)
  static __device__ __forceinline__ void run(const LoraArgs &g, const LoraStack &s, uint32_t e, const uint32_t *list, uint32_t n,
                                             const PartK &part_k, uint8_t *lds, uint32_t lane, uint32_t wave) {
    const uint32_t r = lane >> 3, rank = own_rank(s, e);
    const uint32_t p0 = 8u * row_swizzle<8>(r, lane & 7u), p1 = 8u * row_swizzle<8>(8u + r, lane & 7u);
    const uint32_t i0 = 16u * wave + r, i1 = i0 + 8u, io = 16u * wave + (lane & 15u);
    const uint16_t *const x0 = g.x + list[i0 < n ? i0 : 0u] * g.x_stride + p0;
    const uint16_t *const x1 = g.x + list[i1 < n ? i1 : 0u] * g.x_stride + p1;
    const uint32_t out_row = list[io < n ? io : 0u];
    __syncthreads();
    const auto ra = make_rsrc(s.a + (size_t)e * s.R * g.K, s.R * g.K * 2u);
    for (uint32_t r0 = 0; r0 < s.R; r0 += 16u * RT) {
      f32x4 acc[RT] = {};
      if (r0 < rank) {
        uint32_t oa[kA], pa[kA];
#pragma unroll
        for (uint32_t i = 0; i < kA; ++i) {
          const uint32_t j = (wave * kA + i) % (2u * RT);
          pa[i] = j & 1u ? p1 : p0;
          oa[i] = a_offset(r0 + 8u * j + r, rank, g.K, pa[i] / 8u);
        }
        auto load = [&](uint32_t step, uint8_t *to) {
          const uint32_t at = part_k.at(step);
#pragma unroll
          for (uint32_t i = 0; i < kA; ++i)
            dma(ra, at + pa[i] < part_k.end ? oa[i] + 2u * at : kOutOfRange, to + (wave * kA + i) % (2u * RT) * 1024u);
          dma<kAuxNontemporal>(at + p0 < part_k.end ? x0 + at : (const uint16_t *)g_zeros, to + 2048u * RT + 2048u * wave);
          dma<kAuxNontemporal>(at + p1 < part_k.end ? x1 + at : (const uint16_t *)g_zeros, to + 2048u * RT + 2048u * wave + 1024u);
          keep_order();
        };
#pragma unroll
        for (int i = 0; i < NS - 1; ++i) load(i, lds + i * kStage);
        for (uint32_t b = 0; b < part_k.steps;) {
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            // this wave's loads of step b have landed; the barrier makes all of them visible, and frees step b - 1's stage
            INT8W_VMCNT((NS - 2) * (kA + 2));
            INT8W_LGKMCNT0();
            asm volatile("s_barrier" ::: "memory");
            load(b + NS - 1u, lds + (i + NS - 1) % NS * kStage);
            const uint8_t *const at = lds + i * kStage;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const u32x4 x = get_rows(at + 2048u * RT + 2048u * wave, h, lane);
#pragma unroll
              for (int t = 0; t < RT; ++t) acc[t] = mfma16(get_rows(at + 2048u * t, h, lane), x, acc[t]);
            }
            if (++b >= part_k.steps) break;
          }
        }
        INT8W_VMCNT(0);  // the look-ahead has landed
        __syncthreads();
      }
#pragma unroll
      for (uint32_t t = 0; t < RT; ++t) {
        const uint32_t row = r0 + 16u * t + 4u * (lane >> 4);
        if (io < n && row < s.R)
          *(g_f32x4 *)((g_f32 *)s.u + ((size_t)part_k.part * g.m + out_row) * s.R + row) = within_rank(acc[t], row, rank);
      }
    }
  }
};

// grid (parts, rows, stacks).
template <int RT>
__global__ __launch_bounds__(256) void k_shrink_rows(const LoraArgs g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t *const list = reinterpret_cast<uint32_t *>(lds);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), i = blockIdx.y;
  const uint32_t own = lane < g.m ? g.ids[lane] : INT8W_NO_ADAPTER, id = (uint32_t)__builtin_amdgcn_readlane((int)own, (int)i);
  uint32_t n;
  if (id >= g.num || !gather_rows(own, i, id, lane, list, n)) return;
  __syncthreads();
  ShrinkFew<RT>::run(g, g.s[blockIdx.z], id, list, n, PartK(g, blockIdx.x, g.part_steps), lds, lane, wave);
}

// grid (blocks, 64 plans, stacks): the blocks take the groups' parts in turn.
template <int RT>
__global__ __launch_bounds__(256) void k_shrink_items(const LoraArgs g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t *const list = reinterpret_cast<uint32_t *>(lds);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6);
  const LoraStack s = g.s[blockIdx.z];
  const Groups groups(g, 64u * blockIdx.y, lane);
  uint32_t steps;
  const uint32_t parts = groups.parts(g, steps), end = groups.total * parts;
  each_share(end, [&](uint32_t i) {
    groups.with(i % groups.total, list, [&](uint32_t e, uint32_t n) {
      if (e >= g.num) return;
      const PartK part_k(g, i / groups.total, steps);
      if (n <= kFew)
        ShrinkFew<RT>::run(g, s, e, list, n, part_k, lds, lane, wave);
      else
        ShrinkMany<RT>::run(g, s, e, list, n, part_k, lds, lane, wave);
    });
  });
}

// ---- expand --------------------------------------------------------------------------------
// The product has u's rows as rows and B's as columns: a result register of lane (c, q) holds row
// 4 q + i, column c of a tile.  Tile t of a block's eight takes columns 8 c + t, so that a lane
// has eight neighbouring columns and 16 lanes a row's 256 bytes.
// A block of B, 128 columns, comes by DMA, P chunks of 16 bytes a column at a time (P = 2 or 4: the
// whole rank; 8: 64 of it).  LDS row 16 t + c is column 8 c + t.

template <int P>
__device__ __forceinline__ uint32_t b_swizzle(uint32_t c, uint32_t p) {  // as quarter_at() for 4
  if constexpr (P == 2) return p;
  if constexpr (P == 4) return p ^ ((c >> 1) & 3u);
  return row_swizzle<8>(c, p);
}

// Load j of the 2 P of a block's rank chunk r0.  n0: its first column.  Columns of B beyond the adapter's own rank,
// zeros, are read: they lie in the same cache lines up to rank 64, and the first loads do not wait for the rank.
template <int P>
__device__ __forceinline__ void dma_b(__amdgpu_buffer_rsrc_t rb, uint32_t R, uint32_t n0, uint32_t r0, uint32_t j, uint8_t *to,
                                      uint32_t lane) {
  const uint32_t row = (64u * j + lane) / P, c = row & 15u, t = row >> 4;
  const uint32_t r = r0 + 8u * b_swizzle<P>(c, lane % P), n = n0 + 8u * c + t;  // a column past the last one: zeros by the resource
  dma(rb, r < R ? (n * R + r) * 2u : kOutOfRange, to + 1024u * j);
}

// u of 16 rows as operands: lane (c, q) of row c.  P = 2: one operand, the upper BF16 values in
// lane groups 0 and 1, the lower in 2 and 3, against the same columns of B in both.
template <int P, int NCH>
struct UOperand {
  static constexpr int kSteps = P == 8 ? 2 : 1, kAll = kSteps * NCH;
  u32x4 hi[kAll], lo[P == 2 ? 1 : kAll];
};

// Two BF16 values that add up to each of four.  The upper one is at most BF16's largest, so that a value beyond that,
// an infinity or a NaN is in the lower one.
__device__ __forceinline__ void split_bf16(const f32x4 &v, u32x2 &hi, u32x2 &lo) {
  constexpr float kMost = 0x1.FEp127f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    hi[i] = pack_bf16x2(fminf(fmaxf(v[2 * i], -kMost), kMost), fminf(fmaxf(v[2 * i + 1], -kMost), kMost));
    lo[i] = pack_bf16x2(v[2 * i] - bf16_lo(hi[i]), v[2 * i + 1] - bf16_hi(hi[i]));
  }
}

// COUNT pieces of four values of u, piece i of row(i) from offset at(i) of it: the parts added in their order.
// All pieces of several parts are in flight at a time.
template <int COUNT, class Row, class At>
__device__ __forceinline__ void sum_parts(f32x4 (&v)[COUNT], const LoraArgs &g, const LoraStack &s, uint32_t parts, Row row,
                                          At at) {
  constexpr uint32_t kAhead = 8 / COUNT;
  const size_t next = (size_t)g.m * s.R;
  const g_f32 *from[COUNT];
  bool have[COUNT];
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    have[i] = row(i) < g.m && at(i) < s.R;
    from[i] = (const g_f32 *)s.u + (have[i] ? (size_t)row(i) * s.R + at(i) : 0u);
  }
  for (uint32_t p = 0; p < parts; p += kAhead) {
    f32x4 w[kAhead][COUNT];
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < COUNT; ++i) {
        w[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (p + j < parts && have[i]) w[j][i] = *(const g_f32x4 *)(from[i] + (p + j) * next);
      }
    keep_order();
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] += w[j][i];
  }
}

// Whether eight columns of a row from a multiple of 8 are a 16-byte access.
__device__ __forceinline__ bool wide_rows(const LoraStack &s) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(s.y) | (s.y_stride * 2u) | reinterpret_cast<uintptr_t>(s.base) |
                       (s.base ? s.base_stride * 2u : 0u);
  return (at & 15u) == 0u;
}

// Four rows of a lane: y = base + scale v for eight columns from n.
struct OutRows {
  const g_u16 *base[4];
  g_u16 *y[4];
  bool have[4];
  bool wide;  // 16-byte accesses are aligned
  uint32_t N;
  bool read;
  float scale;  // last, as in k_solo: times u it might pass fp32's range where the product does not
  __device__ __forceinline__ OutRows(const LoraStack &s, float scale_, const uint32_t *list, uint32_t i0, uint32_t n) {
    scale = scale_;
    wide = wide_rows(s);
    read = s.base != nullptr;
    N = s.N;
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
      have[i] = i0 + i < n;
      const uint64_t row = list[have[i] ? i0 + i : 0u];
      base[i] = read ? (const g_u16 *)s.base + row * s.base_stride : (const g_u16 *)(const void *)g_zeros;
      y[i] = (g_u16 *)s.y + row * s.y_stride;
    }
  }
  // Without a branch, and from somewhere in any case: otherwise the compiler waits for all that is in
  // flight, stores too, before it sets the registers of a load that may not happen.
  __device__ __forceinline__ void load(u32x4 (&o)[4], uint32_t n) const {
    if (!wide) return;
    const uint32_t at = read && n + 8u <= N ? n : 0u;
    const bool some = !read || N >= 8u;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = *(const g_u32x4 *)(some ? base[i] + at : (const g_u16 *)(const void *)g_zeros);
  }
  // v[t][i]: row i, column n + t
  __device__ __forceinline__ void add(const u32x4 (&o)[4], const f32x4 (&v)[8], uint32_t n) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!have[i]) continue;
      if (wide && n + 8u <= N) {
        u32x4 w;
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = pack_bf16x2(__builtin_fmaf(scale, v[2 * t][i], bf16_lo(o[i][t])), __builtin_fmaf(scale, v[2 * t + 1][i], bf16_hi(o[i][t])));
        *(g_u32x4 *)(y[i] + n) = w;
      } else {
#pragma unroll
        for (uint32_t t = 0; t < 8u; ++t)
          if (n + t < N) y[i][n + t] = to_bf16_bits(__builtin_fmaf(scale, v[t][i], read ? bf16_bits_to_f32(base[i][n + t]) : 0.f));
      }
    }
  }
};

// Rows without an adapter (base itself) or with an id outside the pool (NaN), columns [n0, end): pieces
// of eight columns, four a thread in flight.
__device__ __forceinline__ void pass_rows(const LoraStack &s, const uint32_t *list, uint32_t n, bool nan, uint32_t n0, uint32_t end) {
  if (!nan && s.base == s.y) return;  // in place
  const bool read = !nan && s.base != nullptr, wide = wide_rows(s);
  const uint32_t across = (end - n0 + 7u) / 8u, all = n * across;
  for (uint32_t p0 = threadIdx.x; p0 < all; p0 += 4u * 256u) {
    u32x4 v[4];
    uint64_t row[4];
    uint32_t c[4];
#pragma unroll
    for (uint32_t j = 0; j < 4u; ++j) {
      const uint32_t p = p0 + 256u * j < all ? p0 + 256u * j : p0;
      row[j] = list[p / across];
      c[j] = n0 + 8u * (p % across);
      v[j] = nan ? u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u} : u32x4{0u, 0u, 0u, 0u};
      if (!read) continue;
      const g_u16 *const from = (const g_u16 *)s.base + row[j] * s.base_stride + c[j];
      if (wide && c[j] + 8u <= end) {
        v[j] = *(const g_u32x4 *)from;
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 8u; ++i)
          if (c[j] + i < end) v[j][i / 2u] |= (uint32_t)from[i] << 16u * (i % 2u);
      }
    }
    keep_order();
#pragma unroll
    for (uint32_t j = 0; j < 4u; ++j) {  // a piece past the last one: the first again
      g_u16 *const to = (g_u16 *)s.y + row[j] * s.y_stride + c[j];
      if (wide && c[j] + 8u <= end) {
        *(g_u32x4 *)to = v[j];
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 8u; ++i)
          if (c[j] + i < end) to[i] = (uint16_t)(v[j][i / 2u] >> 16u * (i % 2u));
      }
    }
  }
}

template <int P, int NCH>
__device__ __forceinline__ void multiply_block(f32x4 (&acc)[8], const UOperand<P, NCH> &u, int ch, const uint8_t *b, uint32_t lane) {
  const uint32_t c = lane & 15u, q = lane >> 4;
#pragma unroll
  for (int k = 0; k < UOperand<P, NCH>::kSteps; ++k) {
    const uint8_t *const at = b + 16u * (c * P + b_swizzle<P>(c, P == 2 ? q & 1u : 4u * k + q));
    const int i = UOperand<P, NCH>::kSteps * ch + k;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const u32x4 bt = *reinterpret_cast<const u32x4 *>(at + 256u * P * t);
      acc[t] = mfma16(u.hi[i], bt, acc[t]);
      if constexpr (P != 2) acc[t] = mfma16(u.lo[i], bt, acc[t]);
    }
  }
}

// The n <= 16 rows in `list`, columns n0 .. n0 + 511: a wave has 128 of them.  u goes through LDS,
// where all 256 threads have summed its parts.
template <int P, int NCH>
struct ExpandFew {
  typedef UOperand<P, NCH> U;
  static constexpr uint32_t kBlock = 2048u * P;             // of B, a wave
  static constexpr uint32_t kRanks = 8u * P * NCH;          // largest rank
  static constexpr uint32_t kRow = 2u * kRanks + 16u;       // a row of u, padded: banks
  static constexpr uint32_t kList = 4u * kBlock + 2u * kFew * kRow, kLds = kList + 4u * kFew;
  static constexpr uint32_t kColumns = 4u * kBlockN;
  static __device__ __forceinline__ void run(const LoraArgs &g, const LoraStack &s, uint32_t e, const uint32_t *list, uint32_t n,
                                             uint32_t n0, uint8_t *lds, uint32_t lane, uint32_t wave) {
    const uint32_t c = lane & 15u, q = lane >> 4, w0 = n0 + kBlockN * wave;
    uint8_t *const b = lds + kBlock * wave, *const hi = lds + 4u * kBlock, *const lo = hi + kFew * kRow;
    const auto rb = make_rsrc(s.b + (size_t)e * s.N * s.R, s.N * s.R * 2u);
#pragma unroll
    for (uint32_t j = 0; j < 2u * P; ++j) dma_b<P>(rb, s.R, w0, 0u, j, b, lane);
    const OutRows out(s, s.scales ? s.scales[e] : 1.f, list, 4u * q, n);
    u32x4 o[4];
    out.load(o, w0 + 8u * c);
    for (uint32_t p = threadIdx.x; p < kFew * kRanks / 4u; p += 256u) {
      const uint32_t i = p / (kRanks / 4u), r = 4u * (p % (kRanks / 4u)), from = i < n ? list[i] : g.m;
      f32x4 v[1];
      sum_parts(v, g, s, g.parts, [&](int) { return from; }, [&](int) { return r; });
      u32x2 h, l;
      split_bf16(v[0], h, l);
      *reinterpret_cast<u32x2 *>(hi + i * kRow + 2u * r) = h;
      *reinterpret_cast<u32x2 *>(lo + i * kRow + 2u * r) = l;
    }
    __syncthreads();
    U u;
#pragma unroll
    for (int k = 0; k < U::kAll; ++k) {
      if constexpr (P == 2) {
        u.hi[0] = *reinterpret_cast<const u32x4 *>((q < 2u ? hi : lo) + c * kRow + 16u * (q & 1u));
      } else {
        u.hi[k] = *reinterpret_cast<const u32x4 *>(hi + c * kRow + 64u * k + 16u * q);
        u.lo[k] = *reinterpret_cast<const u32x4 *>(lo + c * kRow + 64u * k + 16u * q);
      }
    }
    f32x4 acc[8] = {};
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch) {
      if (64u * ch >= s.R) break;
      INT8W_VMCNT(0);
      keep_order();
      multiply_block<P, NCH>(acc, u, ch, b, lane);
      if (ch + 1 < NCH) {
        INT8W_LGKMCNT0();
        keep_order();
#pragma unroll
        for (uint32_t j = 0; j < 2u * P; ++j) dma_b<P>(rb, s.R, w0, 64u * (ch + 1), j, b, lane);
      }
    }
    out.add(o, acc, w0 + 8u * c);
  }
};

// Up to 64 rows, columns [n0, end): a wave has 16 of the rows, blocks of B are shared, one ahead.
template <int P, int NCH>
struct ExpandMany {
  typedef UOperand<P, NCH> U;
  static constexpr uint32_t kBlock = 2048u * P;
  static constexpr uint32_t kList = 2u * kBlock, kLds = kList + 4u * kMany;
  static __device__ __forceinline__ void run(const LoraArgs &g, const LoraStack &s, uint32_t e, const uint32_t *list, uint32_t n,
                                             uint32_t parts, uint32_t n0, uint32_t end, uint8_t *lds, uint32_t lane, uint32_t wave) {
    // Without this the lane's many places in LDS are all kept in registers over the loop around the
    // call, 40 to 60 of which then spill.
    asm volatile("" : "+v"(lane));
    const uint32_t c = lane & 15u, q = lane >> 4;
    const auto rb = make_rsrc(s.b + (size_t)e * s.N * s.R, s.N * s.R * 2u);
    const float scale = s.scales ? s.scales[e] : 1.f;
    const bool idle = 16u * wave >= n;  // a wave without a row loads its share of B
    const uint32_t blocks = (end - n0 + kBlockN - 1u) / kBlockN;
    // Blocks from one that differs from workgroup to workgroup: the same columns of all rows tend to lie in
    // the same memory channels.
    const uint32_t turn = blockIdx.x % blocks;
    auto column = [&](uint32_t i) { return n0 + kBlockN * (i + turn < blocks ? i + turn : i + turn - blocks); };
    auto load_b = [&](uint32_t block, int ch, uint8_t *to) {
#pragma unroll
      for (uint32_t i = 0; i < P / 2u; ++i) dma_b<P>(rb, s.R, column(block), 64u * ch, wave * (P / 2u) + i, to, lane);
    };
    load_b(0, 0, lds);
    keep_order();
    // u of the wave's rows, by way of the second stage: summed with neighbouring lanes on a row
    U u;
    uint8_t *const hi = lds + kBlock + kBlock / 8u * wave, *const lo = hi + kBlock / 2u;
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch) {
      constexpr int kPieces = P / 2;  // a lane: 16 rows of 8 P values
      f32x4 v[kPieces];
      auto piece = [&](int i) { return 64u * i + lane; };
      sum_parts(v, g, s, parts,
                [&](int i) {
                  const uint32_t at = 16u * wave + piece(i) / (2u * P);
                  return at < n ? list[at] : g.m;
                },
                [&](int i) { return 64u * ch + 4u * (piece(i) % (2u * P)); });
      wave_fence();
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint32_t r = piece(i) / (2u * P), half = piece(i) % (2u * P), to = 16u * (r * P + b_swizzle<P>(r, half >> 1)) + 8u * (half & 1u);
        u32x2 h, l;
        split_bf16(v[i], h, l);
        *reinterpret_cast<u32x2 *>(hi + to) = h;
        *reinterpret_cast<u32x2 *>(lo + to) = l;
      }
      wave_fence();
#pragma unroll
      for (int k = 0; k < U::kSteps; ++k) {
        const uint32_t from = 16u * (c * P + b_swizzle<P>(c, P == 2 ? q & 1u : 4u * k + q));
        const int i = U::kSteps * ch + k;
        if constexpr (P == 2) {
          u.hi[0] = *reinterpret_cast<const u32x4 *>((q < 2u ? hi : lo) + from);
        } else {
          u.hi[i] = *reinterpret_cast<const u32x4 *>(hi + from);
          u.lo[i] = *reinterpret_cast<const u32x4 *>(lo + from);
        }
      }
    }
    const OutRows out(s, scale, list, 16u * wave + 4u * q, n);
    f32x4 acc[8];
    u32x4 o[4];
    // One chunk of a block's rank, from stage `at`; the next one goes to `other`.  Two stages with constant places: the
    // compiler can then tell the DMA's writes from this chunk's reads, and does not wait for them.
    const uint32_t rows = 16u * wave < n ? n - 16u * wave : 0u, full_stores = out.wide ? rows < 4u ? rows : 4u : 0u;
    uint32_t stores = 0;  // at least so many of the last block follow the DMA that is waited for, and may go on
    auto chunk = [&](uint32_t i, int ch, const uint8_t *at, uint8_t *other) {
      switch (ch == 0 ? stores : 0u) {
        case 0: INT8W_VMCNT(0); break;
        case 1: INT8W_VMCNT(1); break;
        case 2: INT8W_VMCNT(2); break;
        case 3: INT8W_VMCNT(3); break;
        default: INT8W_VMCNT(4); break;
      }
      INT8W_LGKMCNT0();
      asm volatile("s_barrier" ::: "memory");  // this chunk is there for all waves, the other stage is done with
      if (ch == 0) {
        out.load(o, column(i) + 8u * c);
#pragma unroll
        for (int t = 0; t < 8; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      if (ch + 1 < NCH)
        load_b(i, ch + 1, other);
      else if (i + 1u < blocks)
        load_b(i + 1u, 0, other);
      keep_order();
      if (!idle) multiply_block<P, NCH>(acc, u, ch, at, lane);
      if (ch + 1 == NCH) {
        out.add(o, acc, column(i) + 8u * c);
        stores = column(i) + kBlockN <= s.N ? full_stores : 0u;
      }
    };
    for (uint32_t i = 0; i < blocks;) {
      if constexpr (NCH == 1) {
        chunk(i, 0, lds, lds + kBlock);
        if (++i == blocks) break;
        chunk(i, 0, lds + kBlock, lds);
      } else {
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) chunk(i, ch, lds + (ch & 1) * kBlock, lds + (~ch & 1) * kBlock);
      }
      ++i;
    }
    __syncthreads();
  }
};

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

// grid (column tiles of all stacks, rows).
template <int P, int NCH>
__global__ __launch_bounds__(256) void k_expand_rows(const LoraArgs g) {
  typedef ExpandFew<P, NCH> Few;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t *const list = reinterpret_cast<uint32_t *>(lds + Few::kList);
  uint32_t tile = blockIdx.x;
  const LoraStack s = stack_of(g, tile, Few::kColumns);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6), i = blockIdx.y, n0 = tile * Few::kColumns;
  const uint32_t own = lane < g.m ? g.ids[lane] : INT8W_NO_ADAPTER, id = (uint32_t)__builtin_amdgcn_readlane((int)own, (int)i);
  if (id >= g.num) {
    pass_rows(s, &i, 1u, id != INT8W_NO_ADAPTER, n0, n0 + Few::kColumns < s.N ? n0 + Few::kColumns : s.N);
    return;
  }
  uint32_t n;
  if (!gather_rows(own, i, id, lane, list, n)) return;
  __syncthreads();
  Few::run(g, s, id, list, n, n0, lds, lane, wave);
}

// grid (blocks, 64 plans): the blocks take the groups' runs of 128-column blocks (the stacks' one after the
// other) in turn, as many runs as give each workgroup one.
template <int P, int NCH>
__global__ __launch_bounds__(256, NCH == 1 ? 4 : 2) void k_expand_items(const LoraArgs g, uint32_t column_blocks) {
  // one dynamic array: behind a static one of its own the compiler waits for the DMA before every read
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t *const list = reinterpret_cast<uint32_t *>(lds + ExpandMany<P, NCH>::kList);
  const uint32_t lane = threadIdx.x & 63u, wave = uniform32(threadIdx.x >> 6);
  const Groups groups(g, 64u * blockIdx.y, lane);
  uint32_t steps;
  const uint32_t parts = groups.parts(g, steps);
  uint32_t runs = gridDim.x / groups.total;
  runs = runs < 1u ? 1u : runs > column_blocks ? column_blocks : runs;
  const uint32_t run = (column_blocks + runs - 1u) / runs;
  runs = (column_blocks + run - 1u) / run;
  const auto work = [&](uint32_t group, uint32_t at_run) {
    groups.with(group, list, [&](uint32_t e, uint32_t n) {
      uint32_t at = at_run * run, left = run;
      for (uint32_t k = 0; k < g.count && left; ++k) {
        const LoraStack s = g.s[k];
        const uint32_t blocks = (s.N + kBlockN - 1u) / kBlockN;
        if (at >= blocks) {
          at -= blocks;
          continue;
        }
        const uint32_t here = left < blocks - at ? left : blocks - at, n0 = at * kBlockN;
        const uint32_t end = n0 + here * kBlockN < s.N ? n0 + here * kBlockN : s.N;
        if (e >= g.num)
          pass_rows(s, list, n, e != g.num, n0, end);
        else
          ExpandMany<P, NCH>::run(g, s, e, list, n, parts, n0, end, lds, lane, wave);
        at = 0;
        left -= here;
      }
    });
  };
  // A group to an XCD, whose u then comes into one L2, or some columns of all groups to an XCD.  The first pays where u is much
  // of what is read: many rows of a large rank, or few columns.  On wide outputs of small u it loses, and with fewer
  // than three groups each the XCDs are unevenly loaded.  us of whole calls so / the other way, K 4096: 57 groups of 64 rows, 4096 columns,
  // rank 64 43 / 51, rank 16 28.0 / 29.1, rank 128 72 / 84; 64 of 64, 8192 columns, rank 64 62 / 75; 57 of 4 rows, 4096 columns (K
  // 14336), rank 64 43.4 / 44.1; 64 of 17, 2 x 14336 columns, rank 16 76 / 62; 80 of 17, 14336, rank 32 62 / 51; 12 of 64, 14336, rank
  // 64 30.6 / 28.1.  Over 850 such sizes this rule is within 0.5 % of the better one on average (16 % at worst), either alone 1.7 (26).
  // All groups of an XCD at one run of columns before the next: 8192 rows 110 instead of 113, 2109 18.6 for 17.9.
  constexpr uint32_t kRows = 64u * kLoraPlanRows;  // of a round of plans
  const uint32_t rows = g.m - kRows * blockIdx.y < kRows ? g.m - kRows * blockIdx.y : kRows;
  if (groups.total >= kXcdGroups && (column_blocks * kBlockN <= kXcdColumns || rows * (8u * P * NCH) >= kXcdValues * groups.total)) {
    for (uint32_t j = blockIdx.x / 8u;; j += gridDim.x / 8u) {
      const uint32_t group = j / runs * 8u + blockIdx.x % 8u;
      if (group >= groups.total) break;
      work(group, j % runs);
    }
  } else {
    each_share(groups.total * runs, [&](uint32_t i) { work(i % groups.total, i / groups.total); });
  }
}

// ---- one launch for a few rows ---------------------------------------------------------------
// A workgroup of 16 waves forms all of u for its row, on the vector ALUs with rows of A as they lie in memory, and
// then 512 columns of y: A is read again for each 512 columns, out of the caches, which costs less than a
// second launch as long as it is small.  u stays in fp32.
constexpr uint32_t kSoloColumns = 512;
constexpr uint32_t kSoloK = 16384;  // most of x in LDS

// P2: 16-byte pieces of a column of B a thread, two threads a column (rank up to 16 P2).
template <int P2>
__global__ __launch_bounds__(1024) void k_solo(const LoraArgs g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // x
  __shared__ __attribute__((aligned(16))) float u[16 * P2];
  __shared__ float half_u[16];
  constexpr uint32_t kChunk = 512, kAhead = 8;  // values of a row a load of the wave; loads in flight
  uint32_t tile = blockIdx.x;
  const LoraStack s = stack_of(g, tile, kSoloColumns);
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = uniform32(tid >> 6), i = blockIdx.y, n0 = tile * kSoloColumns;
  const uint32_t id = uniform32(g.ids[i]);
  const g_u16 *const x = (const g_u16 *)g.x + i * g.x_stride;
  for (uint32_t p = 8u * tid; p < g.K; p += 8u * 1024u) *reinterpret_cast<u32x4 *>(lds + 2u * p) = *(const g_u32x4 *)(x + p);
  if (id >= g.num) {
    const uint32_t row[1] = {i}, end = n0 + kSoloColumns < s.N ? n0 + kSoloColumns : s.N;
    if (tid < 256u) pass_rows(s, row, 1u, id != INT8W_NO_ADAPTER, n0, end);
    return;
  }
  const uint32_t rank = own_rank(s, id), n = n0 + tid / 2u;
  const float scale = s.scales ? s.scales[id] : 1.f;
  // this thread's part of its column of B, and base, while A comes
  u32x4 b[P2];
  const auto rb = make_rsrc(s.b + (size_t)id * s.N * s.R, s.N * s.R * 2u);
#pragma unroll
  for (uint32_t j = 0; j < P2; ++j) {
    const uint32_t r = 8u * (P2 * (tid & 1u) + j);
    b[j] = buf_load_b128(rb, r < rank ? (n * s.R + r) * 2u : kOutOfRange);  // past the last column: zeros
  }
  const bool write = (tid & 1u) == 0u && n < s.N;
  const float base = write && s.base ? bf16_bits_to_f32(((const g_u16 *)s.base)[i * s.base_stride + n]) : 0.f;
  keep_order();
  // rows of A: a wave has row wave, wave + 16, ..; of eight rows two waves share each, a half of K apiece
  const bool halves = s.R == 8u;
  const uint32_t chunks = (g.K + kChunk - 1u) / kChunk, c0 = halves && wave >= 8u ? chunks / 2u : 0u, c1 = halves && wave < 8u ? chunks / 2u : chunks;
  const auto ra = make_rsrc(s.a + (size_t)id * s.R * g.K, s.R * g.K * 2u);
  bool staged = false;
  for (uint32_t r = halves ? wave % 8u : wave; r < s.R; r += 16u) {
    float sum = 0.f;
    for (uint32_t c = c0; c < c1 && r < rank; c += kAhead) {
      u32x4 a[kAhead];
#pragma unroll
      for (uint32_t j = 0; j < kAhead; ++j) {
        const uint32_t k = (c + j) * kChunk + 8u * lane;
        a[j] = buf_load_b128(ra, c + j < c1 && k < g.K ? (r * g.K + k) * 2u : kOutOfRange);
      }
      keep_order();
      if (!staged) {
        __syncthreads();
        staged = true;
      }
#pragma unroll
      for (uint32_t j = 0; j < kAhead; ++j) {
        const uint32_t k = (c + j) * kChunk + 8u * lane;
        if (c + j < c1 && k < g.K) {
          const u32x4 v = *reinterpret_cast<const u32x4 *>(lds + 2u * k);
#pragma unroll
          for (int t = 0; t < 4; ++t) sum = dot2(a[j][t], v[t], sum);
        }
      }
    }
    sum = token_sum(sum);
    if (lane == 0u) {
      if (halves && wave >= 8u)
        half_u[r] = sum;
      else
        u[r] = sum;
    }
  }
  if (!staged) __syncthreads();
  if (tid >= s.R && tid < 16u * P2) u[tid] = 0.f;
  __syncthreads();
  float v = 0.f;
#pragma unroll
  for (uint32_t j = 0; j < P2; ++j) {
    const uint32_t r = 8u * (P2 * (tid & 1u) + j);
    const f32x4 lo = *reinterpret_cast<const f32x4 *>(u + r), hi = *reinterpret_cast<const f32x4 *>(u + r + 4u);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float even = t < 2 ? lo[2 * t] : hi[2 * t - 4], odd = t < 2 ? lo[2 * t + 1] : hi[2 * t - 3];
      if (halves && r == 0u) {
        even += half_u[2 * t];
        odd += half_u[2 * t + 1];
      }
      v = __builtin_fmaf(bf16_lo(b[j][t]), even, v);
      v = __builtin_fmaf(bf16_hi(b[j][t]), odd, v);
    }
  }
  v += __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0xB1, 0xF, 0xF, true));  // the neighbour's
  if (write) ((g_u16 *)s.y)[i * s.y_stride + n] = to_bf16_bits(__builtin_fmaf(scale, v, base));
}

// ---- host ----------------------------------------------------------------------------------

bool planned(const LoraArgs &a) { return a.m > kBallotRows; }
uint32_t plans(const LoraArgs &a) { return (a.m + kLoraPlanRows - 1u) / kLoraPlanRows; }

uint32_t max_rank(const LoraArgs &a) {
  uint32_t r = 0;
  for (uint32_t i = 0; i < a.count; ++i) r = a.s[i].R > r ? a.s[i].R : r;
  return r;
}

// One launch for few rows of small A's, by what its workgroups read of A in all and each after the other.  us with one launch /
// with two (a graph of calls; outside one the second launch costs the host 2.5 more):
// 4096x4096, rank 16 (A 128 KiB): 1 row 3.9 / 6.5, 16 rows (17 MB) 5.5 / 6.8, 32 (34 MB) 7.0 / 7.0, 48 10.2 / 8.4;
// q, k and v of rank 32 (256 KiB): 8 rows (25 MB) 7.4 / 7.8, 32 (100 MB) 16.5 / 11.8;
// gate and up of 14336x4096, rank 16: 4 rows (29 MB) 5.1 / 6.8, 8 (57 MB) 8.7 / 7.6;
// 4096x14336, rank 16 (448 KiB): 1 row (3.7 MB) 7.1 / 8.0, 4 (15 MB) 9.4 / 8.5; rank 64 (1.8 MB): 1 row 24.8 / 9.7.
bool solo(const LoraArgs &a) {
  if (planned(a)) return false;  // rows enough to share an adapter's weights, and more than a grid's second axis may hold
  uint64_t all = 0;
  for (uint32_t i = 0; i < a.count; ++i) all += (uint64_t)((a.s[i].N + kSoloColumns - 1u) / kSoloColumns) * a.s[i].R;
  all *= 2u * (uint64_t)a.K * a.m;
  const uint64_t each = 2u * (uint64_t)a.K * max_rank(a);
  return a.K <= kSoloK && max_rank(a) <= 64u && all <= (each <= (256u << 10) ? 40000000u : each <= (512u << 10) ? 8000000u : 0u);
}

uint32_t k_steps(const LoraArgs &a) { return (a.K + kStepK - 1u) / kStepK; }

// Workgroups of each 64 plans.
uint32_t blocks_of(const LoraArgs &a, uint32_t blocks) {
  const uint32_t n = blocks / ((plans(a) + 63u) / 64u);
  return n < 64u ? 64u : n & ~7u;
}

// How K is cut: two steps a wave.  With a plan that is the most; the groups may be too many for it.
void cut_k(LoraArgs &a) {
  a.part_steps = 8u;
  a.parts = (k_steps(a) + 7u) / 8u;
  if (planned(a)) {
    const uint32_t least = ((a.m < 64u * kLoraPlanRows ? a.m : 64u * kLoraPlanRows) + kMany - 1u) / kMany;  // groups of the first plans
    const uint32_t most = kShrinkBlocks / least;
    a.parts = most < 1u ? 1u : a.parts < most ? a.parts : most;
  }
}

// The LDS of a kernel that has dynamic LDS alone.
template <class Kern>
hipError_t allow(LdsAllowance &allowance, Kern kern, uint32_t bytes) {
  return needs_lds_allowance(bytes, 0) ? allow_lds(allowance, kern, (int)bytes) : hipSuccess;
}

template <int P2>
hipError_t launch_solo(const LoraArgs &a, hipStream_t stream) {
  uint32_t tiles = 0;
  for (uint32_t i = 0; i < a.count; ++i) tiles += (a.s[i].N + kSoloColumns - 1u) / kSoloColumns;
  k_solo<P2><<<dim3(tiles, a.m), 1024, (a.K * 2u + 15u) & ~15u, stream>>>(a);
  return hipGetLastError();
}

template <int RT>
hipError_t launch_shrink(const LoraArgs &a, hipStream_t stream) {
  if (!planned(a)) {
    constexpr uint32_t lds = ShrinkFew<RT>::kLds;
    static LdsAllowance allowance;
    const hipError_t e = allow(allowance, k_shrink_rows<RT>, lds);
    if (e != hipSuccess) return e;
    k_shrink_rows<RT><<<dim3(a.parts, a.m, a.count), 256, lds, stream>>>(a);
  } else {
    constexpr uint32_t lds = ShrinkFew<RT>::kLds > ShrinkMany<RT>::kLds ? ShrinkFew<RT>::kLds : ShrinkMany<RT>::kLds;
    static LdsAllowance allowance;
    const hipError_t e = allow(allowance, k_shrink_items<RT>, lds);
    if (e != hipSuccess) return e;
    k_shrink_items<RT><<<dim3(blocks_of(a, kShrinkBlocks), (plans(a) + 63u) / 64u, a.count), 256, lds, stream>>>(a);
  }
  return hipGetLastError();
}

template <int P, int NCH>
hipError_t launch_expand(const LoraArgs &a, hipStream_t stream) {
  typedef ExpandFew<P, NCH> Few;
  uint32_t tiles = 0;
  if (!planned(a)) {
    static LdsAllowance allowance;
    const hipError_t e = allow(allowance, k_expand_rows<P, NCH>, Few::kLds);
    if (e != hipSuccess) return e;
    for (uint32_t i = 0; i < a.count; ++i) tiles += (a.s[i].N + Few::kColumns - 1u) / Few::kColumns;
    k_expand_rows<P, NCH><<<dim3(tiles, a.m), 256, Few::kLds, stream>>>(a);
    return hipGetLastError();
  }
  for (uint32_t i = 0; i < a.count; ++i) tiles += (a.s[i].N + kBlockN - 1u) / kBlockN;
  k_expand_items<P, NCH><<<dim3(blocks_of(a, kExpandBlocks), (plans(a) + 63u) / 64u), 256, ExpandMany<P, NCH>::kLds, stream>>>(a, tiles);
  return hipGetLastError();
}

}  // namespace

uint64_t lora_workspace(const LoraArgs &given, uint64_t *offsets) {
  LoraArgs a = given;
  if (solo(a)) return 0;
  cut_k(a);
  uint64_t bytes = planned(a) ? plans(a) * kLoraPlanBytes : 0u;
  for (uint32_t i = 0; i < a.count; ++i) {
    offsets[i] = bytes;
    bytes += ((uint64_t)a.parts * a.m * a.s[i].R * 4u + 255u) & ~255ull;
  }
  return bytes;
}

hipError_t launch_lora(LoraArgs a, void *ws, hipStream_t stream) {
  const uint32_t R = max_rank(a);
  if (solo(a)) return R <= 16u ? launch_solo<1>(a, stream) : R <= 32u ? launch_solo<2>(a, stream) : launch_solo<4>(a, stream);
  cut_k(a);
  uint64_t offsets[INT8W_MAX_MULTI];
  lora_workspace(a, offsets);
  for (uint32_t i = 0; i < a.count; ++i) a.s[i].u = reinterpret_cast<float *>((uint8_t *)ws + offsets[i]);
  a.plans = ws;
  if (planned(a)) {
    uint32_t bits = 1;
    while (a.num + 1u >> bits) ++bits;  // ids up to num + 1
    k_plan<<<plans(a), kLoraPlanRows, 0, stream>>>(a.ids, a.m, a.num, bits, reinterpret_cast<LoraPlan *>(ws));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const hipError_t e = R <= 16u ? launch_shrink<1>(a, stream) : R <= 32u ? launch_shrink<2>(a, stream) : launch_shrink<4>(a, stream);
  if (e != hipSuccess) return e;
  if (R <= 16u) return launch_expand<2, 1>(a, stream);
  if (R <= 32u) return launch_expand<4, 1>(a, stream);
  if (R <= 64u) return launch_expand<8, 1>(a, stream);
  if (R <= 128u) return launch_expand<8, 2>(a, stream);
  return launch_expand<8, 4>(a, stream);
}

}  // namespace int8w
