// launch.h -- internal host-side launchers of the gfx950 kernels (not part of
// the public C-ABI).  Arguments are already validated by capi.cpp; each
// launcher only sizes the grid and enqueues on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8w.h"
#include "lds_allowance.h"

namespace int8w {

struct WeightView {
  const uint32_t *packed;
  const uint16_t *scales;
  const uint16_t *biases;
  uint32_t N, K, gs;
};

// Number of compute units of the current device (cached per device).
int device_cu_count();

// Lets `kernel` take `bytes` of dynamic LDS on the current device, once on each.
template <class Kern>
hipError_t allow_lds(LdsAllowance &allowance, Kern kernel, int bytes) {
  int device = 0;
  const hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  return allowance.once(device, hipSuccess, [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

hipError_t launch_dequant(const WeightView &w, uint16_t *out, hipStream_t stream);

enum GemvEpilogue { kEpiNone = 0, kEpiSiluGate = 1, kEpiSiluGateResid = 2 };

// y = W a, with a = x (kEpiNone) or silu(gate)*up; plus x_resid for kEpiSiluGateResid.
// gemm with 2 <= m <= 4 rows of X on in_features 1024..4096 (a multiple of
// 1024): the register-resident gemv with several rows (gemv.hip).
bool gemv_rows_supported(uint32_t K, uint32_t m);
hipError_t launch_gemv_rows(const WeightView &w, const uint16_t *X, uint16_t *Y, uint32_t m, hipStream_t stream);
// gemm with m = 2 rows on in_features above 4096 (a multiple of 1024, up to
// 32768) where the small-m kernel is weakest (group size 32, or in_features
// above 16384): the same arithmetic with X's rows in LDS.
bool gemv_rows_lds_supported(uint32_t K, uint32_t gs, uint32_t m);
hipError_t launch_gemv_rows_lds(const WeightView &w, const uint16_t *X, uint16_t *Y, uint32_t m, hipStream_t stream);
hipError_t launch_gemv(const WeightView &w, GemvEpilogue epi, const uint16_t *x_or_gate,
                       const uint16_t *up, const uint16_t *x_resid, uint16_t *y, hipStream_t stream);

// y_i = W_i x for count (1..4) weights with the same K and group size, in one
// launch (each weight's rows streamed by its own share of the waves).
hipError_t launch_gemv_multi(const WeightView *w, uint16_t *const *y, uint32_t count, const uint16_t *x,
                             hipStream_t stream);

// Expert-indexed gemv: w holds E experts of [w.N / E, K] stacked along rows;
// y[p, :] = W_ids[p] x_row(p) for the tokens * topk slots p (x_row(p) is the
// token's row, or the slot's own when x_rows == topk).  ids are read on the
// device; a slot whose id is not below E gets NaN outputs.
hipError_t launch_moe_gemv(const WeightView &w, uint32_t E, const uint16_t *x, uint32_t x_rows, const uint32_t *ids,
                           uint32_t tokens, uint32_t topk, uint16_t *y, hipStream_t stream);

// y = W x for an FP8 E4M3 weight [N, K] (bytes, K a multiple of 16) with a
// per-row f32 scale [N], per-block BF16 or f32 scales [ceil(N/BS),
// ceil(K/BS)] (BS a power of two, 64..1024) or one global scale.
enum Fp8ScaleKind { kFp8PerRow = 0, kFp8BlockBf16 = 1, kFp8BlockF32 = 2, kFp8Single = 3 };
hipError_t launch_fp8_gemv(const uint8_t *codes, const void *scale, Fp8ScaleKind kind, uint32_t block_size,
                           float single, uint32_t N, uint32_t K, const uint16_t *x, uint16_t *y, hipStream_t stream);

// BF16 weight [N, K] -> codes (packed), scales, biases [N, K/gs] (affine min/max).
hipError_t launch_quantize(const uint16_t *w, uint32_t N, uint32_t K, uint32_t gs, uint32_t *packed, uint16_t *scales,
                           uint16_t *biases, hipStream_t stream);

// Y[m, N] = X[m, K] W^T for 2 <= m <= 16 (matrix cores, per-group rescale).
// Only for shapes where smallm_supported(K, gs) (the per-row scale/bias stage
// fits the LDS); others go to launch_gemm_prefill.
bool smallm_supported(uint32_t K, uint32_t gs);
hipError_t launch_gemm_smallm(const WeightView &w, const uint16_t *X, uint16_t *Y, uint32_t m,
                              hipStream_t stream);

// Y[m, N] = X[m, K] W^T for large m (weight tiles dequantized to BF16 in LDS).
// With a workspace (ws != nullptr, at least gemm_prefill_workspace_bytes; no
// initial value) a grid with too few tiles splits K over several work items
// per tile, whose fp32 partials a second launch adds in a fixed order;
// ws == nullptr never splits.
uint64_t gemm_prefill_workspace_bytes(const WeightView &w, uint32_t m);
hipError_t launch_gemm_prefill(const WeightView &w, const uint16_t *X, uint16_t *Y, uint32_t m, void *ws,
                               hipStream_t stream);

// The small-m kernel with two 16-row X tiles per pass (2 <= m <= 32), where
// smallm32_supported(K, gs) (its buffers and scale/bias rows fit the LDS).
bool smallm32_supported(uint32_t N, uint32_t K, uint32_t gs);
hipError_t launch_gemm_smallm32(const WeightView &w, const uint16_t *X, uint16_t *Y, uint32_t m,
                                hipStream_t stream);

// For 16 < m <= 128: the rows per small-m pass (32, or 16 where only the
// one-tile kernel fits) if passes over slices of X are expected to beat the
// tiled kernel (a grid of few tiles, each walking all of K; split over K
// when can_split), else 0.
uint32_t gemm_smallm_slice_rows(const WeightView &w, uint32_t m, bool can_split);

// Calibration streams (not part of the layer path): read `bytes` once, copy
// them, or widen each to 16 bits (2 * bytes written); bytes a multiple of 1024.
hipError_t launch_stream_read(const void *src, uint64_t bytes, uint32_t *sink, hipStream_t stream);
hipError_t launch_stream_copy(const void *src, void *dst, uint64_t bytes, hipStream_t stream);
hipError_t launch_stream_expand(const void *src, void *dst, uint64_t bytes, hipStream_t stream);

// ---- MXFP4 (mxfp4.h): codes [N, K/2], scales [N, K/32], K a multiple of 32
struct MxView {
  const uint8_t *codes;
  const uint8_t *scales;
  uint32_t N, K;
};
// BF16 (or f32) values [rows, K] -> codes, scales; and codes, scales -> BF16 values.
hipError_t launch_mx_quantize(const void *x, bool f32, uint32_t rows, uint32_t K, uint8_t *codes, uint8_t *scales,
                              hipStream_t stream);
hipError_t launch_mx_dequantize(const MxView &w, uint16_t *out, hipStream_t stream);
// Y[m, N] = X[m, K] W^T, X BF16; and X [x.N, K] in MXFP4.
hipError_t launch_mx_gemm(const MxView &w, const uint16_t *x, uint16_t *y, uint32_t m, hipStream_t stream);
hipError_t launch_mx_gemm_mx(const MxView &w, const MxView &x, uint16_t *y, hipStream_t stream);

// ---- mixture-of-experts layer: gate and up [E I, H], down [E H, I] stacked by expert
constexpr uint32_t kMoePassTokens = 64;         // tokens of one pass over the experts
constexpr uint64_t kMoeHeadBytes = 48u << 10;   // routing tables at the head of the workspace
struct MoeArgs {
  uint32_t E;
  const uint16_t *x;    // [tokens, H]
  const void *logits;   // [tokens, E], f32 or BF16; or nullptr:
  const uint32_t *ids;  // [tokens, topk] and
  const float *weights; // [tokens, topk], the given routing
  bool logits_bf16;
  uint32_t tokens, topk;
  bool renorm;
  float scale;
  const uint16_t *resid;  // [tokens, H] or nullptr
  uint16_t *y;            // [tokens, H]
  void *ws;               // head, then for min(tokens, kMoePassTokens) topk slots h [I] BF16, shares [H] f32
};
hipError_t launch_moe_int8(const WeightView &gate, const WeightView &up, const WeightView &down, const MoeArgs &m,
                           hipStream_t stream);
hipError_t launch_moe_mx(const MxView &gate, const MxView &up, const MxView &down, const MoeArgs &m, hipStream_t stream);

// ---- routing by itself
struct RouteArgs {
  const void *logits;  // [tokens, E], f32 or BF16
  const float *bias;   // [E] or nullptr
  uint32_t *ids;       // [tokens, topk]
  float *weights;
  uint32_t tokens, E, topk, groups, topk_groups;
  uint32_t group_size, group_magic, group_lanes;  // set by the launcher, as whole and whole_bias
  bool logits_bf16, sigmoid, top2, renorm, whole, whole_bias;
  float scale;
};
hipError_t launch_route(RouteArgs a, hipStream_t stream);

// ---- low-rank adapters
struct LoraStack {
  const uint16_t *a;      // [num, R, K]
  const uint16_t *b;      // [num, N, R]
  const float *scales;    // [num] or nullptr
  const uint32_t *ranks;  // [num] or nullptr
  const uint16_t *base;   // [m, N] at base_stride, or nullptr
  uint16_t *y;            // [m, N] at y_stride
  uint64_t base_stride, y_stride;
  uint32_t R, N;
  float *u;  // [parts, m, R]: A x, by parts of K
};
struct LoraArgs {
  LoraStack s[INT8W_MAX_MULTI];
  const uint16_t *x;
  uint64_t x_stride;
  const uint32_t *ids;
  uint32_t count, m, K, num;
  uint32_t parts, part_steps;  // of K, set by the launcher
  void *plans;             // the workspace's head: groups of the rows of each kLoraPlanRows
};
constexpr uint32_t kLoraPlanRows = 1024;
constexpr uint64_t kLoraPlanBytes = 273u << 10;
// Bytes of the plans and all the stacks' u, each 256-byte aligned; the offsets of the stacks' u.
uint64_t lora_workspace(const LoraArgs &a, uint64_t *offsets);
hipError_t launch_lora(LoraArgs a, void *ws, hipStream_t stream);

// ---- C-ABI internals shared by capi.cpp and noalloc.hip
// Records the calling thread's last error message and returns code.
int report_error(int code, const char *fmt, ...);
// int8_gemm / int8_gemm_ws: ws == nullptr never splits K.
int gemm_common(const int8w_weight *w, const uint16_t *x, uint16_t *y, uint32_t m, void *ws,
                uint64_t ws_bytes, uint64_t stream);

}  // namespace int8w
