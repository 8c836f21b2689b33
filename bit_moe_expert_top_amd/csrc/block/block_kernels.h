// Host-side launchers of the operators around the expert FFN (internal to the library; the
// public C ABI is include/bitmoe.h).  Each returns hipSuccess or the launch error.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bitmoe {

// ---- residual + RMS norm (norm.hip)
struct NormArgs {
  const void* x;
  const void* residual;  // nullptr: none
  void* residual_out;    // may be nullptr
  const uint16_t* weight;
  uint16_t* y;        // bf16 output, or nullptr
  uint8_t* q;         // MXFP8 elements, or nullptr
  uint8_t* q_scales;  // with q
  float eps;
  int T, H;
};
constexpr int kNormMaxH = 16384;
hipError_t launch_add_rmsnorm(const NormArgs& a, bool x_f32, bool res_f32, hipStream_t s);

// ---- scored routing (route_scored.hip)
struct RouteScoredArgs {
  const float* logits;
  const float* bias;  // [E] or nullptr
  int T, E, k;
  int sigmoid;     // 1: sigmoid of each logit, 0: softmax over the E logits
  int n_group, topk_group, group_top;
  int renormalize;
  float scale;
  int32_t* ids;
  float* gates;
};
hipError_t launch_route_scored(const RouteScoredArgs& a, hipStream_t s);

// ---- dense product (linear.hip)
enum LinearAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4, kActGlu = 5 };
// the operands' type: bf16, e4m3fn with e8m0 scales per 32 k, e4m3fn with fp32 scales per 128 k
enum LinearKind { kBf16 = 0, kMxfp8 = 1, kFp8 = 2 };
struct LinearArgs {
  const uint8_t* x;         // bf16 or e4m3fn [T][K]
  const uint8_t* x_scales;  // e8m0 [T][K/32], or fp32 [T][K/128 rounded up]
  const uint8_t* w;         // [N][K]
  const uint8_t* w_scales;  // as x_scales; fp32 [row blocks of 128][K/128 rounded up], gate and up rows counted apart
  const float* bias;     // [N] or nullptr
  const void* residual;  // [T][n_out] or nullptr
  void* out;             // [T][n_out]
  int T, N, K;
  int n_out;  // N, or N/2 with a gate
  int act;
  int res_f32, out_f32;
  int vec;  // rows of out and residual allow 4-column vector accesses (those of pre always do)
  int glu_act;    // kActGlu: the gate's activation, and where the pre-activations go ([T][2 n_out], or nullptr)
  uint16_t* pre;
};
// few token rows (linear_rows.hip): 16 tt of them to a workgroup, tt = 1, 2 or 4
hipError_t launch_linear_rows(const LinearArgs& a, LinearKind kind, int tt, hipStream_t s);
// FP8 with block scales (linear_fp8.hip)
hipError_t launch_linear_fp8(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear(const LinearArgs& a, LinearKind kind, hipStream_t s);

// ---- FP8 with a scale per block of 128 (fp8_quant.hip): blocks of by x 128 values, by = 1 or 128
hipError_t launch_fp8_quantize(const void* x, bool x_f32, int64_t rows, int K, int by, uint8_t* q, float* scales,
                               hipStream_t s);

// ---- gradients (grad.hip; glu_grad.hip for the gate)
struct GradArgs {
  const uint16_t* dy;  // bf16 [T][N]
  const uint16_t* x;   // bf16 [T][K]
  const uint16_t* w;   // bf16 [N][K]
  void* dx;            // [T][K] or nullptr
  void* dw;            // [N][K] or nullptr
  int dx_f32, dw_f32;
  int accumulate;      // dw is added to
  int T, N, K;
};
// How a call is laid out: its tiles, and the splits of each sum (of per steps) that ws_bytes hold the parts of.
enum GradVariant { kTile64, kTile128, kTile256x128, kTile256 };
struct GradSplit {
  int splits, per, m_tiles, n_tiles;
};
struct GradTiles {
  GradVariant tiles;
  GradSplit dx, dw;
  bool dw_first;
};
struct GradPlan {
  GradTiles plan;
  size_t ws_bytes;
};
GradPlan plan_grad(const GradArgs& a);
size_t grad_ws_bytes(int64_t T, int64_t N, int64_t K);  // of any call of these sizes: dx, dw or both
hipError_t launch_grad(const GradArgs& a, const GradPlan& plan, void* ws, hipStream_t s);
// da [T][2 I] from dh [T][I] and the pre-activations a [T][2 I]
hipError_t launch_glu_grad(const uint16_t* dh, const uint16_t* a, int T, int I, int act, uint16_t* da, hipStream_t s);

}  // namespace bitmoe
