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
enum LinearAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };
struct LinearArgs {
  const uint8_t* x;         // bf16 or e4m3fn [T][K]
  const uint8_t* x_scales;  // e8m0 [T][K/32] (MXFP8)
  const uint8_t* w;         // [N][K]
  const uint8_t* w_scales;
  const float* bias;     // [N] or nullptr
  const void* residual;  // [T][n_out] or nullptr
  void* out;             // [T][n_out]
  int T, N, K;
  int n_out;  // N, or N/2 with SwiGLU
  int act;
  int res_f32, out_f32;
  int vec;  // rows of out and residual allow 4-column vector accesses
};
// few token rows (linear_rows.hip): 16 tt of them to a workgroup, tt = 1, 2 or 4
hipError_t launch_linear_rows(const LinearArgs& a, bool mxfp8, int tt, hipStream_t s);
hipError_t launch_linear(const LinearArgs& a, bool mxfp8, hipStream_t s);

}  // namespace bitmoe
