// The gradient of the gated projection's pre-activations: h = act(g) u gives dg = dh u act'(g), du = dh act(g).
// Memory bound, each value read and written once: 8192 x 2048 (168 MB) 27 us.
#include <algorithm>

#include "../common.h"
#include "block_kernels.h"
#include "row8.h"

namespace bitmoe {

namespace {

constexpr int kThreads = 256;

// act(g) and act'(g) in fp32
template <int ACT>
__device__ __forceinline__ void act_slope(float g, float& value, float& slope) {
  if constexpr (ACT == kActNone) {
    value = g, slope = 1.0f;
  } else if constexpr (ACT == kActRelu) {
    value = g < 0.0f ? 0.0f : g, slope = g > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
    value = g * p, slope = fmaf(value, 1.0f - p, p);
  } else {
    // g p with p = 1 / (1 + exp(-z)), z = 2 sqrt(2/pi) (g + 0.044715 g^3)
    const float z = 1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f);
    const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-z)), t = p * (1.0f - p);
    const float dz = 1.5957691216057308f * fmaf(0.134145f * g, g, 1.0f);
    value = g * p, slope = t > 0.0f ? fmaf(g * t, dz, p) : p;  // t = 0 where dz may be infinite
  }
}

// The matrix cores take the gradients of the pre-activations as bf16: one rounding, of the size of the outputs' own.
template <int ACT>
__global__ __launch_bounds__(kThreads) void glu_grad_kernel(const uint16_t* dh, const uint16_t* a, int T, int I,
                                                            uint16_t* da) {
  const int per = I / 8;
  const int64_t n = (int64_t)T * per;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / per, at = t * 2 * I + 8 * (i - t * per);
    float d[8], g[8], u[8], dg[8], du[8];
    load8(dh + 8 * i, d);
    load8(a + at, g);
    load8(a + at + I, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float value, slope;
      act_slope<ACT>(g[j], value, slope);
      dg[j] = d[j] * u[j] * slope;
      du[j] = d[j] * value;
    }
    store8(da + at, dg);
    store8(da + at + I, du);
  }
}

}  // namespace

hipError_t launch_glu_grad(const uint16_t* dh, const uint16_t* a, int T, int I, int act, uint16_t* da, hipStream_t s) {
  const int64_t want = ((int64_t)T * (I / 8) + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)std::min<int64_t>(want, 1 << 20);
  if (act == kActNone) glu_grad_kernel<kActNone><<<grid, kThreads, 0, s>>>(dh, a, T, I, da);
  if (act == kActRelu) glu_grad_kernel<kActRelu><<<grid, kThreads, 0, s>>>(dh, a, T, I, da);
  if (act == kActGelu) glu_grad_kernel<kActGelu><<<grid, kThreads, 0, s>>>(dh, a, T, I, da);
  if (act == kActSilu) glu_grad_kernel<kActSilu><<<grid, kThreads, 0, s>>>(dh, a, T, I, da);
  return hipGetLastError();
}

}  // namespace bitmoe
