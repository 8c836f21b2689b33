// C ABI of the operators around the expert FFN (declared in include/bitmoe.h): argument checks
// and dispatch.  No allocation, no workspace, no host synchronisation.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../../include/bitmoe.h"
#include "block_kernels.h"

using namespace bitmoe;

namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxTopK = 64;
constexpr int kMaxGroups = 64;
constexpr int kMaxLinear = 1 << 20;    // N and K
constexpr int kMaxLinearRows = 1 << 26;  // T: a launch has fewer than 2^32 threads

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
inline bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}
inline bool float_dtype(int32_t d) { return d == MOE_DT_F32 || d == MOE_DT_BF16; }

}  // namespace

extern "C" {

moe_status moe_add_rmsnorm(const void* x, int32_t x_dtype, const void* residual, int32_t residual_dtype,
                           const uint16_t* weight, float eps, int32_t T, int32_t H, void* residual_out, uint16_t* y,
                           uint8_t* q, uint8_t* q_scales, void* stream) {
  if (T < 0 || H < 1 || !float_dtype(x_dtype) || !float_dtype(residual_dtype)) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 1.17549435e-38f) return MOE_ERR_INVALID_ARG;
  if (q && H % 32) return MOE_ERR_INVALID_ARG;
  if (H % 8 || H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !weight || (!y && !q) || (q && !q_scales) || (q_scales && !q) || (residual_out && !residual))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(weight, 16) ||
      !aligned(y, 16) || !aligned(q, 8))
    return MOE_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.residual_out = residual_out;
  a.weight = weight;
  a.y = y;
  a.q = q;
  a.q_scales = q_scales;
  a.eps = eps;
  a.T = T;
  a.H = H;
  return from_hip(launch_add_rmsnorm(a, x_dtype == MOE_DT_F32, residual_dtype == MOE_DT_F32, as_stream(stream)));
}

moe_status moe_route_scored(const float* logits, const float* bias, int32_t T, int32_t E, int32_t k, int32_t score,
                            int32_t n_group, int32_t topk_group, int32_t group_top, int32_t renormalize, float scale,
                            int32_t* topk_ids, float* topk_w, void* stream) {
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E || k > kMaxTopK) return MOE_ERR_INVALID_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (n_group < 1 || E % n_group || topk_group < 1 || topk_group > n_group) return MOE_ERR_INVALID_ARG;
  if (group_top != 1 && group_top != 2) return MOE_ERR_INVALID_ARG;
  if ((int64_t)topk_group * (E / n_group) < k) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (n_group > kMaxGroups) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return MOE_ERR_INVALID_ARG;
  RouteScoredArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.sigmoid = score == MOE_SCORE_SIGMOID;
  a.n_group = n_group;
  a.topk_group = topk_group;
  a.group_top = group_top;
  a.renormalize = renormalize != 0;
  a.scale = scale;
  a.ids = topk_ids;
  a.gates = topk_w;
  return from_hip(launch_route_scored(a, as_stream(stream)));
}

moe_status moe_linear(const void* x, const uint8_t* x_scales, const void* w, const uint8_t* w_scales, int32_t dtype,
                      int32_t T, int32_t N, int32_t K, const float* bias, int32_t act, const void* residual,
                      int32_t residual_dtype, void* out, int32_t out_dtype, void* stream) {
  if (T < 0 || N < 1 || K < 1 || (dtype != MOE_DT_BF16 && dtype != MOE_DT_MXFP8)) return MOE_ERR_INVALID_ARG;
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU || !float_dtype(residual_dtype) || !float_dtype(out_dtype))
    return MOE_ERR_INVALID_ARG;
  const bool mx = dtype == MOE_DT_MXFP8, gated = act == MOE_ACT_SWIGLU;
  if ((mx && K % 32) || (gated && N % 2)) return MOE_ERR_INVALID_ARG;
  if (K % 8 || N > kMaxLinear || K > kMaxLinear || T > kMaxLinearRows || (mx && out_dtype == MOE_DT_F32))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w || !out || (mx && (!x_scales || !w_scales))) return MOE_ERR_INVALID_ARG;
  const size_t ob = out_dtype == MOE_DT_F32 ? 4 : 2, rb = residual_dtype == MOE_DT_F32 ? 4 : 2;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 4) || !aligned(out, ob) || !aligned(residual, rb))
    return MOE_ERR_INVALID_ARG;
  // a workgroup reads its residual values while others have stored theirs: only the very same values may be shared
  const size_t outs = (size_t)T * (gated ? N / 2 : N);
  if (residual && (residual != out || residual_dtype != out_dtype) && overlap(residual, outs * rb, out, outs * ob))
    return MOE_ERR_INVALID_ARG;
  LinearArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.x_scales = x_scales;
  a.w = static_cast<const uint8_t*>(w);
  a.w_scales = w_scales;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.T = T;
  a.N = N;
  a.K = K;
  a.n_out = gated ? N / 2 : N;
  a.act = act;
  a.res_f32 = residual_dtype == MOE_DT_F32;
  a.out_f32 = out_dtype == MOE_DT_F32;
  a.vec = a.n_out % 4 == 0 && aligned(out, 4 * ob) && aligned(residual, 4 * rb);
  return from_hip(launch_linear(a, mx, as_stream(stream)));
}

}  // extern "C"
