// C ABI of the operators around the expert FFN (declared in include/bitmoe.h): argument checks
// and dispatch.  No allocation and no host synchronisation; a workspace only in the gradient calls, from the caller.
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
// a shares bytes with any of the others; null and empty arrays have none
struct Span {
  const void* p;
  size_t bytes;
};
template <typename... S>
inline bool shares(Span a, S... others) {
  return a.p && a.bytes && ((others.p && others.bytes && overlap(a.p, a.bytes, others.p, others.bytes)) || ...);
}
inline bool float_dtype(int32_t d) { return d == MOE_DT_F32 || d == MOE_DT_BF16; }

// The sizes of a gradient call: rows of 16-byte chunks in all three matrices.
inline bool grad_sizes(int32_t T, int32_t N, int32_t K) {
  return T >= 0 && N > 0 && K > 0 && N % 8 == 0 && K % 8 == 0 && N <= kMaxLinear && K <= kMaxLinear && T <= kMaxLinearRows;
}
inline size_t da_bytes(int64_t T, int64_t I) { return ((size_t)T * I * 4 + 255) / 256 * 256; }

// Checks and fills what both gradient calls share.  dy: [T][N] (the gated call's lies in its workspace); read: the
// other inputs.  No output and no byte of the workspace may be an input's or another output's.
template <typename... S>
moe_status grad_args(GradArgs& g, const uint16_t* dy, const uint16_t* x, const uint16_t* w, int32_t T, int32_t N,
                     int32_t K, void* dx, int32_t dx_dtype, void* dw, int32_t dw_dtype, int32_t accumulate, Span ws,
                     S... read) {
  if (!float_dtype(dx_dtype) || !float_dtype(dw_dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dy || (!dx && !dw) || (dx && !w) || (dw && !x))) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(dx, 16) || !aligned(dw, 16))
    return MOE_ERR_INVALID_ARG;
  const Span sx{dw ? x : nullptr, (size_t)T * K * 2}, sw{dx ? w : nullptr, (size_t)N * K * 2};
  const Span sdx{dx, (size_t)T * K * (dx_dtype == MOE_DT_F32 ? 4 : 2)};
  const Span sdw{dw, (size_t)N * K * (dw_dtype == MOE_DT_F32 ? 4 : 2)};
  if (shares(sdx, sx, sw, sdw, read...) || shares(sdw, sx, sw, read...) || shares(ws, sx, sw, sdx, sdw, read...))
    return MOE_ERR_INVALID_ARG;
  g.dy = dy;
  g.x = x;
  g.w = w;
  g.dx = dx;
  g.dw = dw;
  g.dx_f32 = dx_dtype == MOE_DT_F32;
  g.dw_f32 = dw_dtype == MOE_DT_F32;
  g.accumulate = accumulate != 0;
  g.T = T;
  g.N = N;
  g.K = K;
  return MOE_OK;
}

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
  return from_hip(launch_linear(a, mx ? kMxfp8 : kBf16, as_stream(stream)));
}

moe_status moe_fp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t K, int32_t block_rows, uint8_t* q,
                            float* scales, void* stream) {
  if (rows < 0 || K < 1 || !float_dtype(x_dtype) || (block_rows != 1 && block_rows != 128)) return MOE_ERR_INVALID_ARG;
  // blocks of a row and 128, or of 128 x 128: a launch has fewer than 2^32 threads
  if (K % 16 || K > kMaxLinear || rows > kMaxLinearRows || rows * ((K + 127) / 128) >= (int64_t)1 << 31 ||
      (block_rows == 128 && (rows + 127) / 128 * ((K + 127) / 128) >= 1 << 24))
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scales || !aligned(x, 16) || !aligned(q, 8) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
  const Span sx{x, (size_t)rows * K * (x_dtype == MOE_DT_F32 ? 4 : 2)}, sq{q, (size_t)rows * K};
  const Span ss{scales, (size_t)((rows + block_rows - 1) / block_rows) * ((K + 127) / 128) * 4};
  if (shares(sq, sx, ss) || shares(ss, sx)) return MOE_ERR_INVALID_ARG;
  return from_hip(launch_fp8_quantize(x, x_dtype == MOE_DT_F32, rows, K, block_rows, q, scales, as_stream(stream)));
}

moe_status moe_linear_fp8(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales, int32_t T,
                          int32_t N, int32_t K, const float* bias, int32_t act, const void* residual,
                          int32_t residual_dtype, uint16_t* out, void* stream) {
  if (T < 0 || N < 1 || K < 1 || act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU || !float_dtype(residual_dtype))
    return MOE_ERR_INVALID_ARG;
  const bool gated = act == MOE_ACT_SWIGLU;
  if (gated && N % 2) return MOE_ERR_INVALID_ARG;
  if (K % 16 || N > kMaxLinear || K > kMaxLinear || T > kMaxLinearRows) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !x_scales || !w || !w_scales || !out) return MOE_ERR_INVALID_ARG;
  const size_t rb = residual_dtype == MOE_DT_F32 ? 4 : 2;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(bias, 4) ||
      !aligned(out, 2) || !aligned(residual, rb))
    return MOE_ERR_INVALID_ARG;
  const size_t outs = (size_t)T * (gated ? N / 2 : N);
  if (residual && (residual != out || residual_dtype != MOE_DT_BF16) && overlap(residual, outs * rb, out, outs * 2))
    return MOE_ERR_INVALID_ARG;
  const size_t kb = ((size_t)K + 127) / 128, blocks = gated ? 2 * (((size_t)N / 2 + 127) / 128) : ((size_t)N + 127) / 128;
  if (shares(Span{out, outs * 2}, Span{x, (size_t)T * K}, Span{w, (size_t)N * K}, Span{x_scales, T * kb * 4},
             Span{w_scales, blocks * kb * 4}, Span{bias, (size_t)N * 4}))
    return MOE_ERR_INVALID_ARG;
  LinearArgs a{};
  a.x = x;
  a.x_scales = reinterpret_cast<const uint8_t*>(x_scales);
  a.w = w;
  a.w_scales = reinterpret_cast<const uint8_t*>(w_scales);
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.T = T;
  a.N = N;
  a.K = K;
  a.n_out = gated ? N / 2 : N;
  a.act = act;
  a.res_f32 = residual_dtype == MOE_DT_F32;
  a.vec = a.n_out % 4 == 0 && aligned(out, 8) && aligned(residual, 4 * rb);
  return from_hip(launch_linear(a, kFp8, as_stream(stream)));
}

moe_status moe_glu(const uint16_t* x, const uint16_t* w, int32_t T, int32_t I, int32_t K, int32_t act, uint16_t* a,
                   uint16_t* h, void* stream) {
  if (T < 0 || I < 1 || K < 1 || act < MOE_ACT_NONE || act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  if (K % 8 || I % 8 || I > kMaxLinear / 2 || K > kMaxLinear || T > kMaxLinearRows) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w || !h || !aligned(x, 16) || !aligned(w, 16) || !aligned(h, 16) || !aligned(a, 16)) return MOE_ERR_INVALID_ARG;
  const Span sx{x, (size_t)T * K * 2}, sw{w, (size_t)I * K * 4}, sa{a, (size_t)T * I * 4}, sh{h, (size_t)T * I * 2};
  if (shares(sh, sx, sw, sa) || shares(sa, sx, sw)) return MOE_ERR_INVALID_ARG;
  LinearArgs l{};
  l.x = reinterpret_cast<const uint8_t*>(x);
  l.w = reinterpret_cast<const uint8_t*>(w);
  l.out = h;
  l.T = T;
  l.N = 2 * I;
  l.K = K;
  l.n_out = I;
  l.act = kActGlu;
  l.glu_act = act;
  l.pre = a;
  l.vec = 1;
  return from_hip(launch_linear(l, kBf16, as_stream(stream)));
}

size_t moe_linear_backward_ws_bytes(int32_t T, int32_t N, int32_t K) {
  return grad_sizes(T, N, K) ? grad_ws_bytes(T, N, K) : 0;
}

moe_status moe_linear_backward(const uint16_t* dy, const uint16_t* x, const uint16_t* w, int32_t T, int32_t N, int32_t K,
                               void* dx, int32_t dx_dtype, void* dw, int32_t dw_dtype, int32_t accumulate, void* ws,
                               size_t ws_bytes, void* stream) {
  if (T < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (!grad_sizes(T, N, K)) return MOE_ERR_UNSUPPORTED;
  GradArgs g{};
  const Span sdy{dy, (size_t)T * N * 2}, sws{ws, ws_bytes};
  const moe_status bad = grad_args(g, dy, x, w, T, N, K, dx, dx_dtype, dw, dw_dtype, accumulate, sws, sdy);
  if (bad != MOE_OK) return bad;
  const GradPlan plan = plan_grad(g);
  if (ws_bytes < plan.ws_bytes) return MOE_ERR_WORKSPACE;
  if (plan.ws_bytes && (!ws || !aligned(ws, 16))) return MOE_ERR_INVALID_ARG;
  return from_hip(launch_grad(g, plan, ws, as_stream(stream)));
}

moe_status moe_debug_grad_tiles(int32_t T, int32_t N, int32_t K, int32_t which, int32_t* tiles) {
  if (T < 1 || N < 1 || K < 1 || which < 1 || which > 3 || !tiles) return MOE_ERR_INVALID_ARG;
  if (!grad_sizes(T, N, K)) return MOE_ERR_UNSUPPORTED;
  GradArgs g{};
  g.dx = which & 1 ? tiles : nullptr;  // only whether they are wanted counts here
  g.dw = which & 2 ? tiles : nullptr;
  g.T = T;
  g.N = N;
  g.K = K;
  const GradTiles p = plan_grad(g).plan;
  tiles[0] = p.tiles == kTile64 ? 64 : p.tiles == kTile256 ? 256 : 128;
  tiles[1] = p.tiles == kTile64 ? 64 : p.tiles == kTile128 ? 128 : 256;
  tiles[2] = p.dx.splits;
  tiles[3] = p.dw.splits;
  tiles[4] = p.dw_first;
  return MOE_OK;
}

size_t moe_glu_backward_ws_bytes(int32_t T, int32_t I, int32_t K) {
  return I % 8 == 0 && I <= kMaxLinear / 2 && grad_sizes(T, 2 * I, K) ? da_bytes(T, I) + grad_ws_bytes(T, 2 * I, K) : 0;
}

moe_status moe_glu_backward(const uint16_t* dh, const uint16_t* a, const uint16_t* x, const uint16_t* w, int32_t T,
                            int32_t I, int32_t K, int32_t act, void* dx, int32_t dx_dtype, void* dw, int32_t dw_dtype,
                            int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || I < 1 || K < 1 || act < MOE_ACT_NONE || act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  if (I % 8 || I > kMaxLinear / 2 || !grad_sizes(T, 2 * I, K)) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!dh || !a || !aligned(dh, 16) || !aligned(a, 16))) return MOE_ERR_INVALID_ARG;
  GradArgs g{};
  uint16_t* da = static_cast<uint16_t*>(ws);
  const Span sdh{dh, (size_t)T * I * 2}, sa{a, (size_t)T * I * 4}, sws{ws, ws_bytes};
  const moe_status bad = grad_args(g, da, x, w, T, 2 * I, K, dx, dx_dtype, dw, dw_dtype, accumulate, sws, sdh, sa);
  if (bad != MOE_OK) return bad;
  const GradPlan plan = plan_grad(g);
  const size_t need = da_bytes(T, I) + plan.ws_bytes;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (need && (!ws || !aligned(ws, 16))) return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    const hipError_t e = launch_glu_grad(dh, a, T, I, act, da, as_stream(stream));
    if (e != hipSuccess) return from_hip(e);
  }
  return from_hip(launch_grad(g, plan, static_cast<uint8_t*>(ws) + da_bytes(T, I), as_stream(stream)));
}

}  // extern "C"
