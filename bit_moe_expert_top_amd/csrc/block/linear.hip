// Dense product out = act(x W^T + bias) + residual on the matrix cores, for bf16 operands
// (v_mfma_f32_32x32x16_bf16) and MXFP8 operands (v_mfma_scale_f32_32x32x64_f8f6f4, the e8m0 block
// scales applied by the matrix cores), fp32 sums.
//
// The weight tile is the MFMA's A operand and the token tile its B operand, so a lane holds four
// groups of four consecutive output columns of one token row.
//
// One wave computes a 32 x 32 tile of the output (two weight tiles with SwiGLU: the gate rows and
// the up rows of the same columns) straight from global memory.
#include "linear_dev.h"

namespace bitmoe {

namespace {

template <bool MX, bool GATED>
__global__ __launch_bounds__(256) void linear_wave_kernel(LinearArgs a, int n_tiles, int64_t tiles) {
  constexpr int kEs = MX ? 1 : 2;          // bytes of an element
  constexpr int kStep = MX ? 64 : 16;      // k of one MFMA
  const int lane = wave_lane(), r32 = lane & 31, hl = lane >> 5;
  const int64_t tile = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (tile >= tiles) return;
  const int64_t t0 = tile / n_tiles * 32;
  const int n0 = (int)(tile % n_tiles) * 32;
  const int64_t xt = min(t0 + r32, (int64_t)a.T - 1);
  const int wn = min(n0 + r32, a.n_out - 1);
  const uint8_t* xr = a.x + xt * a.K * kEs;
  const uint8_t* wr[2] = {a.w + (int64_t)wn * a.K * kEs, a.w + (int64_t)(GATED ? a.n_out + wn : wn) * a.K * kEs};
  f32x16_t acc[2];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[g][i] = 0.f;
  const u32x4 zero = {0, 0, 0, 0};
  auto load = [&](const uint8_t* p, int k) { return k < a.K ? *reinterpret_cast<const u32x4*>(p + (int64_t)k * kEs) : zero; };
  for (int k0 = 0; k0 < a.K; k0 += kStep) {
    if constexpr (MX) {
      const int kb = k0 / 32 + hl, ks = a.K / 32;
      const u32x4 b0 = load(xr, k0 + 16 * hl), b1 = load(xr, k0 + 32 + 16 * hl);
      const uint32_t sb = kb < ks ? a.x_scales[xt * ks + kb] : 0;
#pragma unroll
      for (int g = 0; g < (GATED ? 2 : 1); ++g) {
        const uint32_t sa = kb < ks ? a.w_scales[(int64_t)(g ? a.n_out + wn : wn) * ks + kb] : 0;
        acc[g] = mfma_mxfp8_32x32x64(load(wr[g], k0 + 16 * hl), load(wr[g], k0 + 32 + 16 * hl), b0, b1, acc[g], sa, sb);
      }
    } else {
      const u32x4 b = load(xr, k0 + 8 * hl);
#pragma unroll
      for (int g = 0; g < (GATED ? 2 : 1); ++g) acc[g] = mfma_bf16_32x32x16(load(wr[g], k0 + 8 * hl), b, acc[g]);
    }
  }
  const int64_t t = t0 + r32;
  if (t >= a.T) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = n0 + 8 * q + 4 * hl;
    if (n >= a.n_out) continue;
    float v[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = acc[0][4 * q + i], u[i] = acc[1][4 * q + i];
    epilogue4<GATED>(a, t, n, v, u);
  }
}

template <bool MX, bool GATED>
hipError_t go_wave(const LinearArgs& a, hipStream_t s) {
  const int n_tiles = (a.n_out + 31) / 32;
  const int64_t tiles = ((int64_t)a.T + 31) / 32 * n_tiles;
  linear_wave_kernel<MX, GATED><<<(unsigned)((tiles + 3) / 4), 256, 0, s>>>(a, n_tiles, tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, bool mxfp8, hipStream_t s) {
  const bool gated = a.act == kActSwiglu;
  if (mxfp8) return gated ? go_wave<true, true>(a, s) : go_wave<true, false>(a, s);
  return gated ? go_wave<false, true>(a, s) : go_wave<false, false>(a, s);
}

}  // namespace bitmoe
