// Residual addition and RMS norm of token rows, with bf16 and/or MXFP8 output:
//   s = x + residual, rounded to the residual's type (s = x without a residual)
//   y = s * weight / sqrt(mean(s^2) + eps), rounded once to bf16
//   q = MXFP8 of the bf16 y (blocks of 32: shared exponent floor(log2 amax) - 8, e4m3fn
//       elements rounded to nearest even, saturated), bit-equal to quantising y afterwards.
// The norm is taken of s as it is stored, so the fused call equals an addition followed by a norm
// of the stored stream bit for bit.  The row stays in registers between the sum of squares (fp32)
// and the scaling: each input is read once, each output written once.  Memory bound.
#include "../common.h"
#include "../mx_fmt.h"
#include "block_kernels.h"

namespace bitmoe {

namespace {

constexpr int kNormThreads = 256;

// 8 consecutive elements as fp32
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3]),
                    f32x2_to_bf16x2_rne(v[4], v[5]), f32x2_to_bf16x2_rne(v[6], v[7]));
}
__device__ __forceinline__ void unpack8(uint4 a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// G threads per row (64: a wave, 256: the workgroup), NV vectors of 8 elements per thread.
// XT: float or uint16_t (bf16); RES: 0 no residual, 1 bf16, 2 fp32.
template <typename XT, int RES, int G, int NV>
__global__ __launch_bounds__(kNormThreads) void add_rmsnorm_kernel(NormArgs a) {
  constexpr int kRows = kNormThreads / G;
  __shared__ float part[2][kNormThreads / kWave];
  const int g = threadIdx.x % G, H = a.H;
  int parity = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)gridDim.x * kRows, parity ^= 1) {
    const int64_t t = t0 + threadIdx.x / G;
    const bool row = t < a.T;
    float v[NV][8];
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (g + G * i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      if (row && c < H) {
        load8(reinterpret_cast<const XT*>(a.x) + t * H + c, v[i]);
        if (RES == 1) {
          float r[8];
          load8(reinterpret_cast<const uint16_t*>(a.residual) + t * H + c, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += r[j];
          const uint4 p = pack8(v[i]);
          if (a.residual_out) *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.residual_out) + t * H + c) = p;
          unpack8(p, v[i]);
        } else if (RES == 2) {
          float r[8];
          load8(reinterpret_cast<const float*>(a.residual) + t * H + c, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += r[j];
          if (a.residual_out) {
            float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.residual_out) + t * H + c);
            o[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
            o[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(v[i][j], v[i][j], sq);
    }
    sq = wave_sum(sq);
    if (G > kWave) {
      // two buffers in turn: a wave may write the next row's part while another still reads this one's
      if (wave_lane() == 0) part[parity][threadIdx.x / kWave] = sq;
      __syncthreads();
      sq = 0.f;
#pragma unroll
      for (int w = 0; w < G / kWave; ++w) sq += part[parity][w];
    }
    const float inv = rsqrtf(sq / (float)H + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (g + G * i);
      const bool in = row && c < H;
      float wt[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) wt[j] = 0.f;
      if (in) load8(a.weight + c, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * wt[j];
      const uint4 p = pack8(v[i]);
      if (in && a.y) *reinterpret_cast<uint4*>(a.y + t * H + c) = p;
      if (a.q) {
        // a block of 32 is held by four neighbouring lanes (all of them in the row, as H % 32 == 0)
        const uint32_t w4[4] = {p.x, p.y, p.z, p.w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max(w4[j] & 0x7FFFu, (w4[j] >> 16) & 0x7FFFu));
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        const int shared = mx_shared_exp(m ? floor_log2_bf16(m) : 0, m == 0);
        unpack8(p, v[i]);
        if (in) {
          uint2 o = make_uint2(e4m3x4_scaled(v[i][0], v[i][1], v[i][2], v[i][3], shared),
                               e4m3x4_scaled(v[i][4], v[i][5], v[i][6], v[i][7], shared));
          if (m >= 0x7F80u) {  // infinities and NaN: by their bits, as quantising y does
            o = make_uint2(0, 0);
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
              const uint32_t u = j == 0 ? p.x : j == 1 ? p.y : j == 2 ? p.z : p.w;
              const uint32_t b = bf16_to_e4m3_scaled(u & 0xFFFFu, shared) | bf16_to_e4m3_scaled(u >> 16, shared) << 8;
              if (j < 2)
                o.x |= b << (16 * j);
              else
                o.y |= b << (16 * j - 32);
            }
          }
          *reinterpret_cast<uint2*>(a.q + t * H + c) = o;
          if ((g & 3) == 0) a.q_scales[t * (H / 32) + c / 32] = (uint8_t)(shared + 127);
        }
      }
    }
  }
}

template <typename XT, int RES, int G, int NV>
hipError_t go(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = kNormThreads / G;
  const int64_t want = ((int64_t)a.T + kRows - 1) / kRows;
  const int64_t cap = 1 << 20;
  add_rmsnorm_kernel<XT, RES, G, NV><<<(unsigned)(want < cap ? want : cap), kNormThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename XT, int RES>
hipError_t by_width(const NormArgs& a, hipStream_t s) {
  if (a.H <= 512) return go<XT, RES, 64, 1>(a, s);
  if (a.H <= 1024) return go<XT, RES, 64, 2>(a, s);
  if (a.H <= 2048) return go<XT, RES, 256, 1>(a, s);
  if (a.H <= 4096) return go<XT, RES, 256, 2>(a, s);
  if (a.H <= 8192) return go<XT, RES, 256, 4>(a, s);
  return go<XT, RES, 256, 8>(a, s);
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, bool x_f32, bool res_f32, hipStream_t s) {
  const int res = !a.residual ? 0 : (res_f32 ? 2 : 1);
  if (x_f32) return res == 0 ? by_width<float, 0>(a, s) : res == 1 ? by_width<float, 1>(a, s) : by_width<float, 2>(a, s);
  return res == 0 ? by_width<uint16_t, 0>(a, s) : res == 1 ? by_width<uint16_t, 1>(a, s) : by_width<uint16_t, 2>(a, s);
}

}  // namespace bitmoe
