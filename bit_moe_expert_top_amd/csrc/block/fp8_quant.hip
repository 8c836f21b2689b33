// Quantisation to FP8 (e4m3fn) with an fp32 scale for each block of 128 values of a row, or of 128 x 128 values:
//   s = max|x| / 448,  q = x / s rounded to e4m3 (nearest even)
// Both divisions are IEEE fp32.  x / s of a block costs three instructions a value: with r = 1 / s rounded,
// q0 = x r is within an ulp, and q0 - (q0 s - x) r rounds to the correct quotient (Markstein), where nothing
// under- or overflows (in this order -0 stays -0); blocks outside [2^-60, 2^100] are divided plainly.  A block whose scale is 0 has elements 0.
// Memory bound: 32768 x 4096 bf16 71 us (5.7 TB/s), 4096 x 4096 fp32 by 128 x 128 15 us (5.6 TB/s); 64 x 4096 bf16 2.8 us, a
// launch.
#include "../common.h"
#include "block_kernels.h"
#include "row8.h"

namespace bitmoe {

namespace {

constexpr int kThreads = 256;

// The largest magnitude's bits: NaN counts as larger than infinity.
__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

struct Scale {
  float s, r;  // s = top / 448 and 1 / s
  bool plain;  // outside the range of the short division
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {
  Scale c;
  const float m = __uint_as_float(top);
  c.s = m / 448.0f;
  c.plain = !(m >= 0x1p-60f && m <= 0x1p100f);
  c.r = c.plain ? 0.0f : 1.0f / c.s;
  return c;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  auto in = [](float v) { return __builtin_amdgcn_fmed3f(v, 448.0f, -448.0f); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(in(a), in(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(in(c), in(d), lo, true);
}

__device__ __forceinline__ uint2 quantize8(const float (&v)[8], const Scale& c) {
  float q[8];
  if (!c.plain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q0 = v[i] * c.r;
      q[i] = fmaf(-fmaf(q0, c.s, -v[i]), c.r, q0);
    }
    return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
  }
  uint32_t w[2] = {0, 0};
  if (c.s == 0.0f) return make_uint2(0, 0);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = h ? v[4 + i] : v[i];
      const float d = x / c.s;
      const uint32_t b = d == d ? pack4(d, 0.f, 0.f, 0.f) & 0xFFu : 0x7Fu;
      w[h] |= b << (8 * i);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Sixteen values of a row (eight lanes to a block): 32 or 64 bytes in flight a thread and one 16-byte store of elements
// (with eight values a thread bf16 ran at 4.2 TB/s).
typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));  // elements are 8-byte aligned
__device__ __forceinline__ void store16(uint8_t* q, const float (&v)[2][8], const Scale& c) {
  const uint2 a = quantize8(v[0], c), b = quantize8(v[1], c);
  *reinterpret_cast<u32x4_a8*>(q) = u32x4_a8{a.x, a.y, b.x, b.y};
}
constexpr int kLanes = 8;

// A scale per row and 128 values.  blocks < 2^31, and the grid's step is at most 2^25, so 32 bits hold every b (a 64-bit
// division by kb would be 100 instructions).
template <typename XT>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const XT* x, uint32_t blocks, int K, int kb, uint8_t* q,
                                                                 float* scales) {
  for (uint32_t b = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; b < blocks;
       b += gridDim.x * (kThreads / kLanes)) {
    const uint32_t row = b / (uint32_t)kb;
    const int c = 128 * (int)(b - row * (uint32_t)kb) + 16 * (threadIdx.x % kLanes);
    const int64_t at = (int64_t)row * K + c;
    float v[2][8] = {};
    if (c < K) load8(x + at, v[0]), load8(x + at + 8, v[1]);
    uint32_t m = max(top8(v[0]), top8(v[1]));
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    const Scale sc = scale_of(m);
    if (c < K) store16(q + at, v, sc);
    if (threadIdx.x % kLanes == 0) scales[b] = sc.s;
  }
}

// A scale per 128 x 128 values: a workgroup to a block (fewer than 2^24), a thread holds 16 values of 4 rows.
template <typename XT>
__global__ __launch_bounds__(kThreads) void quantize_blocks_kernel(const XT* x, int64_t rows, int K, int kb, uint8_t* q,
                                                                   float* scales) {
  constexpr int kPass = kThreads / kLanes, kPasses = 128 / kPass;  // rows of a pass
  __shared__ uint32_t part[kThreads / kWave];
  const uint32_t b = blockIdx.x, rb = b / (uint32_t)kb;
  const int64_t r0 = 128 * (int64_t)rb + threadIdx.x / kLanes;
  const int c = 128 * (int)(b - rb * (uint32_t)kb) + 16 * (threadIdx.x % kLanes);
  float v[kPasses][2][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][0][k] = v[i][1][k] = 0.f;
    const XT* p = x + (r0 + kPass * i) * K + c;
    if (c < K && r0 + kPass * i < rows) load8(p, v[i][0]), load8(p + 8, v[i][1]);
    m = max(m, max(top8(v[i][0]), top8(v[i][1])));
  }
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
  if (wave_lane() == 0) part[threadIdx.x / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / kWave; ++i) m = max(m, part[i]);
  const Scale sc = scale_of(m);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (c < K && r0 + kPass * i < rows) store16(q + (r0 + kPass * i) * K + c, v[i], sc);
  if (threadIdx.x == 0) scales[b] = sc.s;
}

template <typename XT>
hipError_t go(const XT* x, int64_t rows, int K, int by, uint8_t* q, float* scales, hipStream_t s) {
  const int kb = (K + 127) / 128;
  if (by == 1) {
    // a workgroup takes more than one turn from 2^25 blocks on (a launch has fewer than 2^32 threads; with 2^16 workgroups
    // at most 131072 x 4096 bf16 takes 286 instead of 277 us)
    const int64_t blocks = rows * kb, want = (blocks + kThreads / kLanes - 1) / (kThreads / kLanes);
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : 1 << 20);
    quantize_rows_kernel<XT><<<grid, kThreads, 0, s>>>(x, (uint32_t)blocks, K, kb, q, scales);
  } else {
    quantize_blocks_kernel<XT><<<(unsigned)((rows + 127) / 128 * kb), kThreads, 0, s>>>(x, rows, K, kb, q, scales);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize(const void* x, bool x_f32, int64_t rows, int K, int by, uint8_t* q, float* scales,
                               hipStream_t s) {
  return x_f32 ? go(static_cast<const float*>(x), rows, K, by, q, scales, s)
               : go(static_cast<const uint16_t*>(x), rows, K, by, q, scales, s);
}

}  // namespace bitmoe
