// The epilogue of the dense product, shared by its kernels.
#pragma once

#include "../common.h"
#include "block_kernels.h"

namespace bitmoe {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// D(32x32, f32) += A(32x16, bf16) * B(16x32, bf16): lane l supplies A row l % 32 and B column l % 32
// for k = 8 (l / 32) .. + 7 and receives D[8 (j / 4) + 4 (l / 32) + j % 4][l % 32] in register j.
__device__ __forceinline__ f32x16_t mfma_bf16_32x32x16(u32x4 a, u32x4 b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}
// The same with e4m3 operands of 64 k and e8m0 scales per 32 k.  The matrix cores' sums of these products are not fp32
// sums: one instruction's deviates by up to 3.2e-4 of the rms of such sums (measured on random operands), more than fp32
// rounding and less than the step of the bf16 that the result is rounded to (2^-8 of the value).  It is taken for
// their rate: exact fp32 sums would take the bf16 instructions at half of it.
// Lane l (half h = l / 32) supplies k = 32 c + 16 h
// + [0, 16) in its 16-byte chunks c = 0, 1 and the scale byte of the 32-k block h.
__device__ __forceinline__ f32x16_t mfma_mxfp8_32x32x64(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x16_t c,
                                                        uint32_t sa, uint32_t sb) {
  const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}
// D(16x16, f32) += A(16x128, e4m3) * B(128x16, e4m3) without scales (scale operands of 0 select that instruction): lane l
// supplies row l % 16, k = 64 c + 16 (l / 16) + [0, 16) in its 16-byte chunks c = 0, 1 and receives D[4 (l / 16) + i][l % 16].
// Its sums are as near as those of the instruction above.
__device__ __forceinline__ f32x4 mfma_fp8_16x16x128(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c) {
  const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
// The same with an e8m0 scale for each row of A and column of B, in the lanes that supply them.
__device__ __forceinline__ f32x4 mfma_fp8_16x16x128(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c, uint32_t sa,
                                                    uint32_t sb) {
  const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

// FP8 products multiply the fp32 scales of both sides, which stays in the range of fp32 where each is 0 or in
// [2^-63, 2^63).  A workgroup that meets another scale computes its sums once more with each scale taken apart, s = m
// 2^(e - 127): the powers of two go into the matrix instruction as its e8m0 scales, and only the mantissas (below 2) are
// multiplied outside it.  Within the range both give the same bits.  (Always taken apart: 6 to 20 % slower, 8192 x 4096 x 4096
// 119 -> 128 us, 64 x 4096 x 2048 6.4 -> 7.8 us; with this test 0 to 1 %, 3 % for few rows: 6.4 -> 6.5 us.)
// The test keeps the largest of the scales' exponents from -62 up, as unsigned numbers; 0, infinities and NaN (whose
// products need no range) have the exponent 0 here.
__device__ __forceinline__ uint32_t scale_range(uint32_t most, uint32_t bits) {
  return max(most, (uint32_t)(__builtin_amdgcn_frexp_expf(__uint_as_float(bits)) + 62));
}
__device__ __forceinline__ bool far_scales(uint32_t most) { return most > 125; }
struct SplitScale {
  float m;
  uint32_t e;
};
__device__ __forceinline__ SplitScale split_scale(float s) {
  const uint32_t bits = __float_as_uint(s), e = bits >> 23 & 0xFFu;
  if (e == 0) return {s * 0x1p127f, 0};  // zero and subnormal
  if (e == 255) return {s, 127};
  return {__uint_as_float((bits & 0x807FFFFFu) | 0x3F800000u), e};
}

typedef __attribute__((address_space(3))) void lds_void;

// s_waitcnt vmcnt(N) (and lgkmcnt(0) if LGKM), the other counters not waited on
template <int N, bool LGKM>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (LGKM ? 0 : 0xF00) | ((N >> 4) << 14));
}

// An empty asm that reads a result in ordinary registers: what computes it is not moved past.
__device__ __forceinline__ void hold(const f32x16_t& v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" ::"v"(v));
#endif
}

// The activations in fp32 (a few ulp each: v_exp_f32 and v_rcp_f32 are good to one).  exp overflows
// to inf for very negative arguments, whose reciprocal gives the right limit 0.
__device__ __forceinline__ float silu_f32(float a) { return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }
template <int N>
__device__ __forceinline__ void activate(float (&r)[N], int act) {
  if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = r[i] < 0.0f ? 0.0f : r[i];  // a NaN stays one
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = silu_f32(r[i]);
  } else if (act == kActGelu) {
    // 0.5 a (1 + tanh u) = a / (1 + exp(-2u)), u = sqrt(2/pi) (a + 0.044715 a^3)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = 1.5957691216057308f * r[i] * fmaf(0.044715f * r[i], r[i], 1.0f);
      r[i] = r[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-u));
    }
  }
}

// The epilogue works on four consecutive columns n .. n + 3 of a token row at a time; columns at and
// beyond n_out are left out.

// Four residual values as they are stored: 16 bytes of fp32 or 8 of bf16.  at: t * n_out + n.
struct Four {
  uint32_t w[4];
};
__device__ __forceinline__ Four load_residual4(const LinearArgs& a, int64_t at, int n) {
  Four r{};
  if (a.vec) {
    if (a.res_f32) {
      const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(a.residual) + at);
      r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.residual) + at);
      r.w[0] = q.x, r.w[1] = q.y;
    }
    return r;
  }
  if (a.res_f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.n_out) r.w[i] = reinterpret_cast<const uint32_t*>(a.residual)[at + i];
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.residual) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.n_out) r.w[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
  }
  return r;
}

// The bias of four columns (and of their up rows with a gate), zero without one.
struct FourBias {
  float g[4], u[4];
};
template <int GATED>
__device__ __forceinline__ FourBias load_bias4(const LinearArgs& a, int n) {
  FourBias b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = min(n + i, a.n_out - 1);
    b.g[i] = a.bias ? a.bias[c] : 0.0f;
    b.u[i] = GATED && a.bias ? a.bias[a.n_out + c] : 0.0f;
  }
  return b;
}

// What becomes of the weight rows' halves: kPlain no halves, kSwiglu silu(gate) * up, kGlu act(gate) * up with the
// activation a.glu_act and, where a.pre is given, the pre-activations stored (rounded to bf16) for the backward pass
// (non-temporally in the larger tiles: 8192 x 4096 x 4096 229 -> 225 us, as fast as without them).
constexpr int kPlain = 0, kSwiglu = 1, kGlu = 2;

// Four bf16 values to p, 8-byte aligned.
template <bool STREAM>
__device__ __forceinline__ void store_bf16x4(uint16_t* p, const float (&v)[4]) {
  const u32x2 q = {f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3])};
  if (STREAM)
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(p));
  else
    *reinterpret_cast<u32x2*>(p) = q;
}

// v (and, with a gate, the up columns u): the sums without bias.  Adds the bias, applies the
// activation, adds the residual and stores, rounding once.  STREAM: non-temporal stores, for the larger tiles, whose
// outputs are larger than the caches (with buffers that change from call to call, 8192 x 4096 in bf16, K = 4096:
// 227 -> 220 us, SwiGLU 219 -> 216; in MXFP8, K = 2048: 106 -> 88, with a bf16 residual 112 -> 108; with the same
// buffers each time 2 % at most).
template <int GATED, bool STREAM>
__device__ __forceinline__ void epilogue4(const LinearArgs& a, int64_t at, int n, const float (&v)[4],
                                          const float (&u)[4], const FourBias& bias, const Four& res) {
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = v[i] + bias.g[i];
  if constexpr (GATED == kGlu) {
    if (a.pre) {
      uint16_t* gate = a.pre + 2 * at - n;  // row t of 2 n_out columns, at = t n_out + n; n_out is a multiple of 8
      store_bf16x4<STREAM>(gate, v);
      store_bf16x4<STREAM>(gate + a.n_out, u);
    }
    activate(r, a.glu_act);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] *= u[i];
  } else if constexpr (GATED == kSwiglu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = silu_f32(r[i]) * (u[i] + bias.u[i]);
  } else {
    activate(r, a.act);
  }
  if (a.residual) {
    if (a.res_f32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] += __uint_as_float(res.w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] += __uint_as_float(i % 2 ? res.w[i / 2] & 0xFFFF0000u : res.w[i / 2] << 16);
    }
  }
  if (a.vec) {
    if (a.out_f32) {
      f32x4* o = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at);
      const f32x4 q = {r[0], r[1], r[2], r[3]};
      if (STREAM)
        __builtin_nontemporal_store(q, o);
      else
        *o = q;
    } else {
      u32x2* o = reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at);
      const u32x2 q = {f32x2_to_bf16x2_rne(r[0], r[1]), f32x2_to_bf16x2_rne(r[2], r[3])};
      if (STREAM)
        __builtin_nontemporal_store(q, o);
      else
        *o = q;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.n_out) break;
    if (a.out_f32)
      reinterpret_cast<float*>(a.out)[at + i] = r[i];
    else
      reinterpret_cast<uint16_t*>(a.out)[at + i] = (uint16_t)f32_to_bf16_rne(r[i]);
  }
}

}  // namespace bitmoe
