// The dense product for few token rows (one decoded token to a small batch): bound by reading the
// weights, and for the smallest ones by latency.  A workgroup computes 16 TT tokens x 16 weight rows
// (8 gate and 8 up rows with SwiGLU); its NW waves split K in runs of 128 bytes of a row, taken in
// turn.  A wave fetches its runs by direct global -> LDS loads into slots of its own, U runs ahead,
// and no barrier stands before the sums are joined.  LDS is there for the order of the loads alone:
// eight neighbouring lanes read one row's 128 bytes, where the matrix cores' operand layout would
// have each of them read another row (measured at 64 x 384 x 4096: 10.0 us with loads straight into
// that layout).  The 16-byte chunks of a row sit XOR-swizzled by row / 2, so the operand reads have
// no bank conflicts.  The partial sums are joined in LDS in wave order: no atomics, no workspace, the
// same bits on every call.
//
// v_mfma_f32_16x16x32_bf16: lane l supplies row l % 16 and 8 k of the quarter l / 16.
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l supplies row l % 16, k = 64 c + 16 (l / 16) + [0, 16) in
// its 16-byte chunks c = 0, 1 and the e8m0 scale of the 32-k block l / 16.  (Its sums are not fp32 sums: see
// mfma_mxfp8_32x32x64.)
// v_mfma_f32_16x16x128_f8f6f4 without scales for FP8: a run of 128 bytes is one block of K, and its sum is added with both
// fp32 scales (1 x 4096 x 4096 SwiGLU 5.8 us, 64 x 4096 x 4096 9.4 us a launch); scales whose product may leave the range of
// fp32 are told on the way, and the sums made again with them apart (see scale_range).
// Lane l receives output rows (weight rows) 4 (l / 16) + i of token column l % 16.
#include <type_traits>

#include "linear_dev.h"

namespace bitmoe {

namespace {

__device__ __forceinline__ f32x4 mfma_mxfp8_16x16x128(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c, uint32_t sa,
                                                      uint32_t sb) {
  const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

// NW waves, U runs of K in flight per wave, XR token rows in a slot (16 TT, or 8 for at most 8 tokens:
// the matrix cores' other token columns then repeat them, and are not stored)
template <LinearKind KIND, int GATED, int TT, int NW, int U, int XR>
__global__ __launch_bounds__(64 * NW, NW / 4) void linear_rows_kernel(LinearArgs a, int n_tiles) {
  constexpr bool MX = KIND == kMxfp8, FP8 = KIND == kFp8;
  constexpr int kEs = KIND == kBf16 ? 2 : 1, kRun = 128, kRows = 16 + XR, kSlot = kRows * kRun;
  constexpr int LD = kRows / 8;               // direct loads per run
  constexpr int kSc = (kRows + 63) / 64;      // scale dwords per lane and run
  static_assert(U >= 2 && U <= 4 && NW >= TT && TT * 1024 <= kSlot, "shape");
  static_assert(XR == 16 * TT || (XR == 8 && TT == 1), "token rows");
  // one object per slot of the ring: a read of one does not wait for the loads into another
  __shared__ __align__(16) uint8_t s0[NW * kSlot], s1[NW * kSlot], s2[U > 2 ? NW * kSlot : 16], s3[U > 3 ? NW * kSlot : 16];
  const int lane = wave_lane(), r16 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t t0 = (int64_t)(blockIdx.x / n_tiles) * (16 * TT);
  const int n0 = (int)(blockIdx.x % n_tiles) * (GATED ? 8 : 16);
  const int kb_bytes = a.K * kEs, ks = FP8 ? (a.K + 127) / 128 * 4 : a.K / 32, runs = (kb_bytes + kRun - 1) / kRun;
  // resources that end with the tile's last row: weight rows 0-7 and 8-15 (gate and up with SwiGLU)
  // and the tokens; what lies past them, or past K, has an offset past the resource and reads zeros
  const int rows_x = (int)min((int64_t)(16 * TT), a.T - t0);
  const int rows_w0 = min(8, a.n_out - n0), rows_w1 = GATED ? rows_w0 : max(0, min(8, a.n_out - n0 - 8));
  const int64_t w1 = GATED ? (int64_t)a.n_out + n0 : (int64_t)n0 + (rows_w1 > 0 ? 8 : 0);
  const buf_rsrc rw0 = make_rsrc(a.w + (int64_t)n0 * kb_bytes, (uint32_t)rows_w0 * kb_bytes);
  const buf_rsrc rw1 = make_rsrc(a.w + w1 * kb_bytes, (uint32_t)rows_w1 * kb_bytes);
  const buf_rsrc rx = make_rsrc(a.x + t0 * kb_bytes, (uint32_t)rows_x * kb_bytes);
  // load i fills slot rows 8 i + lane / 8; this lane's chunk of a row for even and odd i
  const int row8 = lane >> 3, ch[2] = {16 * ((lane & 7) ^ (lane >> 4)), 16 * ((lane & 7) ^ (4 + (lane >> 4)))};
  uint32_t off[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const bool in = i == 0 ? row8 < rows_w0 : i == 1 ? row8 < rows_w1 : 8 * (i - 2) + row8 < rows_x;
    off[i] = in ? (uint32_t)(i < 2 ? row8 : 8 * (i - 2) + row8) * kb_bytes + (uint32_t)ch[i & 1] : kOffNone;
  }
  // MXFP8: lane l fetches the four scales of a run of slot rows l and 64 + l; FP8: their one fp32 scale (ks: bytes of a
  // row of scales, four for a run in both).  The 8 weight rows of a half lie in one block row.
  const int up_blocks = (a.n_out + 127) / 128;  // block rows of the gate
  const uint8_t* srow[kSc];
  if (MX || FP8) {
#pragma unroll
    for (int c = 0; c < kSc; ++c) {
      const int r = lane + 64 * c;
      srow[c] = nullptr;
      if (r < 8) {
        if (r < rows_w0) srow[c] = a.w_scales + (FP8 ? (int64_t)(n0 / 128) : (int64_t)n0 + r) * ks;
      } else if (r < 16) {
        if (r - 8 < rows_w1)
          srow[c] = a.w_scales + (FP8 ? (int64_t)((GATED ? up_blocks : 0) + n0 / 128) : w1 + r - 8) * ks;
      } else if (r - 16 < rows_x) {
        srow[c] = a.x_scales + (t0 + r - 16) * ks;
      }
    }
  }
  uint32_t sreg[U][kSc];
  auto slot = [&](int u) -> uint8_t* { return (u == 0 ? s0 : u == 1 ? s1 : u == 2 ? s2 : s3) + w * kSlot; };
  auto load = [&](int u, int run) {
    const int b = run * kRun;
    if (MX || FP8) {
#pragma unroll
      for (int c = 0; c < kSc; ++c) {
        uint32_t v = 0;
        if (srow[c]) {
          const int left = ks - 4 * run;
          if (FP8 || left >= 4) {
            __builtin_memcpy(&v, srow[c] + 4 * run, 4);
          } else {
            for (int i = 0; i < left; ++i) v |= (uint32_t)srow[c][4 * run + i] << (8 * i);
          }
        }
        sreg[u][c] = v;
      }
    }
    const bool whole = b + kRun <= kb_bytes;
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const uint32_t o = whole || b + ch[i & 1] < kb_bytes ? off[i] : kOffNone;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(i == 0 ? rw0 : i == 1 ? rw1 : rx, (lds_void*)(slot(u) + 1024 * i), 16,
                                               (int)o, b, 0, 0);
    }
  };
  f32x4 acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a lane's two chunks of slot row r
  auto chunks = [&](int r, uint32_t(&p)[2]) {
    p[0] = 128u * r + 16u * (uint32_t)(g ^ ((r >> 1) & 7));
    p[1] = 128u * r + 16u * (uint32_t)((4 + g) ^ ((r >> 1) & 7));
  };
  uint32_t wpos[2], xpos[2];
  chunks(r16, wpos);
  chunks(r16 % XR, xpos);
  uint32_t range = 0;  // FP8: of the scales met
  auto compute = [&](int u, auto apart) {
    const uint8_t* st = slot(u);
    u32x4 wv[2], xv[TT][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      wv[c] = *reinterpret_cast<const u32x4*>(st + wpos[c]);
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[t][c] = *reinterpret_cast<const u32x4*>(st + 2048 * (t + 1) + xpos[c]);
    }
    if constexpr (MX) {
      // byte g of slot row 16 i + r16
      auto scale = [&](int i) {
        return ((uint32_t)__builtin_amdgcn_ds_bpermute(4 * (16 * (i % 4) + r16), (int)sreg[u][i / 4]) >> (8 * g)) & 0xFFu;
      };
      const uint32_t sw = scale(0);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t sx = scale(t + 1);
        acc[t] = mfma_mxfp8_16x16x128(wv[0], wv[1], xv[t][0], xv[t][1], acc[t], sw, sx);
      }
    } else if constexpr (FP8) {
      // a run is one block of K: its sum by itself, then times both scales into the fp32 sum
      auto scale = [&](int row, int c) {
        return __int_as_float(__builtin_amdgcn_ds_bpermute(4 * row, (int)sreg[u][c]));
      };
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      const float sw = scale(4 * g, 0);
      if constexpr (!decltype(apart)::value) {
#pragma unroll
        for (int c = 0; c < kSc; ++c) range = scale_range(range, sreg[u][c]);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const float sx = scale(16 * ((t + 1) % 4) + r16, (t + 1) / 4);
        float sc;
        f32x4 p;
        if constexpr (decltype(apart)::value) {
          // the mantissa of the weight rows whose sums a lane receives, the power of two of the one that it supplies
          const SplitScale cw = split_scale(sw), cx = split_scale(sx);
          sc = cw.m * cx.m;
          p = mfma_fp8_16x16x128(wv[0], wv[1], xv[t][0], xv[t][1], zero, split_scale(scale(r16, 0)).e, cx.e);
        } else {
          sc = sw * sx;
          p = mfma_fp8_16x16x128(wv[0], wv[1], xv[t][0], xv[t][1], zero);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(sc, p[j], acc[t][j]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        acc[t] = mfma_16x16x32_bf16(wv[0], xv[t][0], acc[t]);
        acc[t] = mfma_16x16x32_bf16(wv[1], xv[t][1], acc[t]);
      }
    }
  };
  // runs w, w + NW, ...: U of them in flight
  auto all_runs = [&](auto apart) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (w + NW * u < runs) load(u, w + NW * u);
    for (int run = w; run < runs; run += NW * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = run + NW * u;
        if (r >= runs) break;
        if (r + NW * (U - 1) < runs)
          wait_vm<(U - 1) * LD, false>();  // the U - 1 later runs may be in flight
        else
          wait_vm<0, false>();
        asm volatile("" ::: "memory");
        compute(u, apart);
        if (r + NW * U < runs) {
          wait_vm<63, true>();  // this wave's reads of the slot are done
          asm volatile("" ::: "memory");
          load(u, r + NW * U);
        }
      }
    }
  };
  float* part = reinterpret_cast<float*>(s0);  // [NW][TT][64][4]
  auto put_parts = [&] {
    __syncthreads();  // all waves have read their slots
#pragma unroll
    for (int t = 0; t < TT; ++t)
      *reinterpret_cast<float4*>(part + ((w * TT + t) * 64 + lane) * 4) = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
  };
  all_runs(std::false_type{});
  if constexpr (FP8) {
    __shared__ uint32_t far_of[NW];
    const bool wave_far = __ballot(far_scales(range)) != 0;
    if (lane == 0) far_of[w] = wave_far;
    put_parts();
    uint32_t any_far = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) any_far |= far_of[i];
    if (__builtin_amdgcn_readfirstlane(any_far) != 0) {
      // the sums once more with the scales taken apart (see scale_range)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      all_runs(std::true_type{});
      put_parts();
    }
  } else {
    put_parts();
  }
  if (w >= TT) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const float4 p = *reinterpret_cast<const float4*>(part + ((i * TT + w) * 64 + lane) * 4);
    v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
  }
  const int64_t t = t0 + 16 * w + r16;
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = GATED ? __shfl_xor(v[i], 32) : v[i];  // the up row 8 further on
  const int n = n0 + 4 * g;
  if (t >= a.T || n >= a.n_out || (GATED && g >= 2)) return;
  const int64_t at = t * a.n_out + n;
  Four res{};
  if (a.residual) res = load_residual4(a, at, n);
  epilogue4<GATED, false>(a, at, n, v, u, load_bias4<GATED>(a, n), res);
}

template <LinearKind KIND, int GATED, int TT, int NW, int U, int XR = 16 * TT>
hipError_t go_rows(const LinearArgs& a, hipStream_t s) {
  const int per = GATED ? 8 : 16, n_tiles = (a.n_out + per - 1) / per;
  const int64_t m_tiles = ((int64_t)a.T + 16 * TT - 1) / (16 * TT);
  linear_rows_kernel<KIND, GATED, TT, NW, U, XR><<<(unsigned)(m_tiles * n_tiles), 64 * NW, 0, s>>>(a, n_tiles);
  return hipGetLastError();
}

template <LinearKind KIND, int GATED>
hipError_t launch(const LinearArgs& a, int tt, hipStream_t s) {
  // 1 x 4096 x 4096: 7.8 us with 8 token rows in a slot, 8.2 us with 16; 1 x 384 x 4096: 4.1 and 4.6 us
  if (tt == 1 && a.T <= 8) return go_rows<KIND, GATED, 1, 8, 3, 8>(a, s);
  if (tt == 1) return go_rows<KIND, GATED, 1, 8, 4>(a, s);
  if (tt == 2) return go_rows<KIND, GATED, 2, 8, 3>(a, s);
  return go_rows<KIND, GATED, 4, 4, 3>(a, s);
}

}  // namespace

hipError_t launch_linear_rows(const LinearArgs& a, LinearKind kind, int tt, hipStream_t s) {
  const bool gated = a.act == kActSwiglu;
  if (kind == kMxfp8) return gated ? launch<kMxfp8, kSwiglu>(a, tt, s) : launch<kMxfp8, kPlain>(a, tt, s);
  if (kind == kFp8) return gated ? launch<kFp8, kSwiglu>(a, tt, s) : launch<kFp8, kPlain>(a, tt, s);
  if (a.act == kActGlu) return launch<kBf16, kGlu>(a, tt, s);
  return gated ? launch<kBf16, kSwiglu>(a, tt, s) : launch<kBf16, kPlain>(a, tt, s);
}

}  // namespace bitmoe
