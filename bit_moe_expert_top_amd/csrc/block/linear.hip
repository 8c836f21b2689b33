// Dense product out = act(x W^T + bias) + residual on the matrix cores, for bf16 operands
// (v_mfma_f32_32x32x16_bf16) and MXFP8 operands (v_mfma_scale_f32_32x32x64_f8f6f4, the e8m0 block
// scales applied by the matrix cores), fp32 sums.
//
// The weight tile is the MFMA's A operand and the token tile its B operand, so a lane holds four
// groups of four consecutive output columns of one token row.
//
// linear_tile_kernel: a workgroup computes a BM x BN tile (BM tokens, BN weight rows).  Both operands
// run through a ring of S LDS stages of 128 bytes per row (64 k in bf16, 128 k in MXFP8), filled by
// direct global -> LDS loads.  The 16-byte chunks of a row sit XOR-swizzled by row / 2: LDS serves a
// 128-bit read 16 lanes at a time, two 128-byte rows span its banks, and one chunk of 16 consecutive
// rows then hits 16 different bank groups.  A step reads its operands one MFMA sub-step ahead of the
// matrix cores; before the last sub-step's MFMAs the waves meet at the step's one barrier, the buffer
// just read is refilled and the next step's first operands are read.
// With SwiGLU each 32-row weight tile holds 16 gate and 16 up rows, so a lane holds both of an output.
// The sums pass through LDS once more in the epilogue, so that a store covers whole lines of a row.
#include <type_traits>

#include "linear_dev.h"

namespace bitmoe {

namespace {

constexpr int kXcds = 8;
template <bool MX, bool GATED, int BM, int BN, int WM, int WN, int S, int OCC>
__global__ __launch_bounds__(64 * WM * WN, OCC) void linear_tile_kernel(LinearArgs a, int m_tiles, int n_tiles) {
  constexpr int NW = WM * WN, kThreads = 64 * NW;
  constexpr int AT = BM / WM / 32, BT = BN / WN / 32;   // token and weight MFMA tiles of a wave
  constexpr int kEs = MX ? 1 : 2, kRow = 128, kStepK = kRow / kEs;
  constexpr int kSub = MX ? 2 : 4;                      // MFMA sub-steps of a step
  constexpr int kCh = MX ? 2 : 1;                       // 16-byte chunks of a lane per operand and sub-step
  constexpr int UA = BM / (8 * NW), UB = BN / (8 * NW);
  constexpr int LD = UA + UB;  // direct loads per wave and stage (the waits below count at least these)
  constexpr int kStage = (BM + BN) * kRow, kScale = MX ? (BM + BN) * 4 : 16;
  static_assert(S == 2 || S == 4, "ring depth");
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && NW % 4 == 0 && (!MX || BM + BN <= kThreads), "loads");
  // one object per stage: the compiler tracks direct loads per object, so a read of one stage does
  // not wait for another's
  __shared__ __align__(16) uint8_t st0[kStage], st1[kStage], st2[S > 2 ? kStage : 16], st3[S > 2 ? kStage : 16];
  __shared__ uint32_t sc0[kScale / 4], sc1[kScale / 4], sc2[S > 2 ? kScale / 4 : 4], sc3[S > 2 ? kScale / 4 : 4];
  const int tid = threadIdx.x, lane = wave_lane();
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = w % WM, wn = w / WM, r32 = lane & 31, hl = lane >> 5;
  const int K = a.K, kb_bytes = K * kEs, nk = (K + kStepK - 1) / kStepK;
  const bool tail = K % kStepK != 0;

  // Workgroups go to the 8 XCDs round robin.  Each XCD takes a contiguous run of tiles, ordered in
  // bands of 8 token tiles, column by column, so that the tiles running on it at a time share their
  // rows and columns in its L2.
  int tile;
  {
    const int total = m_tiles * n_tiles, per = total / kXcds, rest = total % kXcds;
    const int x = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
    tile = x * per + min(x, rest) + i;
  }
  constexpr int kBand = 8;
  const int band = tile / (kBand * n_tiles), in_band = tile - band * kBand * n_tiles;
  const int band_rows = min(kBand, m_tiles - band * kBand);
  const int64_t t0 = (int64_t)(band * kBand + in_band % band_rows) * BM;
  const int n0 = in_band / band_rows * (GATED ? BN / 2 : BN);  // first output column

  // global addresses: a resource per operand that spans the tile's rows, a byte offset per lane and
  // 8-row load; rows past the end have an offset past the resource and read zeros
  const int rows_x = (int)min((int64_t)BM, a.T - t0), rows_w = min(GATED ? BN / 2 : BN, a.n_out - n0);
  const bool up = GATED && ((w >> 1) & 1);  // this wave's loads fetch up rows
  const buf_rsrc rx = make_rsrc(a.x + t0 * kb_bytes, (uint32_t)rows_x * kb_bytes);
  const int64_t w_first = (up ? a.n_out : 0) + (int64_t)n0;
  const buf_rsrc rw = make_rsrc(a.w + w_first * kb_bytes, (uint32_t)rows_w * kb_bytes);
  const int prow = lane >> 3;
  const uint32_t chunk = 16u * (uint32_t)((lane & 7) ^ ((4 * w + (prow >> 1)) & 7));
  uint32_t xoff[UA], woff[UB];
#pragma unroll
  for (int u = 0; u < UA; ++u) {
    const int r = 8 * (NW * u + w) + prow;
    xoff[u] = r < rows_x ? (uint32_t)r * kb_bytes + chunk : kOffNone;
  }
  // LDS weight row j -> weight row of the tile (among the gate or up rows with SwiGLU)
  auto wrow = [&](int j) { return GATED ? 16 * (j >> 5) + (j & 15) : j; };
#pragma unroll
  for (int u = 0; u < UB; ++u) {
    const int r = wrow(8 * (NW * u + w) + prow);
    woff[u] = r < rows_w ? (uint32_t)r * kb_bytes + chunk : kOffNone;
  }
  // MXFP8: thread j < BM + BN fetches the four scales of stage row j
  const uint8_t* scale_row = nullptr;
  if (MX && tid < BM + BN) {
    const int ks = K / 32;
    if (tid < BM) {
      if (tid < rows_x) scale_row = a.x_scales + (t0 + tid) * ks;
    } else {
      const int j = tid - BM, r = wrow(j);
      if (r < rows_w) scale_row = a.w_scales + ((GATED && (j & 16) ? a.n_out : 0) + (int64_t)n0 + r) * ks;
    }
  }
  uint32_t sreg[S];

  // the stage buffers by index (a constant wherever they are used)
  auto stage = [&](int d) -> uint8_t* { return d == 0 ? st0 : d == 1 ? st1 : d == 2 ? st2 : st3; };
  auto scales = [&](int d) -> uint32_t* { return d == 0 ? sc0 : d == 1 ? sc1 : d == 2 ? sc2 : sc3; };
  auto load = [&](int d, int kb) {
    uint8_t* st = stage(d);
    const int ko = kb * kRow;
    if (MX) {
      uint32_t v = 0;
      if (scale_row) {
        const int left = K / 32 - 4 * kb;
        const uint8_t* p = scale_row + 4 * kb;
        if (left >= 4) {
          __builtin_memcpy(&v, p, 4);
        } else {
          for (int i = 0; i < left; ++i) v |= (uint32_t)p[i] << (8 * i);
        }
      }
      sreg[d] = v;
    }
    if (tail && kb == nk - 1) {
      const bool in = ko + (int)chunk < kb_bytes;  // a chunk is all inside the row or all outside
#pragma unroll
      for (int u = 0; u < UA; ++u)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(st + 1024 * (NW * u + w)), 16,
                                                 (int)(in ? xoff[u] : kOffNone), ko, 0, 0);
#pragma unroll
      for (int u = 0; u < UB; ++u)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(st + BM * kRow + 1024 * (NW * u + w)), 16,
                                                 (int)(in ? woff[u] : kOffNone), ko, 0, 0);
      return;
    }
#pragma unroll
    for (int u = 0; u < UA; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(st + 1024 * (NW * u + w)), 16, (int)xoff[u], ko, 0, 0);
#pragma unroll
    for (int u = 0; u < UB; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(st + BM * kRow + 1024 * (NW * u + w)), 16, (int)woff[u],
                                               ko, 0, 0);
  };

  // a lane's chunk offsets: rows 32 t + r32 share (row / 2) % 8, so the swizzle is the same for
  // every tile.  Sub-step j: bf16 chunk 2 j + hl; MXFP8 chunks 4 j + hl and 4 j + 2 + hl.
  uint32_t cofs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) cofs[j] = 16u * (uint32_t)((2 * j + hl) ^ ((r32 >> 1) & 7));
  const uint32_t xbase = (uint32_t)(32 * AT * wm + r32) * kRow, wbase = (uint32_t)(BM + 32 * BT * wn + r32) * kRow;
  struct Ops {
    u32x4 x[AT][kCh], w[BT][kCh];
    uint32_t sx[AT], sw[BT];
  };
  auto read = [&](Ops& o, int d, int j) {
    const uint8_t* st = stage(d);
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
#pragma unroll
      for (int t = 0; t < BT; ++t)
        o.w[t][c] = *reinterpret_cast<const u32x4*>(st + wbase + cofs[kCh * j + c] + 32 * kRow * t);
#pragma unroll
      for (int t = 0; t < AT; ++t)
        o.x[t][c] = *reinterpret_cast<const u32x4*>(st + xbase + cofs[kCh * j + c] + 32 * kRow * t);
    }
    if (MX) {
      const uint8_t* sc = reinterpret_cast<const uint8_t*>(scales(d)) + 2 * j + hl;
#pragma unroll
      for (int t = 0; t < BT; ++t) o.sw[t] = sc[4 * (BM + 32 * (BT * wn + t) + r32)];
#pragma unroll
      for (int t = 0; t < AT; ++t) o.sx[t] = sc[4 * (32 * (AT * wm + t) + r32)];
    }
  };
  f32x16_t acc[AT][BT];
#pragma unroll
  for (int t = 0; t < AT; ++t)
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[t][b][i] = 0.f;
  auto mfma = [&](const Ops& o) {
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int b = 0; b < BT; ++b) {
        if constexpr (MX)
          acc[t][b] = mfma_mxfp8_32x32x64(o.w[b][0], o.w[b][1], o.x[t][0], o.x[t][1], acc[t][b], o.sw[b], o.sx[t]);
        else
          acc[t][b] = mfma_bf16_32x32x16(o.w[b][0], o.x[t][0], acc[t][b]);
      }
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int b = 0; b < BT; ++b) hold(acc[t][b]);
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  auto put_scales = [&](int d) {
    if (MX && tid < BM + BN) scales(d)[tid] = sreg[d];
  };
#pragma unroll
  for (int d = 0; d < S; ++d)
    if (d < nk) load(d, d);
  if (nk >= S)
    wait_vm<(S - 1) * LD, false>();
  else
    wait_vm<0, false>();
  put_scales(0);
  wait_vm<63, true>();
  asm volatile("s_barrier" ::: "memory");
  Ops op[2];
  read(op[0], 0, 0);
  // step kb, its stage in buffer D and in LDS for all waves, its first operands in op[0]
  auto step = [&](auto D, int kb) {
    constexpr int d = decltype(D)::value;
    constexpr int next = (d + 1) % S;
#pragma unroll
    for (int j = 0; j + 1 < kSub; ++j) {
      read(op[(j + 1) & 1], d, j + 1);
      __builtin_amdgcn_sched_barrier(0);
      mfma(op[j & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (kb + 1 < nk) {
      // this wave's loads of the next stage have landed (those of later ones may be in flight)
      if (S > 2 && kb + S <= nk)
        wait_vm<(S - 2) * LD, false>();
      else
        wait_vm<0, false>();
      put_scales(next);
      wait_vm<63, true>();
      asm volatile("s_barrier" ::: "memory");
      if (kb + S < nk) load(d, kb + S);
      read(op[0], next, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    mfma(op[(kSub - 1) & 1]);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int kb = 0; kb < nk; kb += S) {
    step(I0{}, kb);
    if (kb + 1 < nk) step(I1{}, kb + 1);
    if constexpr (S > 2) {
      if (kb + 2 < nk) step(I2{}, kb + 2);
      if (kb + 3 < nk) step(I3{}, kb + 3);
    }
  }

  // ---- epilogue: 32 token rows of the wave at a time through the wave's part of the first stage
  // (rows of 32 BT sums and a pad of four), then four consecutive columns per lane
  constexpr int kPitch = 32 * BT + 4, kCols = GATED ? 16 * BT : 32 * BT, kLanes = kCols / 4;
  static_assert(NW * 32 * kPitch * 4 <= 2 * kStage, "epilogue staging");
  __syncthreads();
  constexpr bool kTwo = NW * 32 * kPitch * 4 > kStage;  // half the waves in each of two stages
  float* ep = reinterpret_cast<float*>(kTwo && w >= NW / 2 ? st1 : st0) + (kTwo ? w % (NW / 2) : w) * 32 * kPitch;
  const int ec = 4 * (lane % kLanes), n = n0 + kCols * wn + ec;
#pragma unroll
  for (int t = 0; t < AT; ++t) {
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(ep + r32 * kPitch + 32 * b + 8 * q + 4 * hl) =
            make_float4(acc[t][b][4 * q], acc[t][b][4 * q + 1], acc[t][b][4 * q + 2], acc[t][b][4 * q + 3]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += kWave / kLanes) {
      const int r = r0 + lane / kLanes;
      const int64_t tok = t0 + 32 * (AT * wm + t) + r;
      // with SwiGLU column c of the wave has its gate sum at 32 (c / 16) + c % 16, its up sum 16 further on
      const float* p = ep + r * kPitch + (GATED ? 32 * (ec / 16) + ec % 16 : ec);
      const float4 v4 = *reinterpret_cast<const float4*>(p);
      const float4 u4 = GATED ? *reinterpret_cast<const float4*>(p + 16) : v4;
      const float v[4] = {v4.x, v4.y, v4.z, v4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
      if (tok < a.T && n < a.n_out) epilogue4<GATED>(a, tok, n, v, u);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <bool MX, bool GATED, int BM, int BN, int WM, int WN, int S, int OCC>
hipError_t go_tile(const LinearArgs& a, hipStream_t s) {
  const int64_t m_tiles = ((int64_t)a.T + BM - 1) / BM;
  const int bn = GATED ? BN / 2 : BN, n_tiles = (a.n_out + bn - 1) / bn;
  linear_tile_kernel<MX, GATED, BM, BN, WM, WN, S, OCC>
      <<<(unsigned)(m_tiles * n_tiles), 64 * WM * WN, 0, s>>>(a, (int)m_tiles, n_tiles);
  return hipGetLastError();
}

template <bool MX, bool GATED>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  auto tiles = [&](int bm, int bn) { return (((int64_t)a.T + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  if constexpr (MX) {
    if (tiles(256, 128) >= 256) return go_tile<MX, GATED, 256, 128, 4, 2, 2, 2>(a, s);
  } else {
    if (tiles(256, 256) >= 128) return go_tile<MX, GATED, 256, 256, 2, 4, 2, 2>(a, s);
  }
  if (tiles(128, 128) >= 192) return go_tile<MX, GATED, 128, 128, 2, 2, 2, 2>(a, s);
  if (a.T > 64 && tiles(64, 64) >= 64) return go_tile<MX, GATED, 64, 64, 2, 2, 4, 2>(a, s);
  return launch_linear_rows(a, MX, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, bool mxfp8, hipStream_t s) {
  const bool gated = a.act == kActSwiglu;
  if (mxfp8) return gated ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return gated ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace bitmoe
