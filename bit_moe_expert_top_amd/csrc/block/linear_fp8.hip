// The dense product of FP8 operands with an fp32 scale for each block of 128 (1 x 128 of the tokens, 128 x 128 of the
// weights) on v_mfma_f32_16x16x128_f8f6f4, whose K is a block: with the tokens' scale a[t][b] and the weights' c[n][b]
//   sum[t][n] = sum over blocks b of a[t][b] c[n][b] p_b,   p_b = sum over the block's k of x[t][k] w[n][k]
// so one instruction gives p_b of 16 x 16 outputs, from zero, and one fp32 FMA a value adds it with both scales.
// A lane holds four outputs of one token and one block of weight rows, so the scale is one product a token tile.  Scales
// whose products may leave the range of fp32 are told on the way, and the tile's sums made again (see scale_range).
// The FMAs of a token tile stand between the MFMAs of the next one, on the other pipe (8192 x 4096 x 4096 on 256 x 256
// tiles: 121 us, without the FMAs 108, without the direct loads 105; MFMAs alone would take 64 at the clock of 2.06 GHz that
// they leave: the LDS traffic of a step, 128 bytes a cycle, takes as long as its MFMAs).
//
// A workgroup computes BM x BN (tokens x weight rows); S LDS stages of one block of K (128 bytes a row) are filled by
// direct global -> LDS loads.  The weight tiles of a step stay in registers, the token tiles pass through two buffers.
// 16-byte chunks of a row sit XOR-swizzled by row / 2 (16 lanes that read a chunk of 16 rows hit 16 bank groups).
// With SwiGLU the 16-row weight tiles are gate and up in turn, so a lane holds both of an output.
#include <type_traits>

#include "linear_dev.h"

namespace bitmoe {

namespace {

constexpr int kXcds = 8;
constexpr int kRow = 128;                                // bytes of a row in a stage: one block of K
constexpr int kRows = 1024 / kRow, kChunks = kRow / 16;  // rows of a load, 16-byte chunks of a row

// An empty asm that reads and writes a value in ordinary registers: what computes it is not moved past.
__device__ __forceinline__ void keep(f32x4& v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
}

template <int GATED, int BM, int BN, int WM, int WN, int S, int kSpread>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_fp8_kernel(LinearArgs a, int m_tiles, int n_tiles) {
  constexpr int NW = WM * WN, kThreads = 64 * NW;
  constexpr int AT = BM / WM / 16, BT = BN / WN / 16;  // token and weight MFMA tiles of a wave
  constexpr int UA = BM / (kRows * NW), UB = BN / (kRows * NW), LD = UA + UB;  // direct loads per wave and stage
  constexpr int kStage = (BM + BN) * kRow;
  constexpr int NS = GATED ? 2 : 1;                              // weight scales of a wave: gate and up
  constexpr int kBlocks = GATED ? 2 : BN > 128 ? BN / 128 : 1;  // weight scales of the tile
  static_assert(BM % (kRows * NW) == 0 && BN % (kRows * NW) == 0 && NW % 4 == 0 && AT % 2 == 0, "loads");
  static_assert((S == 2 || S == 4) && BM % kWave == 0 && BM + kBlocks <= kThreads, "ring");
  static_assert(GATED ? BT % 2 == 0 && BN <= 256 : 128 % (16 * BT) == 0, "a wave's rows have one block row each");
  // one object per stage: the compiler tracks direct loads per object
  __shared__ __align__(16) uint8_t st0[kStage], st1[kStage], st2[S == 4 ? kStage : 16], st3[S == 4 ? kStage : 16];
  __shared__ float sc0[kThreads], sc1[kThreads], sc2[S == 4 ? kThreads : 4], sc3[S == 4 ? kThreads : 4];
  __shared__ uint32_t far_of[NW];  // whether a wave has met scales out of range
  const int tid = threadIdx.x, lane = wave_lane(), r16 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave), wm = w % WM, wn = w / WM;
  const int K = a.K, nk = (K + kRow - 1) / kRow;

  // Workgroups go to the 8 XCDs round robin.  Each XCD takes a contiguous run of tiles, ordered in bands of 8 token
  // tiles, column by column, so that the tiles running on it at a time share their rows and columns in its L2.
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

  // global addresses: a resource per operand that spans the tile's rows, a byte offset per lane and 8-row load; rows
  // past the end have an offset past the resource and read zeros
  const int rows_x = (int)min((int64_t)BM, a.T - t0), rows_w = min(GATED ? BN / 2 : BN, a.n_out - n0);
  const bool up = GATED && ((w * kRows >> 4) & 1);  // this wave's loads fetch up rows
  const buf_rsrc rx = make_rsrc(a.x + t0 * K, (uint32_t)rows_x * K);
  const buf_rsrc rw = make_rsrc(a.w + ((up ? a.n_out : 0) + (int64_t)n0) * K, (uint32_t)rows_w * K);
  const int prow = lane / kChunks;
  auto swizzle = [](int row) { return row >> 1 & 7; };
  const uint32_t chunk = 16u * (uint32_t)(lane % kChunks ^ swizzle(kRows * w + prow));
  uint32_t xoff[UA], woff[UB];
#pragma unroll
  for (int u = 0; u < UA; ++u) {
    const int r = kRows * (NW * u + w) + prow;
    xoff[u] = r < rows_x ? (uint32_t)r * K + chunk : kOffNone;
  }
#pragma unroll
  for (int u = 0; u < UB; ++u) {
    const int j = kRows * (NW * u + w) + prow, r = GATED ? 16 * (j >> 5) + (j & 15) : j;
    woff[u] = r < rows_w ? (uint32_t)r * K + chunk : kOffNone;
  }
  // Thread j fetches the scales of token row j, or of block row j - BM of the weights, those of four stages at a time
  // (64 lanes read 64 rows: a load costs the same for 4 bytes as for 16).  The last four end with the row.
  const bool of_x = w * kWave < BM;
  const int block = GATED ? (tid - BM) * ((a.n_out + 127) / 128) + n0 / 128 : n0 / 128 + tid - BM;
  const int blocks = GATED ? 2 * ((a.n_out + 127) / 128) : (a.N + 127) / 128;
  const buf_rsrc rs = of_x ? make_rsrc(a.x_scales + t0 * nk * 4, (uint32_t)rows_x * nk * 4)
                           : make_rsrc(a.w_scales, (uint32_t)blocks * nk * 4);
  const uint32_t soff = of_x                                         ? (tid < rows_x ? (uint32_t)tid * nk * 4 : kOffNone)
                        : tid - BM < kBlocks && block < blocks ? (uint32_t)block * nk * 4
                                                                     : kOffNone;
  u32x4 sreg = {0, 0, 0, 0};
  auto group = [&](int q) { return min(4 * q, max(nk - 4, 0)); };  // the first stage of the q-th four
  auto load_scales = [&](int q) {
    if (nk >= 4) {
      sreg = buf_load16s(rs, soff, 4 * group(q));
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i) sreg[i] = buf_load4(rs, i < nk ? soff + 4 * i : kOffNone);
    }
  };

  // the stage buffers by index (a constant wherever they are used)
  auto stage = [&](int d) -> uint8_t* { return d == 0 ? st0 : d == 1 ? st1 : d == 2 ? st2 : st3; };
  auto scales = [&](int d) -> float* { return d == 0 ? sc0 : d == 1 ? sc1 : d == 2 ? sc2 : sc3; };
  // direct load i of UA + UB (the token rows, then the weight rows) of stage kb into buffer d; zeros past K
  auto load_one = [&](int d, int kb, int i) {
    const bool is_x = i < UA, in = kb * kRow + (int)chunk < K;
    uint8_t* dst = stage(d) + (is_x ? 1024 * (NW * i + w) : BM * kRow + 1024 * (NW * (i - UA) + w));
    const uint32_t off = is_x ? xoff[is_x ? i : 0] : woff[is_x ? 0 : i - UA];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(is_x ? rx : rw, (lds_void*)dst, 16, (int)(in ? off : kOffNone), kb * kRow, 0, 0);
  };
  // the scales of stage kb into buffer d
  uint32_t range = 0, put = 0;  // of the scales met (see scale_range), and the last one
  auto put_scales = [&](int d, int kb) {
    const int i = kb - group(kb / 4);
    put = i == 0 ? sreg[0] : i == 1 ? sreg[1] : i == 2 ? sreg[2] : sreg[3];
    scales(d)[tid] = __uint_as_float(put);
  };

  // a lane's two chunks of a row: the swizzle has a period of 16 rows, so they are the same for every tile
  const uint32_t c0 = 16u * (uint32_t)(g ^ swizzle(r16)), c1 = 16u * (uint32_t)((4 + g) ^ swizzle(r16));
  const uint32_t xbase = (uint32_t)(16 * AT * wm + r16) * kRow, wbase = (uint32_t)(BM + 16 * BT * wn + r16) * kRow;
  u32x4 wv[BT][2], xv[2][2];
  float sx[2], sw[NS], prod[2][NS];
  f32x4 tmp[BT], acc[AT][BT];
  auto read_w = [&](int d, int b) {
    wv[b][0] = *reinterpret_cast<const u32x4*>(stage(d) + wbase + c0 + 16 * kRow * b);
    wv[b][1] = *reinterpret_cast<const u32x4*>(stage(d) + wbase + c1 + 16 * kRow * b);
  };
  auto read_x = [&](int d, int t, int into) {
    xv[into][0] = *reinterpret_cast<const u32x4*>(stage(d) + xbase + c0 + 16 * kRow * t);
    xv[into][1] = *reinterpret_cast<const u32x4*>(stage(d) + xbase + c1 + 16 * kRow * t);
    sx[into] = scales(d)[16 * (AT * wm + t) + r16];
  };
  auto read_sw = [&](int d) {
#pragma unroll
    for (int h = 0; h < NS; ++h) sw[h] = scales(d)[BM + (GATED ? h : 16 * BT * wn / 128)];
  };
  // adds the block sums in tmp[b], of token tile t
  auto add = [&](int t, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][b][i] = fmaf(prod[t & 1][GATED ? b & 1 : 0], tmp[b][i], acc[t][b][i]);
    keep(acc[t][b]);
  };
#pragma unroll
  for (int b = 0; b < BT; ++b) tmp[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < AT; ++t)
#pragma unroll
    for (int b = 0; b < BT; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < NS; ++h) prod[1][h] = 0.f;

  load_scales(0);
#pragma unroll
  for (int d = 0; d < S; ++d)
#pragma unroll
    for (int i = 0; i < LD; ++i)
      if (d < S - 1 || i * kSpread * BT / LD < BT) load_one(d, d, i);
  wait_vm<(S - 2) * LD + LD / kSpread, false>();
  put_scales(0, 0);
  range = scale_range(range, put);
  wait_vm<63, true>();
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int b = 0; b < BT; ++b) read_w(0, b);
  read_sw(0);
  read_x(0, 0, 0);

  // Step kb = 4 j + I, its stage in buffer I % S and in LDS for all waves, its weight tiles and first token tile in
  // registers.  A step loads and waits without a branch: past the last stage it loads zeros, which nothing reads.
  auto step = [&](auto I_, int kb) {
    constexpr int I = decltype(I_)::value, d = I % S, next = (I + 1) % S;
#pragma unroll
    for (int t = 0; t < AT; ++t) {
      const bool last = t == AT - 1;
      if (!last) read_x(d, t + 1, (t + 1) & 1);
#pragma unroll
      for (int h = 0; h < NS; ++h) prod[t & 1][h] = sx[t & 1] * sw[h];
      if (last) {
        // this wave's loads of the next stage have landed (those of later ones may be in flight) and it has read this stage
        wait_vm<(S - 2) * LD, true>();
        asm volatile("s_barrier" ::: "memory");
        read_x(next, 0, 0);
        read_sw(next);
      }
      if (t == 0) {
        // the next stage's scales: its buffer was last read before the barrier that this step stands behind
        put_scales(next, kb + 1);
        if constexpr (I == 2) load_scales(kb / 4 + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < BT; ++b) {
        add(t == 0 ? AT - 1 : t - 1, b);
        tmp[b] = mfma_fp8_16x16x128(wv[b][0], wv[b][1], xv[t & 1][0], xv[t & 1][1], f32x4{0.f, 0.f, 0.f, 0.f});
        keep(tmp[b]);
        if (t == 0 && b == 0) range = scale_range(range, put);  // behind an MFMA (in front 1 % slower)
        if (last) read_w(next, b);
        // the refill of a stage is spread over the last token tile of its step and the first ones of the next
        const int part = (t + 1) % AT * BT + b, fd = last ? d : (d + S - 1) % S, fk = last ? kb + S : kb - 1 + S;
#pragma unroll
        for (int i = 0; i < LD; ++i)
          if (i * kSpread * BT / LD == part) load_one(fd, fk, i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  int kb = 0;
  // no way out but the loop's end: the compiler would wait at its head for what any of the ways leaves in flight
  for (; kb + 4 <= nk; kb += 4) {
    step(I0{}, kb);
    step(I1{}, kb + 1);
    step(I2{}, kb + 2);
    step(I3{}, kb + 3);
  }
  if (kb < nk) step(I0{}, kb);
  if (kb + 1 < nk) step(I1{}, kb + 1);
  if (kb + 2 < nk) step(I2{}, kb + 2);
#pragma unroll
  for (int b = 0; b < BT; ++b) add(AT - 1, b);
  wait_vm<0, true>();
  const bool wave_far = __ballot(far_scales(range)) != 0;
  if (lane == 0) far_of[w] = wave_far;

  // ---- epilogue: 32 token rows of the wave at a time pass through the wave's part of the stages (rows of 16 BT sums and
  // a pad of four), then a lane takes four consecutive columns, so that a store covers whole lines of a row.  The residual
  // values of the next 32 rows are fetched before this turn's stores (out may be the residual).
  constexpr int kPitch = 16 * BT + 4, kCols = GATED ? 8 * BT : 16 * BT, kLanes = kCols / 4;
  constexpr int kStep = kWave / kLanes, kStores = 32 / kStep;  // rows of a store, stores of a turn
  const int ec = 4 * (lane % kLanes), n = n0 + kCols * wn + ec, er = lane / kLanes;
  const int64_t row0 = t0 + 16 * AT * wm + er;  // this lane's first row
  const int rows = n < a.n_out ? (int)max((int64_t)0, min((int64_t)16 * AT, a.T - (row0 - er))) - er : 0;
  const int64_t at0 = row0 * a.n_out + n;
  const FourBias bias = load_bias4<GATED>(a, n);
  Four res[kStores];
  auto fetch = [&](int t) {
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < kStores; ++i)
        if (32 * t + i * kStep < rows) res[i] = load_residual4(a, at0 + (int64_t)(32 * t + i * kStep) * a.n_out, n);
    }
  };
  fetch(0);
  __syncthreads();  // all waves have read the last stage
  uint32_t any_far = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) any_far |= far_of[i];
  if (__builtin_amdgcn_readfirstlane(any_far) != 0) {
    // the sums once more, a stage at a time, with the scales taken apart (see scale_range)
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int b = 0; b < BT; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int k = 0; k < nk; ++k) {
#pragma unroll
      for (int i = 0; i < LD; ++i) load_one(0, k, i);
      load_scales(k / 4);
      put_scales(0, k);
      wait_vm<0, true>();
      asm volatile("s_barrier" ::: "memory");
      read_sw(0);
      SplitScale cw[NS];
#pragma unroll
      for (int h = 0; h < NS; ++h) cw[h] = split_scale(sw[h]);
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        read_x(0, t, 0);
        const SplitScale cx = split_scale(sx[0]);
#pragma unroll
        for (int b = 0; b < BT; ++b) {
          const SplitScale& c = cw[GATED ? b & 1 : 0];
          read_w(0, b);
          tmp[b] = mfma_fp8_16x16x128(wv[b][0], wv[b][1], xv[0][0], xv[0][1], f32x4{0.f, 0.f, 0.f, 0.f}, c.e, cx.e);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][b][i] = fmaf(cx.m * c.m, tmp[b][i], acc[t][b][i]);
          keep(acc[t][b]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_vm<0, true>();
      asm volatile("s_barrier" ::: "memory");
    }
  }
  constexpr int kFit = kStage / (32 * kPitch * 4);  // waves whose part fits one stage
  static_assert(kFit > 0 && (NW + kFit - 1) / kFit <= S, "epilogue staging");
  float* ep = reinterpret_cast<float*>(stage(w / kFit)) + w % kFit * 32 * kPitch;
  const float* get = ep + er * kPitch + (GATED ? 32 * (ec / 16) + ec % 16 : ec);
  // the loop is not unrolled, for the size of its code; the sums are picked with constant indexes
#pragma unroll 1
  for (int t = 0; t < AT / 2; ++t) {
#pragma unroll
    for (int i = 0; i < AT; ++i)
      if (t == i / 2) {
#pragma unroll
        for (int b = 0; b < BT; ++b)
          *reinterpret_cast<float4*>(ep + (16 * (i & 1) + r16) * kPitch + 16 * b + 4 * g) =
              make_float4(acc[i][b][0], acc[i][b][1], acc[i][b][2], acc[i][b][3]);
      }
    __builtin_amdgcn_wave_barrier();
    Four now[kStores];
#pragma unroll
    for (int i = 0; i < kStores; ++i) now[i] = res[i];
    if (t + 1 < AT / 2) fetch(t + 1);
#pragma unroll
    for (int i = 0; i < kStores; ++i) {
      const float4 v4 = *reinterpret_cast<const float4*>(get + i * kStep * kPitch);
      const float4 u4 = GATED ? *reinterpret_cast<const float4*>(get + i * kStep * kPitch + 16) : v4;
      const float v[4] = {v4.x, v4.y, v4.z, v4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
      if (32 * t + i * kStep < rows)
        epilogue4<GATED, (BM * BN > 64 * 64)>(a, at0 + (int64_t)(32 * t + i * kStep) * a.n_out, n, v, u, bias, now[i]);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int GATED, int BM, int BN, int WM, int WN, int S, int kSpread>
hipError_t go(const LinearArgs& a, hipStream_t s) {
  const int64_t m_tiles = ((int64_t)a.T + BM - 1) / BM;
  const int bn = GATED ? BN / 2 : BN, n_tiles = (a.n_out + bn - 1) / bn;
  linear_fp8_kernel<GATED, BM, BN, WM, WN, S, kSpread>
      <<<(unsigned)(m_tiles * n_tiles), 64 * WM * WN, 0, s>>>(a, (int)m_tiles, n_tiles);
  return hipGetLastError();
}

// Which kernel: the one whose launch takes the least time by its rounds, a round being the workgroups that run at once
// (one or two to a CU).  The times of a round were measured at K = 4096 without a residual (us, back to back, buffers in
// turn of three):
//   token rows x weight rows                       at once    us
//   16 x 16, 32 x 16, 64 x 16  (linear_rows)       256        5.8, 7.0, 9.8  (6.0, 6.9, 9.4 with the test of the scales' range)
//   64 x 64, four stages                           256        12.7
//   64 x 64, four stages                           512        18.2
//   128 x 128, eight waves, four stages            256        24
//   128 x 128, four waves, two stages              512        41
//   256 x 256                                      256        60
// e.g. 1024 x 4096: 128 x 128 with four stages 26 us, with two 30, 64 x 64 33, 256 x 256 48; 2048 x 4096: 47, 41, 65, 51;
// 512 x 4096: 19.8, 27, 18.2, 48; 64 x 4096: 64 x 16 9.9 us, 64 x 64 12.3.  Over 22 products (1 to 8192 token rows, K from 512
// to 4096) the chosen one is the fastest or within 5 % of it.
enum Variant { kRows16, kRows32, kRows64, kTile64, kTile128Deep, kTile128, kTile256 };
Variant choose(const LinearArgs& a) {
  Variant best = kRows16;
  double least = 1e30;
  auto consider = [&](Variant v, int bm, int bn, int at_once, double round) {
    const int64_t n = (((int64_t)a.T + bm - 1) / bm) * (((int64_t)a.N + bn - 1) / bn);
    const double t = (double)((n + at_once - 1) / at_once) * round;
    if (t < least) least = t, best = v;
  };
  consider(kRows16, 16, 16, 256, 5.8);
  consider(kRows32, 32, 16, 256, 7.0);
  consider(kRows64, 64, 16, 256, 9.8);
  consider(kTile64, 64, 64, 256, 12.7);
  consider(kTile64, 64, 64, 512, 18.2);
  consider(kTile128Deep, 128, 128, 256, 24.0);
  consider(kTile128, 128, 128, 512, 41.0);
  consider(kTile256, 256, 256, 256, 60.0);
  return best;
}

template <int GATED>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  const Variant v = choose(a);
  if (v <= kRows64) return launch_linear_rows(a, kFp8, v == kRows16 ? 1 : v == kRows32 ? 2 : 4, s);
  if (v == kTile64) return go<GATED, 64, 64, 2, 2, 4, 2>(a, s);
  if (v == kTile128Deep) return go<GATED, 128, 128, 4, 2, 4, 2>(a, s);
  if (v == kTile128) return go<GATED, 128, 128, 2, 2, 2, 1>(a, s);
  return go<GATED, 256, 256, 2, 4, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_linear_fp8(const LinearArgs& a, hipStream_t s) {
  return a.act == kActSwiglu ? launch<kSwiglu>(a, s) : launch<kPlain>(a, s);
}

}  // namespace bitmoe
