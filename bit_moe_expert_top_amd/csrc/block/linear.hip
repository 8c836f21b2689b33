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
constexpr int kRow = 128;                          // bytes of a row in a stage
constexpr int kRows = 1024 / kRow, kChunks = kRow / 16;  // rows of a load, 16-byte chunks of a row
template <bool MX, bool GATED, int BM, int BN, int WM, int WN, int WK, int S, int OCC, int kSpread>
__global__ __launch_bounds__(64 * WM * WN * WK, OCC) void linear_tile_kernel(LinearArgs a, int m_tiles, int n_tiles) {
  constexpr int NW = WM * WN, kThreads = 64 * NW;      // of one K group
  constexpr int AT = BM / WM / 32, BT = BN / WN / 32;   // token and weight MFMA tiles of a wave
  constexpr int kEs = MX ? 1 : 2, kStepK = kRow / kEs;
  constexpr int kCh = MX ? 2 : 1;                       // 16-byte chunks of a lane per operand and sub-step
  constexpr int kSub = kRow / (32 * kCh);               // MFMA sub-steps of a step
  constexpr int UA = BM / (kRows * NW), UB = BN / (kRows * NW);
  constexpr int LD = UA + UB;  // direct loads per wave and stage (the waits below count at least these)
  constexpr int kStage = (BM + BN) * kRow, kScale = MX ? BM + BN : 4;
  static_assert(LD % (kSpread * AT) == 0 || kSpread == 1, "refill parts");
  static_assert((S == 2 || S == 4) && (WK == 1 || WK == 2), "ring");
  static_assert(BM % (kRows * NW) == 0 && BN % (kRows * NW) == 0 && NW % 4 == 0, "loads");
  // one object per stage: the compiler tracks direct loads per object, so a read of one stage does
  // not wait for another's
  __shared__ __align__(16) uint8_t st0[WK * kStage], st1[WK * kStage], st2[S == 4 ? WK * kStage : 16],
      st3[S == 4 ? WK * kStage : 16];
  __shared__ uint32_t sc0[WK * kScale], sc1[WK * kScale], sc2[S == 4 ? WK * kScale : 4], sc3[S == 4 ? WK * kScale : 4];
  const int tid = threadIdx.x % kThreads, lane = wave_lane();
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int group = WK == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  const int wm = w % WM, wn = w / WM, r32 = lane & 31, hl = lane >> 5;
  const int K = a.K, kb_bytes = K * kEs, nk = ((K + kStepK - 1) / kStepK + WK - 1) / WK;
  // the group's steps are the row's steps first_step + [0, nk); what lies past K is zeros
  const int first_step = group * nk;
  const bool tail = WK > 1 || K % kStepK != 0;

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
  const bool up = GATED && ((w * kRows >> 4) & 1);  // this wave's loads fetch up rows
  const buf_rsrc rx = make_rsrc(a.x + t0 * kb_bytes, (uint32_t)rows_x * kb_bytes);
  const int64_t w_first = (up ? a.n_out : 0) + (int64_t)n0;
  const buf_rsrc rw = make_rsrc(a.w + w_first * kb_bytes, (uint32_t)rows_w * kb_bytes);
  const int prow = lane / kChunks;
  auto swizzle = [](int row) { return row >> 1 & 7; };
  const uint32_t chunk = 16u * (uint32_t)(lane % kChunks ^ swizzle(kRows * w + prow));
  uint32_t xoff[UA], woff[UB];
#pragma unroll
  for (int u = 0; u < UA; ++u) {
    const int r = kRows * (NW * u + w) + prow;
    xoff[u] = r < rows_x ? (uint32_t)r * kb_bytes + chunk : kOffNone;
  }
  // LDS weight row j -> weight row of the tile (among the gate or up rows with SwiGLU)
  auto wrow = [&](int j) { return GATED ? 16 * (j >> 5) + (j & 15) : j; };
#pragma unroll
  for (int u = 0; u < UB; ++u) {
    const int r = wrow(kRows * (NW * u + w) + prow);
    woff[u] = r < rows_w ? (uint32_t)r * kb_bytes + chunk : kOffNone;
  }
  // MXFP8: thread j fetches the scales of stage rows j, j + kThreads, ..., those of four stages at a time
  // (64 lanes read 64 rows: a load costs the same for 4 bytes as for 16; 8192 x 4096 x 2048: 95 -> 88 us)
  constexpr int SR = MX ? (BM + BN + kThreads - 1) / kThreads : 1;
  const uint8_t* scale_row[SR];
  if (MX) {
    const int ks = K / 32;
#pragma unroll
    for (int c = 0; c < SR; ++c) {
      const int j = tid + c * kThreads, r = wrow(j - BM);
      scale_row[c] = nullptr;
      if (j < BM) {
        if (j < rows_x) scale_row[c] = a.x_scales + (t0 + j) * ks;
      } else if (j < BM + BN && r < rows_w) {
        scale_row[c] = a.w_scales + ((GATED && ((j - BM) & 16) ? a.n_out : 0) + (int64_t)n0 + r) * ks;
      }
    }
  }
  uint32_t scur[SR][4], snext[SR][4];  // the scales of the four stages in use and of the next four

  // the stage buffers by index (a constant wherever they are used)
  auto stage = [&](int d) -> uint8_t* { return (d == 0 ? st0 : d == 1 ? st1 : d == 2 ? st2 : st3) + group * kStage; };
  auto scales = [&](int d) -> uint32_t* { return (d == 0 ? sc0 : d == 1 ? sc1 : d == 2 ? sc2 : sc3) + group * kScale; };
  // the scales of stages 4 q .. 4 q + 3
  auto load_scales = [&](uint32_t(&v)[SR][4], int q) {
#pragma unroll
    for (int c = 0; c < SR; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = 0;
      const int left = K / 32 - 4 * first_step - 16 * q;
      if (!scale_row[c] || left <= 0) continue;
      const uint8_t* p = scale_row[c] + 4 * first_step + 16 * q;
      if (left >= 16) {
        __builtin_memcpy(v[c], p, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 15; ++i)
          if (i < left) v[c][i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
      }
    }
  };
  // Direct load i of UA + UB (the token rows, then the weight rows) of stage kb into buffer d.
  auto load_one = [&](int d, int kb, int i, bool in) {
    const bool is_x = i < UA;
    uint8_t* dst = stage(d) + (is_x ? 1024 * (NW * i + w) : BM * kRow + 1024 * (NW * (i - UA) + w));
    const uint32_t off = is_x ? xoff[is_x ? i : 0] : woff[is_x ? 0 : i - UA];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(is_x ? rx : rw, (lds_void*)dst, 16, (int)(in ? off : kOffNone),
                                             (first_step + kb) * kRow, 0, 0);
  };
  // the first n direct loads of a stage; inner: not the last stage
  auto load = [&](int d, int kb, bool inner, int n) {
    // a chunk is all inside its row or all outside
    const bool in = (WK == 1 && inner) || !tail || (first_step + kb) * kRow + (int)chunk < kb_bytes;
#pragma unroll
    for (int i = 0; i < LD; ++i)
      if (i < n) load_one(d, kb, i, in);
  };

  // a lane's chunk offsets: the swizzle has a period of 16 rows, so it is the same for every tile.
  // Sub-step j: bf16 chunk 2 j + hl; MXFP8 chunks 4 j + hl and 4 j + 2 + hl.
  uint32_t cofs[kChunks / 2];
#pragma unroll
  for (int j = 0; j < kChunks / 2; ++j) cofs[j] = 16u * (uint32_t)((2 * j + hl) ^ swizzle(r32));
  const uint32_t xbase = (uint32_t)(32 * AT * wm + r32) * kRow, wbase = (uint32_t)(BM + 32 * BT * wn + r32) * kRow;
  struct Ops {
    u32x4 x[AT][kCh], w[BT][kCh];
    uint32_t sx[AT], sw[BT];
  };
  // the operands of sub-step j of buffer d: weight tile b, token tile t
  auto read_w = [&](Ops& o, int d, int j, int b) {
#pragma unroll
    for (int c = 0; c < kCh; ++c)
      o.w[b][c] = *reinterpret_cast<const u32x4*>(stage(d) + wbase + cofs[kCh * j + c] + 32 * kRow * b);
    if (MX) o.sw[b] = reinterpret_cast<const uint8_t*>(scales(d) + BM + 32 * (BT * wn + b) + r32)[2 * j + hl];
  };
  auto read_x = [&](Ops& o, int d, int j, int t) {
#pragma unroll
    for (int c = 0; c < kCh; ++c)
      o.x[t][c] = *reinterpret_cast<const u32x4*>(stage(d) + xbase + cofs[kCh * j + c] + 32 * kRow * t);
    if (MX) o.sx[t] = reinterpret_cast<const uint8_t*>(scales(d) + 32 * (AT * wm + t) + r32)[2 * j + hl];
  };
  f32x16_t acc[AT][BT];
#pragma unroll
  for (int t = 0; t < AT; ++t)
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[t][b][i] = 0.f;
  // the MFMAs of token tile t
  auto mfma = [&](const Ops& o, int t) {
#pragma unroll
    for (int b = 0; b < BT; ++b) {
      if constexpr (MX)
        acc[t][b] = mfma_mxfp8_32x32x64(o.w[b][0], o.w[b][1], o.x[t][0], o.x[t][1], acc[t][b], o.sw[b], o.sx[t]);
      else
        acc[t][b] = mfma_bf16_32x32x16(o.w[b][0], o.x[t][0], acc[t][b]);
    }
    // The largest tile keeps its sums in the ordinary registers; there the compiler is held to issue
    // these MFMAs here (212 -> 207 us for 8192 x 4096 x 4096 with an earlier loop; 216 us with and without it now).
    if constexpr (AT * BT == 8) {
#pragma unroll
      for (int b = 0; b < BT; ++b) hold(acc[t][b]);
    }
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  // the scales of stage kb, the stages in turn, into buffer d
  auto put_scales = [&](int d, int kb) {
    if (!MX) return;
    const int i = kb & 3;
#pragma unroll
    for (int c = 0; c < SR; ++c)
      if (tid + c * kThreads < BM + BN)
        scales(d)[tid + c * kThreads] = i == 0 ? scur[c][0] : i == 1 ? scur[c][1] : i == 2 ? scur[c][2] : scur[c][3];
    if (i == 3) {
#pragma unroll
      for (int c = 0; c < SR; ++c)
#pragma unroll
        for (int b = 0; b < 4; ++b) scur[c][b] = snext[c][b];
      load_scales(snext, kb / 4 + 2);
    }
  };
  if (MX) {
    load_scales(scur, 0);
    load_scales(snext, 1);
  }
  // Stages 0 .. S - 1; of the last one only the first part of kSpread, the others are fetched by step 0.
  if (nk > S) {
#pragma unroll
    for (int d = 0; d < S; ++d) load(d, d, true, d < S - 1 ? LD : LD / kSpread);
    wait_vm<(S - 2) * LD + LD / kSpread, false>();
  } else {
#pragma unroll
    for (int d = 0; d < S; ++d)
      if (d < nk) load(d, d, false, d < S - 1 ? LD : LD / kSpread);
    wait_vm<0, false>();
  }
  put_scales(0, 0);
  wait_vm<63, true>();
  asm volatile("s_barrier" ::: "memory");
  Ops op[2];
#pragma unroll
  for (int b = 0; b < BT; ++b) read_w(op[0], 0, 0, b);
#pragma unroll
  for (int t = 0; t < AT; ++t) read_x(op[0], 0, 0, t);
  // The epilogue takes 32 token rows of the wave at a time through the wave's part of the stages (rows of
  // 32 BT sums and a pad of four), then four consecutive columns per lane.  The residual values of the
  // next 32 rows are fetched before this turn's stores: out may be the residual, so a load behind a
  // store would wait for it.
  constexpr int kPitch = 32 * BT + 4, kCols = GATED ? 16 * BT : 32 * BT, kLanes = kCols / 4;
  constexpr int kStep = kWave / kLanes, kStores = 32 / kStep;  // rows of a store, stores of a turn
  const int ec = 4 * (lane % kLanes), n = n0 + kCols * wn + ec, er = lane / kLanes;
  const int64_t row0 = t0 + 32 * AT * wm + er;  // this lane's first row
  const int rows = n < a.n_out ? (int)max((int64_t)0, min((int64_t)32 * AT, a.T - (row0 - er))) - er : 0;
  const int64_t at0 = row0 * a.n_out + n;
  // MXFP8: bf16 values of the first 32 rows are fetched before the last step, which covers their latency (8192 x
  // 4096 x 2048 122 -> 108 us, 1000 x 2048 x 1024 9.7 -> 9.0 us, buffers changing from call to call).  fp32 values do
  // not fit the registers of 128 x 128: 30 spill, and it took 138 us instead of 113 (it takes 114 now).  In bf16
  // products it gained less than 2 %.
  constexpr bool kEarly = MX && WK == 1;
  const bool early = kEarly && a.residual && a.vec && !a.res_f32;
  uint2 first[kStores];
  // Step kb, its stage in buffer D and in LDS for all waves, its first operands in op[0].  MAIN: the
  // stages it fetches exist and are not the last, so this step loads and waits without a branch.  (Branches
  // around loads and waits let the compiler think at the loop's head that a buffer may still be
  // filling, and wait there for every load in flight.)
  auto step = [&](auto D, auto MAIN_, int kb) {
    constexpr int d = decltype(D)::value, next = (d + 1) % S;
    constexpr bool kMain = decltype(MAIN_)::value;
    if constexpr (kEarly && !kMain) {
      if (early && kb + 1 == nk) {
        const uint16_t* from = reinterpret_cast<const uint16_t*>(a.residual) + at0;
#pragma unroll
        for (int i = 0; i < kStores; ++i)
          if (i * kStep < rows) first[i] = *reinterpret_cast<const uint2*>(from + (int64_t)(i * kStep) * a.n_out);
      }
    }
    // Sub-step j: per token tile, the reads of a share of the next sub-step's operands, then the MFMAs.
    // In the last sub-step those are the next stage's, behind the barrier, and the direct loads that
    // refill this buffer are issued between the MFMAs too.
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      const bool last = j == kSub - 1;
      const bool more = !last || kMain || kb + 1 < nk;
      // sub-step part p of the refill of a buffer: p = 0 in the last sub-step of the step that read it,
      // the others in the first sub-steps of the next step
      const int p = last ? 0 : j + 1, fd = last ? d : (d + S - 1) % S, fk = last ? kb + S : kb - 1 + S;
      static_assert(kSpread <= kSub, "a refill ends before the next step's barrier");
      const bool refill = p < kSpread && (kMain || fk < nk);
      const bool in = (WK == 1 && kMain) || !tail || (first_step + fk) * kRow + (int)chunk < kb_bytes;
      if (last && more) {
        // this wave's loads of the next stage have landed (those of later ones may be in flight)
        if (kMain || kb + S <= nk)
          wait_vm<(S - 2) * LD, false>();
        else
          wait_vm<0, false>();
        put_scales(next, kb + 1);
        wait_vm<63, true>();
        asm volatile("s_barrier" ::: "memory");
      }
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        if (more) {
          // three tiles' reads per token tile, the weight tiles first (all MFMAs of a token tile need
          // them), so that the last ones have landed when the sub-step ends
#pragma unroll
          for (int i = 0; i < BT + AT; ++i) {
            if (i / 3 != t && !(t == AT - 1 && i / 3 > t)) continue;
            if (i < BT)
              read_w(op[(j + 1) & 1], last ? next : d, last ? 0 : j + 1, i < BT ? i : 0);
            else
              read_x(op[(j + 1) & 1], last ? next : d, last ? 0 : j + 1, i < BT ? 0 : i - BT);
          }
        }
        if (refill) {
#pragma unroll
          for (int i = 0; i < LD; ++i)
            if (i * AT * kSpread / LD == p * AT + t) load_one(fd, fk, i, in);
        }
        __builtin_amdgcn_sched_barrier(0);
        mfma(op[j & 1], t);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int kb = 0;
  for (; kb + 2 * S < nk; kb += S) {
    step(I0{}, std::true_type{}, kb);
    step(I1{}, std::true_type{}, kb + 1);
    if constexpr (S == 4) {
      step(I2{}, std::true_type{}, kb + 2);
      step(I3{}, std::true_type{}, kb + 3);
    }
  }
  // at most 2 S steps are left
#pragma unroll
  for (int i = 0; i < 2; ++i, kb += S) {
    if (kb < nk) step(I0{}, std::false_type{}, kb);
    if (kb + 1 < nk) step(I1{}, std::false_type{}, kb + 1);
    if constexpr (S == 4) {
      if (kb + 2 < nk) step(I2{}, std::false_type{}, kb + 2);
      if (kb + 3 < nk) step(I3{}, std::false_type{}, kb + 3);
    }
  }

  if constexpr (WK == 2) {
    // the second group's sums join the first's through its own buffers
    static_assert(NW * 64 * 16 * AT * BT * 4 <= kStage, "join");
    f32x4* join = reinterpret_cast<f32x4*>(st0 + kStage) + tid;
    __syncthreads();
    if (group == 1) {
#pragma unroll
      for (int t = 0; t < AT; ++t)
#pragma unroll
        for (int b = 0; b < BT; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            join[((t * BT + b) * 4 + q) * kThreads] =
                f32x4{acc[t][b][4 * q], acc[t][b][4 * q + 1], acc[t][b][4 * q + 2], acc[t][b][4 * q + 3]};
    }
    __syncthreads();
    if (group == 1) return;
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int b = 0; b < BT; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = join[((t * BT + b) * 4 + q) * kThreads];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][b][4 * q + i] += v[i];
        }
  }

  // ---- epilogue
  const FourBias bias = load_bias4<GATED>(a, n);
  Four res[kStores];
  auto fetch = [&](int t) {
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < kStores; ++i)
        if (32 * t + i * kStep < rows) res[i] = load_residual4(a, at0 + (int64_t)(32 * t + i * kStep) * a.n_out, n);
    }
  };
  if (early) {
#pragma unroll
    for (int i = 0; i < kStores; ++i) res[i].w[0] = first[i].x, res[i].w[1] = first[i].y;
  } else {
    fetch(0);
  }
  if constexpr (WK == 1) __syncthreads();  // all waves have read the last stage
  constexpr int kFit = kStage / (32 * kPitch * 4);  // waves whose part fits one stage
  static_assert((NW + kFit - 1) / kFit <= S, "epilogue staging");
  float* ep = reinterpret_cast<float*>(stage(w / kFit)) + w % kFit * 32 * kPitch;
  auto put = [&](const f32x16_t(&v)[BT]) {
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(ep + r32 * kPitch + 32 * b + 8 * q + 4 * hl) =
            make_float4(v[b][4 * q], v[b][4 * q + 1], v[b][4 * q + 2], v[b][4 * q + 3]);
  };
  // with SwiGLU column c of the wave has its gate sum at 32 (c / 16) + c % 16, its up sum 16 further on
  const float* get = ep + er * kPitch + (GATED ? 32 * (ec / 16) + ec % 16 : ec);
  // the loop is not unrolled, for the size of its code; the sums are picked with constant indexes
#pragma unroll 1
  for (int t = 0; t < AT; ++t) {
#pragma unroll
    for (int i = 0; i < AT; ++i)
      if (t == i) put(acc[i]);
    __builtin_amdgcn_wave_barrier();
    Four now[kStores];
#pragma unroll
    for (int i = 0; i < kStores; ++i) now[i] = res[i];
    if (t + 1 < AT) fetch(t + 1);
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

template <bool MX, bool GATED, int BM, int BN, int WM, int WN, int WK, int S, int OCC, int kSpread>
hipError_t go_tile(const LinearArgs& a, hipStream_t s) {
  const int64_t m_tiles = ((int64_t)a.T + BM - 1) / BM;
  const int bn = GATED ? BN / 2 : BN, n_tiles = (a.n_out + bn - 1) / bn;
  linear_tile_kernel<MX, GATED, BM, BN, WM, WN, WK, S, OCC, kSpread>
      <<<(unsigned)(m_tiles * n_tiles), 64 * WM * WN * WK, 0, s>>>(a, (int)m_tiles, n_tiles);
  return hipGetLastError();
}

// Which kernel: the one whose launch takes the least time by its rounds, a round being the workgroups
// that run at once (one or two to a CU).  The times of a round were measured at K = 4096 without a residual (us, by
// HIP graph replays):
//   token rows x weight rows   at once    bf16    MXFP8
//   16 x 16  (linear_rows)     256         8.2     6.1
//   32 x 16  (linear_rows)     256         9.7     7.0
//   64 x 16  (linear_rows)     256        12.7     9.8
//   64 x 64                    256        14.5    18.5 (15.1 with K split over two groups of waves)
//   64 x 64                    512        29      21.7
//   64 x 128, four stages      256        23.5    (23.2: never the least)
//   128 x 128, four stages     256        36      (28.8: never the least)
//   128 x 128                  512        67      41 (30.5 for 256)
//   256 x 256                  256       105      -  (does not fit the registers)
// e.g. bf16 of 1001 x 4096: 128 x 128 with four stages 38 us, 64 x 64 55 us; 2048 x 4096: 128 x 128 67 us,
// 64 x 128 89 us; 192 x 1024: 64 x 16 11.3 us, 64 x 64 14.5 us.
// The rule does not look at K or the epilogue, which the launch and a tile's fill and epilogue would need for small K.
// Against every variant, forced in turn (8 to 8192 token rows, 384 and 4096 weight rows, K = 256 to 4096, with and
// without a residual; buffers repeated and changing): the chosen one is within 5 % of the best from K = 1024 on, but
// for bf16 8192 x 384 x 1024 (14.6 us, 64 x 64 13.3), and up to 16 % off at K <= 512 in bf16 (8192 x 4096 x 512 with
// an fp32 residual: 256 x 256 88 us, 128 x 128 78; 512 x 4096 x 256: 7.0 and 64 x 64 6.2).
enum Variant { kRows16, kRows32, kRows64, kTile64, kTile64Split, kTile64x128, kTile128Deep, kTile128, kTile256 };
template <bool MX>
Variant choose(const LinearArgs& a) {
  Variant best = kRows16;
  double least = 1e30;
  auto consider = [&](Variant v, int bm, int bn, int at_once, double round) {
    const int64_t n = (((int64_t)a.T + bm - 1) / bm) * (((int64_t)a.N + bn - 1) / bn);
    const double t = (double)((n + at_once - 1) / at_once) * round;
    if (t < least) least = t, best = v;
  };
  consider(kRows16, 16, 16, 256, MX ? 6.1 : 8.2);
  consider(kRows32, 32, 16, 256, MX ? 7.0 : 9.7);
  consider(kRows64, 64, 16, 256, MX ? 9.8 : 12.7);
  if (MX) {
    consider(kTile64Split, 64, 64, 256, 15.1);
    consider(kTile64, 64, 64, 512, 21.7);
    consider(kTile128, 128, 128, 256, 30.5);
    consider(kTile128, 128, 128, 512, 41.0);
  } else {
    consider(kTile64, 64, 64, 256, 14.5);
    consider(kTile64x128, 64, 128, 256, 23.5);
    consider(kTile128Deep, 128, 128, 256, 36.0);
    consider(kTile128, 128, 128, 512, 67.0);
    consider(kTile256, 256, 256, 256, 105.0);
  }
  return best;
}

template <bool MX, bool GATED>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  const Variant v = choose<MX>(a);
  if (v <= kRows64) return launch_linear_rows(a, MX, v == kRows16 ? 1 : v == kRows32 ? 2 : 4, s);
  if (v == kTile64) return go_tile<MX, GATED, 64, 64, 2, 2, 1, 4, 2, 1>(a, s);
  if (v == kTile128) return go_tile<MX, GATED, 128, 128, 2, 2, 1, 2, 2, 1>(a, s);
  if constexpr (MX) return go_tile<MX, GATED, 64, 64, 2, 2, 2, 4, 2, 1>(a, s);
  if constexpr (!MX) {
    if (v == kTile64x128) return go_tile<MX, GATED, 64, 128, 2, 2, 1, 4, 2, 1>(a, s);
    if (v == kTile128Deep) return go_tile<MX, GATED, 128, 128, 2, 2, 1, 4, 1, 1>(a, s);
    return go_tile<MX, GATED, 256, 256, 2, 4, 1, 2, 2, 2>(a, s);
  }
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, bool mxfp8, hipStream_t s) {
  const bool gated = a.act == kActSwiglu;
  if (mxfp8) return gated ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return gated ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace bitmoe
