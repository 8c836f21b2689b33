// The products behind the gradients, bf16 on v_mfma_f32_32x32x16_bf16 with fp32 sums:
//   dx = dy W     out[t][k] = sum over n of dy[t][n] w[n][k]     the weights' sum runs along their rows
//   dW = dy^T x   out[n][k] = sum over t of dy[t][n] x[t][k]     both operands' sums run along their rows
// In the terms of moe_linear: out [T][N] = x W^T, where an operand that is stored [K][rows] ("K-major") is transposed on
// its way from LDS into the registers: ds_read_b64_tr_b16 gives lane i of 16 the i-th value of each of four rows of 16, of
// which every lane points at four values; two of them make a lane's 8 k of one row of the operand.
//
// Both products of a call run in one launch: together they fill the GPU where one leaves places free (1001 x 1008 x 2016: 14 us,
// one after the other 25; 16384 x 2048 x 512: 76 and 91).
// Stages of SK (64 or 32) k in LDS, filled by direct global -> LDS loads.  A row-major operand lies there as rows of 2 SK
// bytes, its 16-byte chunks XOR-swizzled by row / 2 % 8 (row / 4 % 4 for SK = 32), so that one chunk of 16 consecutive rows
// hits 16 bank groups; a K-major one as SK rows of its BM (or BN) values.  There a half wave reads 64 bytes of each of four
// rows, and these lie in different quarters of the banks where the chunks are XOR-swizzled by 4 (k % 4) (rows of 256 bytes and
// more) or 4 (k / 2 % 2) (128 bytes).
// A step loads and waits without a branch: past the last k it loads zeros.  The rest is moe_linear's: the weight tile is the
// MFMA's A operand, operands are read one sub-step of 16 k ahead, the sums pass through LDS in the epilogue.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "linear_dev.h"

namespace bitmoe {

namespace {

constexpr int kXcds = 8;

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// LDS offsets of a stage are below 2^16
__device__ __forceinline__ u32x4 read_tr(const uint8_t* p0, const uint8_t* p1) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p0));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p1));
  return u32x4{a[0], a[1], b[0], b[1]};
}

// Where a wave's direct loads of one operand (BR rows of it in the tile, NW waves) come from and go to.
template <bool KM, int BR, int NW, int SK>
struct Source {
  static constexpr int kLoads = BR * 2 * SK / 1024 / NW;  // of a wave and stage
  static constexpr int kPitch = KM ? 2 * BR : 2 * SK, kRows = 1024 / kPitch, kChunks = kPitch / 16;
  static_assert(BR * 2 * SK % (1024 * NW) == 0, "loads");
  uint32_t off[kLoads];
  uint32_t chunk;  // row-major: the lane's chunk of a row
  const uint8_t* base;
  int64_t ld;      // bytes from row to row as stored
  int rows;        // row-major: rows of the operand in the tile
  __device__ static int swizzle(int row) {
    if (KM) return BR >= 128 ? 4 * (row & 3) : 4 * (row >> 1 & 1);
    return SK == 64 ? row >> 1 & 7 : row >> 2 & 3;
  }
  // row0: the tile's first row of the operand, of `total`; K: length of the sum
  __device__ void init(const uint8_t* p, int64_t row0, int64_t total, int K, int w, int lane) {
    const int r0 = lane / kChunks, c = lane % kChunks;
    rows = (int)min((int64_t)BR, total - row0);
    ld = 2 * (KM ? total : (int64_t)K);
    base = KM ? p + 2 * row0 : p + row0 * ld;
    chunk = 16u * (uint32_t)(c ^ swizzle(kRows * w + r0));
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int r = kRows * (NW * u + w) + r0;
      off[u] = !KM && r >= rows ? kOffNone : (uint32_t)(r * ld) + 16u * (uint32_t)(c ^ swizzle(r));
    }
  }
  // load u of the stage that starts at k0 (K, the sum's end, lies within 64 rows of a K-major operand's resource)
  __device__ void load(uint8_t* stage, int u, int64_t k0, int64_t K, int64_t total, int64_t row0, int w) const {
    lds_void* dst = (lds_void*)(stage + 1024 * (NW * u + w));
    if constexpr (KM) {
      const int left = (int)max((int64_t)0, min((int64_t)SK, K - k0));
      const buf_rsrc r = make_rsrc(base + k0 * ld, (uint32_t)max(left * (int)ld - (int)(2 * row0), 0));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, (int)off[u], 0, 0, 0);
    } else {
      const buf_rsrc r = make_rsrc(base, (uint32_t)(rows * ld));
      const bool in = 2 * k0 + (int64_t)chunk < 2 * K;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, (int)(in ? off[u] : kOffNone), (int)(2 * k0), 0, 0);
    }
  }
};

// A lane's reads of one operand's 32-row tiles i0 .. i0 + N - 1.
template <bool KM, int BR, int N, int SK>
struct Reader {
  uint32_t at[KM ? N : SK / 16];
  uint32_t first;
  __device__ void init(int i0, int lane) {
    const int r32 = lane & 31, hl = lane >> 5;
    if constexpr (KM) {
      // 16 lanes point at four k rows (lane / 4 % 4) of 16 values each
      const int k4 = lane >> 2 & 3, k = 8 * hl + k4;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = 32 * (i0 + i) + 16 * (lane >> 4 & 1) + 4 * (lane & 3);  // value of the row
        at[i] = (uint32_t)(k * 2 * BR) + 16u * (uint32_t)(v / 8 ^ Source<KM, BR, 1, SK>::swizzle(k4)) + 2u * (uint32_t)(v % 8);
      }
      first = 0;
    } else {
#pragma unroll
      for (int j = 0; j < SK / 16; ++j) at[j] = 16u * (uint32_t)((2 * j + hl) ^ Source<KM, BR, 1, SK>::swizzle(r32));
      first = (uint32_t)(32 * i0 + r32) * 2 * SK;
    }
  }
  __device__ u32x4 read(const uint8_t* stage, int j, int i) const {
    if constexpr (KM) {
      const uint8_t* p = stage + at[i] + 16 * j * 2 * BR;
      return read_tr(p, p + 4 * 2 * BR);
    } else {
      return *reinterpret_cast<const u32x4*>(stage + first + at[j] + 32 * 2 * SK * i);
    }
  }
};

// One product: its operands and output, m_tiles x n_tiles tiles of it, and the splits of its sum, of `per` steps of kStepK
// each, whose parts lie one behind the other in out (fp32, where there are several).  No tiles: not wanted.
constexpr int kStepK = 64;
struct Product {
  LinearArgs a;
  int m_tiles, n_tiles, splits, per;
  __host__ __device__ int groups() const { return m_tiles * n_tiles * splits; }
};

// Workgroup `group` of a product.  x: T rows, w: N rows, sums of K; w is K-major, x is if XT.
template <bool XT, int BM, int BN, int WM, int WN, int SK, int S, int kSpread>
__device__ __forceinline__ void product_tile(const Product& p, int group, uint8_t* st0, uint8_t* st1, uint8_t* st2,
                                             uint8_t* st3) {
  LinearArgs a = p.a;
  a.act = kActNone;  // known to the compiler
  const int m_tiles = p.m_tiles, n_tiles = p.n_tiles, per = p.per * (kStepK / SK);
  constexpr int NW = WM * WN;
  constexpr int AT = BM / WM / 32, BT = BN / WN / 32;  // token and weight MFMA tiles of a wave
  typedef Source<XT, BM, NW, SK> SX;
  typedef Source<true, BN, NW, SK> SW;
  constexpr int UA = SX::kLoads, UB = SW::kLoads, LD = UA + UB;
  constexpr int kXStage = BM * 2 * SK, kStage = kXStage + BN * 2 * SK, kSub = SK / 16;
  static_assert((S == 2 || S == 4) && kSpread <= kSub && LD % kSpread == 0, "ring");
  const int tid = threadIdx.x, lane = wave_lane(), r32 = lane & 31, hl = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave), wm = w % WM, wn = w / WM;

  // Workgroups go to the 8 XCDs round robin.  Each XCD takes a contiguous run of tiles, ordered in bands of 8 token
  // tiles, column by column, so that the tiles running on it at a time share their rows and columns in its L2.
  const int total = m_tiles * n_tiles, split = group / total;
  int tile;
  {
    const int b = group - split * total, each = total / kXcds, rest = total % kXcds;
    const int x = b % kXcds, i = b / kXcds;
    tile = x * each + min(x, rest) + i;
  }
  constexpr int kBand = 8;
  const int band = tile / (kBand * n_tiles), in_band = tile - band * kBand * n_tiles;
  const int band_rows = min(kBand, m_tiles - band * kBand);
  const int64_t t0 = (int64_t)(band * kBand + in_band % band_rows) * BM;
  const int n0 = in_band / band_rows * BN;  // first output column
  const int64_t k_first = (int64_t)split * per * SK, k_end = min((int64_t)a.K, k_first + (int64_t)per * SK);
  const int nk = (int)((k_end - k_first + SK - 1) / SK);

  SX sx;
  SW sw;
  sx.init(a.x, t0, a.T, a.K, w, lane);
  sw.init(a.w, n0, a.N, a.K, w, lane);
  Reader<XT, BM, AT, SK> rx;
  Reader<true, BN, BT, SK> rw;
  rx.init(AT * wm, lane);
  rw.init(BT * wn, lane);
  // the stage buffers by index (a constant wherever they are used)
  auto stage = [&](int d) -> uint8_t* { return d == 0 ? st0 : d == 1 ? st1 : d == 2 ? st2 : st3; };
  // direct load i of stage kb into buffer d: the token operand's, then the weights'
  auto load_one = [&](int d, int kb, int i) {
    const int64_t k0 = k_first + (int64_t)kb * SK;
    if (i < UA)
      sx.load(stage(d), i, k0, k_end, a.T, t0, w);
    else
      sw.load(stage(d) + kXStage, i - UA, k0, k_end, a.N, n0, w);
  };
  struct Ops {
    u32x4 x[AT], w[BT];
  } op[2];
  f32x16_t acc[AT][BT];
#pragma unroll
  for (int t = 0; t < AT; ++t)
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[t][b][i] = 0.f;
  auto read_w = [&](Ops& o, int d, int j, int b) { o.w[b] = rw.read(stage(d) + kXStage, j, b); };
  auto read_x = [&](Ops& o, int d, int j, int t) { o.x[t] = rx.read(stage(d), j, t); };

#pragma unroll
  for (int d = 0; d < S; ++d)
#pragma unroll
    for (int i = 0; i < LD; ++i)
      if (d < S - 1 || i < LD / kSpread) load_one(d, d, i);
  wait_vm<(S - 2) * LD + LD / kSpread, false>();
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int b = 0; b < BT; ++b) read_w(op[0], 0, 0, b);
#pragma unroll
  for (int t = 0; t < AT; ++t) read_x(op[0], 0, 0, t);

  // Step kb, its stage in buffer I and in LDS for all waves, its first operands in op[0].
  auto step = [&](auto I_, int kb) {
    constexpr int d = decltype(I_)::value, next = (d + 1) % S;
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      const bool last = j == kSub - 1;
      // part p of a refill: 0 in the last sub-step of the step that read the buffer, the others in the first sub-steps of the
      // next step
      const int p = last ? 0 : j + 1, fd = last ? d : (d + S - 1) % S, fk = last ? kb + S : kb - 1 + S;
      if (last) {
        // this wave's loads of the next stage have landed (those of later ones may be in flight) and it has read this stage
        wait_vm<(S - 2) * LD, true>();
        asm volatile("s_barrier" ::: "memory");
      }
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        // a share of the next sub-step's operands, the weight tiles first (all MFMAs of a token tile need them)
#pragma unroll
        for (int i = 0; i < BT + AT; ++i) {
          constexpr int kShare = (BT + AT + AT - 1) / AT + (AT > 2 ? 1 : 0);
          if (i / kShare != t && !(t == AT - 1 && i / kShare > t)) continue;
          if (i < BT)
            read_w(op[(j + 1) & 1], last ? next : d, last ? 0 : j + 1, i < BT ? i : 0);
          else
            read_x(op[(j + 1) & 1], last ? next : d, last ? 0 : j + 1, i < BT ? 0 : i - BT);
        }
        if (p < kSpread) {
#pragma unroll
          for (int i = 0; i < LD; ++i)
            if (i * AT * kSpread / LD == p * AT + t) load_one(fd, fk, i);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < BT; ++b) acc[t][b] = mfma_bf16_32x32x16(op[j & 1].w[b], op[j & 1].x[t], acc[t][b]);
        if constexpr (AT * BT == 8) {  // held to issue here, in the ordinary registers
#pragma unroll
          for (int b = 0; b < BT; ++b) hold(acc[t][b]);
        }
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
  for (; kb + S <= nk; kb += S) {
    step(I0{}, kb);
    step(I1{}, kb + 1);
    if constexpr (S == 4) {
      step(I2{}, kb + 2);
      step(I3{}, kb + 3);
    }
  }
  if (kb < nk) step(I0{}, kb);
  if constexpr (S == 4) {
    if (kb + 1 < nk) step(I1{}, kb + 1);
    if (kb + 2 < nk) step(I2{}, kb + 2);
  }
  wait_vm<0, true>();

  // ---- epilogue: 32 token rows of the wave at a time pass through the wave's part of the stages (rows of 32 BT sums and a
  // pad of four), then a lane takes four consecutive columns.  What is added to is fetched before the turn's stores.
  constexpr int kPitch = 32 * BT + 4, kCols = 32 * BT, kLanes = kCols / 4;
  constexpr int kStep = kWave / kLanes, kStores = 32 / kStep;  // rows of a store, stores of a turn
  const int ec = 4 * (lane % kLanes), n = n0 + kCols * wn + ec, er = lane / kLanes;
  const int64_t row0 = t0 + 32 * AT * wm + er;  // this lane's first row
  const int rows = n < a.n_out ? (int)max((int64_t)0, min((int64_t)32 * AT, a.T - (row0 - er))) - er : 0;
  const int64_t at0 = row0 * a.n_out + n;
  if (split > 0) a.out = reinterpret_cast<float*>(a.out) + (int64_t)split * a.T * a.n_out;
  const FourBias none{};
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
  constexpr int kFit = kStage / (32 * kPitch * 4);  // waves whose part fits one stage
  static_assert(kFit > 0 && (NW + kFit - 1) / kFit <= S, "epilogue staging");
  float* ep = reinterpret_cast<float*>(stage(w / kFit)) + w % kFit * 32 * kPitch;
  const float* get = ep + er * kPitch + ec;
  // the loop is not unrolled, for the size of its code; the sums are picked with constant indexes
#pragma unroll 1
  for (int t = 0; t < AT; ++t) {
#pragma unroll
    for (int i = 0; i < AT; ++i)
      if (t == i) {
#pragma unroll
        for (int b = 0; b < BT; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(ep + r32 * kPitch + 32 * b + 8 * q + 4 * hl) =
                make_float4(acc[i][b][4 * q], acc[i][b][4 * q + 1], acc[i][b][4 * q + 2], acc[i][b][4 * q + 3]);
      }
    __builtin_amdgcn_wave_barrier();
    Four now[kStores];
#pragma unroll
    for (int i = 0; i < kStores; ++i) now[i] = res[i];
    if (t + 1 < AT) fetch(t + 1);
#pragma unroll
    for (int i = 0; i < kStores; ++i) {
      const float4 v4 = *reinterpret_cast<const float4*>(get + i * kStep * kPitch);
      const float v[4] = {v4.x, v4.y, v4.z, v4.w};
      if (32 * t + i * kStep < rows)
        epilogue4<kPlain, (BM * BN > 64 * 64)>(a, at0 + (int64_t)(32 * t + i * kStep) * a.n_out, n, v, v, none, now[i]);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The products of a gradient call in one launch: dx (its token operand row-major, BX x BY tiles by WX x WY waves) and dW (both
// K-major, BY x BX tiles by VX x VY waves), the one whose workgroups take longer first.
template <int BX, int BY, int WX, int WY, int VX, int VY, int SK, int S, int kSpread>
__global__ __launch_bounds__(64 * WX * WY, 2) void grad_tile_kernel(Product dx, Product dw, int dw_first) {
  static_assert(WX * WY == VX * VY, "waves");
  constexpr int kStage = (BX + BY) * 2 * SK;
  // one object per stage: the compiler tracks direct loads per object
  __shared__ __align__(16) uint8_t st0[kStage], st1[kStage], st2[S == 4 ? kStage : 16], st3[S == 4 ? kStage : 16];
  const int first = dw_first ? dw.groups() : dx.groups(), b = blockIdx.x;
  if ((b < first) == (dw_first != 0))
    product_tile<true, BY, BX, VX, VY, SK, S, kSpread>(dw, b < first ? b : b - first, st0, st1, st2, st3);
  else
    product_tile<false, BX, BY, WX, WY, SK, S, kSpread>(dx, b < first ? b : b - first, st0, st1, st2, st3);
}

// out = the sum of the splits' parts [splits][n], in their order, added to what out holds if add; four values a thread.
struct Join {
  const float* parts;
  void* out;
  int64_t n;
  int splits, out_f32, add;
  unsigned groups;
};
__global__ __launch_bounds__(256) void join_kernel(Join dx, Join dw) {
  const Join& j = blockIdx.x < dx.groups ? dx : dw;
  const unsigned b = blockIdx.x < dx.groups ? blockIdx.x : blockIdx.x - dx.groups;
  for (int64_t i = 4 * ((int64_t)b * 256 + threadIdx.x); i < j.n; i += (int64_t)j.groups * 1024) {
    f32x4 v = *reinterpret_cast<const f32x4*>(j.parts + i);
    for (int s = 1; s < j.splits; ++s) v += *reinterpret_cast<const f32x4*>(j.parts + s * j.n + i);
    if (j.out_f32) {
      f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(j.out) + i);
      *o = j.add ? v + *o : v;
    } else {
      u32x2* o = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(j.out) + i);
      if (j.add) {
        const u32x2 q = *o;
        v += f32x4{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xFFFF0000u), __uint_as_float(q[1] << 16),
                   __uint_as_float(q[1] & 0xFFFF0000u)};
      }
      *o = u32x2{f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3])};
    }
  }
}

// Which tiles, and over how many splits of each sum: what takes the least time by this model.  Workgroups run on `at_once`
// places; one takes base + slope per 1024 of its sum's length (us, measured on sums of 1024 to 8192 over full rounds):
//   dx, dW tiles                                          at once    base   slope
//   64 x 64, four stages                                  256        6      2.8
//   64 x 64, four stages                                  512        5.5    6
//   128 x 128, eight waves, four stages                   256        7      7.8
//   128 x 256, 256 x 128, eight waves, four stages
//   of 32 k                                               256        8      13.6
//   256 x 256, eight waves, two stages                    256        12.5   23.7
// (The K-major operand is the wide one: rows of 32 k of the other are half a cache line.)
// The parts of several splits are written and read once more in fp32, at about 5 TB/s and 4 us for the launch.
// Sums below 1024 (few tokens) are outside these measurements, and the model there is only near: against every tile and split,
// N x K = 4096 x 4096 and 4096 x 2048, 1 to 512 tokens, the chosen layout takes 12 to 18 % longer than the best for both products
// (T = 1: 26.0 and 23.0 us, T = 64: 27.5 and 23.8, T = 512: 60.6 and 51.2, each the best with 128 x 128 tiles), up to 40 % for dx
// alone (8 tokens: 12.7 and 9.1; 64 and more: at most 16 %), 2 % for dW alone; at 1024 x 2048 4 %.  (They take about twice their bytes' time
// in any layout: one round of tiles with short sums is mostly fill and epilogue.)
// Not kept (us at 8192 x 4096, sums of 4096, and 4096 x 2048, sums of 8192, the kept ones 216 and 118): 256 x 128 in two
// stages of 64 k 273 and 149; 256 x 256 in four stages of 32 k 219 and 173, by four waves with the sums in the
// accumulation registers 220 and 174; 128 x 128 by four waves, two workgroups to a CU, 257 and 135.  What
// bounds 256 x 256 is power: 8192 x 4096 with sums of 4096 takes 390 thousand cycles at 1.76 GHz (MFMAs alone: 262 thousand);
// without the direct loads 378 at 1.91 GHz, without the operand reads 369 at 2.2: they are nearly hidden, but lower the clock.
using Variant = GradVariant;
using Plan = GradTiles;
using Split = GradSplit;
struct Sum {  // of one product: rows, columns, length; rows = 0 where it is not wanted
  int64_t T, N, K;
};

// The time until n1 workgroups of t1 each and then n2 of t2 are done, on `at_once` places.
double makespan(double n1, double t1, double n2, double t2, double at_once) {
  const double full = std::floor(n1 / at_once), rest = n1 - full * at_once;
  double a = (full + (rest > 0 ? 1 : 0)) * t1, b = full * t1;  // rest places are free at a, the others at b
  const double end = a, whole = std::max(std::floor(n2 / at_once) - 1, 0.0);
  a += whole * t2, b += whole * t2;
  for (double left = n2 - whole * at_once; left > 0;) {
    if (b <= a) {
      left -= at_once - rest;
      b += t2;
    } else {
      left -= rest;
      a += t2;
    }
  }
  return n2 > 0 ? std::max(std::max(a, b), end) : end;
}

// A call takes about half a microsecond: what does not depend on the tiles is taken out of their loops.
Plan choose(const Sum& dx, const Sum& dw) {
  constexpr int kSplits = 5;  // 1, 2, 4, 8, 16
  struct Option {
    int splits, per;
    double join;
  };
  auto options = [](const Sum& p, Option(&o)[kSplits]) {
    if (p.T == 0) {
      o[0] = {1, 0, 0.0};
      return 1;
    }
    const int steps = std::max((int)((p.K + kStepK - 1) / kStepK), 1);
    int n = 0;
    for (int i = 0; i < kSplits; ++i) {
      const int per = (steps + (1 << i) - 1) >> i, splits = (steps + per - 1) / per;
      if (i > 0 && (per < 4 || splits == o[n - 1].splits)) break;
      o[n++] = {splits, per, splits > 1 ? 1.6e-6 * (double)p.T * (double)p.N * splits : 0.0};
    }
    return n;
  };
  Option ox[kSplits], ow[kSplits];
  const int cx = options(dx, ox), cw = options(dw, ow);
  Plan best{};
  double least = 1e30;
  // tiles of dx of 2^bx rows and 2^by columns, of dW turned round
  auto consider = [&](Variant v, int bx, int by, double at_once, double base, double slope) {
    auto tiles = [](int64_t n, int b) { return (int)((n + ((int64_t)1 << b) - 1) >> b); };
    const int xm = tiles(dx.T, bx), xn = tiles(dx.N, by), wm = tiles(dw.T, by), wn = tiles(dw.N, bx);
    for (int i = 0; i < cx; ++i) {
      const double nx = (double)xm * xn * ox[i].splits, tx = base + slope * ox[i].per / 16;
      if (i > 0 && nx > 512) break;
      for (int j = 0; j < cw; ++j) {
        const double nw = (double)wm * wn * ow[j].splits, tw = base + slope * ow[j].per / 16;
        if (j > 0 && nw > 512) break;
        const double join = ox[i].join + ow[j].join + (ox[i].splits + ow[j].splits > 2 ? 4.0 : 0.0);
        if ((nx * tx + nw * tw) / at_once + join >= least) continue;
        const bool dw_first = tw > tx;
        const double t = join + (dw_first ? makespan(nw, tw, nx, tx, at_once) : makespan(nx, tx, nw, tw, at_once));
        if (t >= least) continue;
        least = t;
        best = {v, {ox[i].splits, ox[i].per, xm, xn}, {ow[j].splits, ow[j].per, wm, wn}, dw_first};
      }
    }
  };
  consider(kTile128, 7, 7, 256, 7.0, 7.8);
  consider(kTile64, 6, 6, 256, 6.0, 2.8);
  consider(kTile64, 6, 6, 512, 5.5, 6.0);
  consider(kTile256x128, 7, 8, 256, 8.0, 13.6);
  consider(kTile256, 8, 8, 256, 12.5, 23.7);
  return best;
}

template <int BX, int BY, int WX, int WY, int VX, int VY, int SK, int S, int kSpread>
hipError_t go(const Product& dx, const Product& dw, bool dw_first, hipStream_t s) {
  grad_tile_kernel<BX, BY, WX, WY, VX, VY, SK, S, kSpread>
      <<<(unsigned)(dx.groups() + dw.groups()), 64 * WX * WY, 0, s>>>(dx, dw, dw_first);
  return hipGetLastError();
}

// out [T][N] = sums of K of x and the K-major w
Product product(const void* x, const void* w, const Sum& p, const Split& split, void* out, int out_f32, bool add,
                float* parts) {
  Product r{};
  if (p.T == 0) return r;
  r.a.x = static_cast<const uint8_t*>(x);
  r.a.w = static_cast<const uint8_t*>(w);
  r.a.T = (int)p.T, r.a.N = r.a.n_out = (int)p.N, r.a.K = (int)p.K;
  r.a.vec = 1;
  r.a.out = split.splits > 1 ? parts : out;
  r.a.res_f32 = r.a.out_f32 = split.splits > 1 ? 1 : out_f32;
  r.a.residual = add && split.splits == 1 ? out : nullptr;
  r.m_tiles = split.m_tiles, r.n_tiles = split.n_tiles, r.splits = split.splits, r.per = split.per;
  return r;
}

Join join(const Sum& p, const Split& split, const float* parts, void* out, int out_f32, bool add) {
  if (p.T == 0 || split.splits == 1) return Join{};
  const int64_t n = p.T * p.N;
  return {parts, out, n, split.splits, out_f32, add, (unsigned)std::min<int64_t>((n / 4 + 255) / 256, 1 << 16)};
}

int64_t parts_of(const Sum& p, const Split& split) { return split.splits > 1 ? p.T * p.N * split.splits : 0; }
Sum sum_dx(bool wanted, int64_t T, int64_t N, int64_t K) { return {wanted ? T : 0, K, N}; }
Sum sum_dw(bool wanted, int64_t T, int64_t N, int64_t K) { return {wanted ? N : 0, K, T}; }

}  // namespace

size_t grad_ws_bytes(int64_t T, int64_t N, int64_t K) {
  int64_t most = 0;
  for (int which = 1; which <= 3; ++which) {  // dx, dW, both
    const Sum x = sum_dx(which & 1, T, N, K), w = sum_dw(which & 2, T, N, K);
    const Plan p = choose(x, w);
    most = std::max(most, parts_of(x, p.dx) + parts_of(w, p.dw));
  }
  return (size_t)most * 4;
}

GradPlan plan_grad(const GradArgs& g) {
  const Sum x = sum_dx(g.dx, g.T, g.N, g.K), w = sum_dw(g.dw, g.T, g.N, g.K);
  const Plan p = choose(x, w);
  return {p, (size_t)(parts_of(x, p.dx) + parts_of(w, p.dw)) * 4};
}

hipError_t launch_grad(const GradArgs& g, const GradPlan& plan, void* ws, hipStream_t s) {
  const Sum x = sum_dx(g.dx, g.T, g.N, g.K), w = sum_dw(g.dw, g.T, g.N, g.K);
  if (x.T == 0 && w.T == 0) return hipSuccess;
  const Plan& p = plan.plan;
  float* parts_x = static_cast<float*>(ws);
  float* parts_w = parts_x + parts_of(x, p.dx);
  const Product dx = product(g.dy, g.w, x, p.dx, g.dx, g.dx_f32, false, parts_x);
  const Product dw = product(g.dy, g.x, w, p.dw, g.dw, g.dw_f32, g.accumulate, parts_w);
  const hipError_t e = p.tiles == kTile64        ? go<64, 64, 2, 2, 2, 2, 64, 4, 1>(dx, dw, p.dw_first, s)
                       : p.tiles == kTile128     ? go<128, 128, 4, 2, 4, 2, 64, 4, 2>(dx, dw, p.dw_first, s)
                       : p.tiles == kTile256x128 ? go<128, 256, 2, 4, 4, 2, 32, 4, 1>(dx, dw, p.dw_first, s)
                                                 : go<256, 256, 2, 4, 2, 4, 64, 2, 2>(dx, dw, p.dw_first, s);
  if (e != hipSuccess) return e;
  const Join jx = join(x, p.dx, parts_x, g.dx, g.dx_f32, false), jw = join(w, p.dw, parts_w, g.dw, g.dw_f32, g.accumulate);
  if (jx.groups + jw.groups == 0) return hipSuccess;
  join_kernel<<<jx.groups + jw.groups, 256, 0, s>>>(jx, jw);
  return hipGetLastError();
}

}  // namespace bitmoe
