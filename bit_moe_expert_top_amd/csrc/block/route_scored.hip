// Scored top-k routing: softmax or sigmoid scores over all experts, a bias for the choice,
// group-limited selection, gates from the unbiased scores.  One wavefront per token, or per four.
//   p = sigmoid(l) or softmax(l);  c = p + bias
//   a group's score is the sum of its group_top largest c; the topk_group best groups stay
//   the k largest c of the groups that stay (without a bias: the k largest l, the same order)
//   gate = p / sum of the chosen p * scale, or p * scale
// Ties go to the lower group and the lower expert.  An expert whose c is -inf or NaN is taken
// after every other and gets gate 0; a group counts its other experts only.
//
// The choice has to be that of 64-bit scores, and scores next to each other are told apart only
// there.  So a token is routed in fp32 with a bound on the error of every comparison that its choice
// hangs on, and where one is closer than its bound, 64 bits decide: the group sums are formed again,
// or the candidates (one to a lane) are ranked again.
//   A lane sorts its E / 64 keys once in registers (a network on the order-preserving 32-bit image of
//   c, the low bits replaced by the key's place in the lane) and k + 1 rounds of a wave maximum (six
//   DPP steps) each pop the head of one lane's list: about 20 instructions a round.  The group sums
//   come from c in LDS, 64 / G lanes to a group.
// Rows of equal logits without a bias or with equal ones (padding, or a mask that leaves nothing) tie everywhere:
// they get the first k experts.  What is left (a NaN or +inf among the logits, experts out of service among the
// chosen, more than 64 candidates that 64 bits would have to rank) is routed plainly in 64 bits.  A logit of
// -inf, a mask's value, has p = 0 exactly and stays in fp32.
#include "../common.h"
#include "../route_dev.h"
#include "block_kernels.h"

namespace bitmoe {

namespace {

// LDS words that hold values of more than one type in turn
typedef float __attribute__((may_alias)) aliased_float;
typedef uint64_t __attribute__((may_alias)) aliased_u64;
typedef float __attribute__((ext_vector_type(4), may_alias)) aliased_f32x4;

constexpr int kRouteWaves = 4;
constexpr uint64_t kKeyDead = 1;  // below the key of every selectable expert; 0: not available

__device__ __forceinline__ uint64_t order_key64(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);  // -0 -> +0
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ int wave_min_i32(int v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = min(v, __shfl_xor(v, off));
  return v;
}

// ---- One token plainly in 64 bits.  Rare, so it is written for few registers: its values stay in LDS
// (row: the logits, c_lds: E doubles of this wave) and its loops are not unrolled.
__device__ void route_token64(const RouteScoredArgs& a, const float* row, int64_t t, double* c_lds) {
  const int lane = wave_lane(), E = a.E;
  double lmax = 0.0, inv_sum = 1.0;
  if (!a.sigmoid) {
    float m = -__builtin_inff();
#pragma unroll 1
    for (int e = lane; e < E; e += kWave) m = fmaxf(m, row[e]);
#pragma unroll 1
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    lmax = m;
    double z = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += kWave) z += exp((double)row[e] - lmax);
    inv_sum = 1.0 / wave_sum(z);
  }
  auto score = [&](float v) {
    const double z = exp(a.sigmoid ? -(double)v : (double)v - lmax);
    return a.sigmoid ? 1.0 / (1.0 + z) : z * inv_sum;
  };
#pragma unroll 1
  for (int e = lane; e < E; e += kWave) {
    const double c = score(row[e]) + (a.bias ? (double)a.bias[e] : 0.0);
    c_lds[e] = c > -__builtin_inf() ? c : -__builtin_inf();
  }
  __builtin_amdgcn_wave_barrier();
  uint64_t kept = ~0ull;
  const int gs = E / a.n_group;
  if (a.n_group > 1) {
    double c1 = -__builtin_inf(), c2 = -__builtin_inf();
    if (lane < a.n_group) {
#pragma unroll 1
      for (int j = 0; j < gs; ++j) {
        const double c = c_lds[lane * gs + j];
        c2 = fmax(c2, fmin(c, c1));
        c1 = fmax(c1, c);
      }
    }
    const double total = a.group_top == 2 && c2 > -__builtin_inf() ? c1 + c2 : c1;
    int better = 0;
#pragma unroll 1
    for (int g = 0; g < a.n_group; ++g) {
      const double o = __shfl(total, g);
      better += o > total || (o == total && g < lane);
    }
    kept = __ballot(lane < a.n_group && better < a.topk_group);
  }
  // c turns into keys in place
  aliased_u64* key = reinterpret_cast<aliased_u64*>(c_lds);
  __builtin_amdgcn_wave_barrier();
#pragma unroll 1
  for (int e = lane; e < E; e += kWave) {
    const double c = c_lds[e];
    uint64_t v = c > -__builtin_inf() ? order_key64(a.bias ? c : (double)row[e]) : kKeyDead;
    if (!((kept >> (e / gs & 63)) & 1)) v = 0;
    key[e] = v;
  }
  int mine = 0;
  bool mine_live = false;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
#pragma unroll 1
    for (int e = lane; e < E; e += kWave) best = max_u64(best, key[e]);
    best = wave_max_u64(best);
    int win = E;  // the lowest expert with this key
#pragma unroll 1
    for (int e = lane; e < E && win == E; e += kWave)
      if (key[e] == best) win = e;
    win = wave_min_i32(win);
    if (lane == (win & 63)) key[win] = 0;
    __builtin_amdgcn_wave_barrier();
    if (lane == j) mine = win, mine_live = best > kKeyDead;
  }
  double p = 0.0;
  if (lane < a.k && mine_live) p = score(row[mine]);
  const double sum = wave_sum(p);
  if (a.renormalize) p = sum > 0.0 ? p / sum : 0.0;
  if (lane < a.k) {
    a.ids[t * a.k + lane] = mine;
    a.gates[t * a.k + lane] = (float)(p * (double)a.scale);
  }
}

// ---- fp32
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {  // lanes without a source, and rows left out, get 0
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// Reductions over the wave, the result uniform: exchanges within rows of 16 lanes, then the rows'
// last lanes carried on (row_bcast 15 into rows 1 and 3, row_bcast 31 into rows 2 and 3).
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {
  v = op(v, dpp0<0xB1, 0xF>(v));   // quad_perm [1,0,3,2]
  v = op(v, dpp0<0x4E, 0xF>(v));   // quad_perm [2,3,0,1]
  v = op(v, dpp0<0x141, 0xF>(v));  // row_half_mirror
  v = op(v, dpp0<0x140, 0xF>(v));  // row_mirror
  v = op(v, dpp0<0x142, 0xA>(v));  // row_bcast 15
  v = op(v, dpp0<0x143, 0xC>(v));  // row_bcast 31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ float wave_add_f32(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// The largest logit of a lane, a NaN if there is one: v_maximum3_f32, two logits an instruction.
template <int N>
__device__ __forceinline__ float largest(const float (&l)[N]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = __builtin_elementwise_maximum(m, l[i]);
  return m;
}

// Sorts in descending order by Batcher's merge exchange (Knuth, algorithm 5.2.2M), all indexes
// constants after unrolling.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&v)[N]) {
  constexpr int kTop = N > 8 ? 8 : N > 4 ? 4 : N > 2 ? 2 : 1;
#pragma unroll
  for (int p = kTop; p > 0; p >>= 1) {
#pragma unroll
    for (int q = kTop; q >= p; q >>= 1) {
      const int r = q == kTop ? 0 : p, d = q == kTop ? p : 2 * q - p;
#pragma unroll
      for (int i = 0; i + d < N; ++i)
        if ((i & p) == r) {
          const uint32_t hi = max(v[i], v[i + d]), lo = min(v[i], v[i + d]);
          v[i] = hi, v[i + d] = lo;
        }
    }
  }
}

// Routes one token; false if it is one for route_token64 (nothing is written then).
// The errors of fp32 scores, in units u = 2^-23 and in the worst case.  exp(x) is off by (0.61 |x| + 1) u of its
// value (the product with log2(e) and that constant's rounding, one ulp of the instruction; measured 0.61 |x| + 0.68).
//   sigmoid: p is off by p (1 - p) (0.61 |l| + 1) + 1.5 p <= 1.9 u (measured 0.93).
//   softmax, x = max - l (its rounding adds 0.5 x): a score's own error is p (1.11 x + 1.5) u.  The sum's is common to
//   the token's scores: S = (additions) / 2 + 1.11 ln E + 1.5 (the terms' errors weighted by p, sum of p x <= ln E),
//   14 additions and E <= 512: S <= 16 u, 22 and 1024: 21.3 u.  Scores that sum to at most 1 differ by at most 1, so
//   two of them, or two sums of two (p x <= 0.72 in all), are off against each other by S + 2.3 u.
// Adding the bias is off by |c| u / 2, dropping B <= 3 bits (4 above 512 experts) of the lower c by 8 (16) |c| u.
// Two scores compare as in 64 bits where they differ by more than kNear (1 + |c|), 32 (64) u.  A group counts another
// as surely better or worse if they differ by more than its own kNear (1 + |c1| + |c2|); two groups' sums are off by
// less than the mean of their two bounds.  That is enough: of two groups in the wrong order, the one with the larger
// bound counts the other as possible, and so every group that is as good as the other; one of them is not certain then.
// What a lane knows of its experts lane, lane + 64, ... before it sees a token.
template <int VPL>
struct LaneExperts {
  float bias[VPL];
  uint32_t group[VPL];  // the first of the group's lanes (see below); 0 for places past the last expert
};

// Whether all experts have the same logit and the same bias: then all scores and all groups tie, and the first k
// experts are chosen (the first topk_group groups' are the first ones).
__device__ __forceinline__ bool equal_row(const RouteScoredArgs& a, const float* l_lds) {
  const int lane = wave_lane();
  const float l0 = l_lds[0];
  if (__ballot(l_lds[lane] != l0)) return false;  // (past the last expert its logit is repeated)
  const float b0 = a.bias ? a.bias[0] : 0.f;
  bool same = b0 > -__builtin_inff();
#pragma unroll 1
  for (int e = lane; e < a.E; e += kWave) same &= l_lds[e] == l0 && (!a.bias || a.bias[e] == b0);
  return !__ballot(!same);
}

template <int VPL, bool SIGMOID, bool GROUPED>
__device__ __forceinline__ bool route_token(const RouteScoredArgs& a, const float (&l)[VPL], const LaneExperts<VPL>& my,
                                            int log_g, int64_t t, double* c_lds, const float* l_lds) {
  constexpr int B = VPL > 8 ? 4 : VPL > 4 ? 3 : VPL > 2 ? 2 : VPL > 1 ? 1 : 0;
  constexpr uint32_t kPlace = (1u << B) - 1;
  constexpr float kNear = VPL > 8 ? 1.0f / (1 << 17) : 1.0f / (1 << 18);
  const int lane = wave_lane(), E = a.E;
  const bool by_logit = !a.bias;
  uint32_t key[VPL];
  float lmax = 0.f, inv_sum = 1.f;
  {
    const float m = largest(l);
    if (__ballot(!(m < __builtin_inff()))) return false;
    if (!SIGMOID) {
      lmax = key_to_float(wave_max_u32(order_key(m)));
      if (lmax == -__builtin_inff()) {
        if (a.bias) return false;
        lmax = 0.f;  // p = 0 for all
      }
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) z += lane + kWave * i < E ? __expf(l[i] - lmax) : 0.f;
      z = wave_add_f32(z);
      inv_sum = z > 0.f ? 1.0f / z : 0.f;
    }
  }
  bool even = false;  // known as an equal row
  auto score = [&](float v) {
    return SIGMOID ? __builtin_amdgcn_rcpf(1.0f + __expf(-v)) : __expf(v - lmax) * inv_sum;
  };
  // the same in 64 bits; the softmax's sum only when it is needed
  auto sum64 = [&]() {
    double z = 0.0;
    if (!SIGMOID) {
#pragma unroll 1
      for (int e = lane; e < E; e += kWave) z += exp((double)l_lds[e] - (double)lmax);
      z = 1.0 / wave_sum(z);
    }
    return z;
  };
  auto score64 = [&](float v, double inv) {
    const double z = exp(SIGMOID ? -(double)v : (double)v - (double)lmax);
    return SIGMOID ? 1.0 / (1.0 + z) : z * inv;
  };
  aliased_float* cf_lds = reinterpret_cast<aliased_float*>(c_lds);  // the same memory, in fp32
  if (by_logit && !GROUPED) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = lane + kWave * i < E ? (order_key(l[i]) & ~kPlace) | i : 0;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // places past the last expert have a bias of -inf
      const float c = score(l[i]) + my.bias[i];
      key[i] = c > -__builtin_inff() ? (order_key(by_logit ? l[i] : c) & ~kPlace) | i : 0;
      if (GROUPED) cf_lds[lane + kWave * i] = c > -__builtin_inff() ? c : -__builtin_inff();
    }
  }
  if constexpr (GROUPED) {
    // 64 / G' lanes to a group (G' = 2^log_g, the power of two at or above n_group)
    const int gs = E / a.n_group, lanes = 64 >> log_g;
    const int g = lane >> (6 - log_g);
    float c1 = -__builtin_inff(), c2 = c1;
    if (g < a.n_group) {
      const aliased_float* cg = cf_lds + g * gs;
#pragma unroll 4
      for (int j = lane & (lanes - 1); j < gs; j += lanes) {
        const float c = cg[j];
        c2 = __builtin_amdgcn_fmed3f(c1, c2, c);  // c1 >= c2: the second of the three
        c1 = fmaxf(c1, c);
      }
    }
    for (int off = 1; off < lanes; off <<= 1) {
      const float o1 = __shfl_xor(c1, off), o2 = __shfl_xor(c2, off);
      c2 = fmaxf(fmaxf(c2, o2), fminf(c1, o1));
      c1 = fmaxf(c1, o1);
    }
    const float total = a.group_top == 2 && c2 > -__builtin_inff() ? c1 + c2 : c1;
    // (c2 is -inf where the sum leaves it out)
    const float near = kNear * (1.0f + fabsf(c1) + fabsf(total - c1));
    int sure = 0, maybe = -1;  // groups that are better beyond doubt, and that may be (but for itself)
    const float hi = total + near, lo = total - near;
    for (int o = 0; o < a.n_group; ++o) {
      const float other = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(total), o * lanes));
      sure += other > hi;
      maybe += !(other < lo);
    }
    bool in = g < a.n_group && maybe < a.topk_group;
    // (a group whose experts are all out of service, total = -inf, needs no decision: it has no key to lose)
    const bool close_groups = __ballot(!in && g < a.n_group && total > -__builtin_inff() && sure < a.topk_group) != 0;
    if (close_groups) even = equal_row(a, l_lds);
    if (even) {
      in = g < a.topk_group;
    } else if (close_groups) {
      // too close: the groups' sums in 64 bits
      const double inv = sum64();
#pragma unroll 1
      for (int e = lane; e < E; e += kWave) {
        const double c = score64(l_lds[e], inv) + (a.bias ? (double)a.bias[e] : 0.0);
        c_lds[e] = c > -__builtin_inf() ? c : -__builtin_inf();
      }
      __builtin_amdgcn_wave_barrier();
      double d1 = -__builtin_inf(), d2 = d1;
      if (g < a.n_group) {
#pragma unroll 1
        for (int j = lane & (lanes - 1); j < gs; j += lanes) {
          const double c = c_lds[g * gs + j];
          d2 = fmax(d2, fmin(d1, c));
          d1 = fmax(d1, c);
        }
      }
#pragma unroll 1
      for (int off = 1; off < lanes; off <<= 1) {
        const double o1 = __shfl_xor(d1, off), o2 = __shfl_xor(d2, off);
        d2 = fmax(fmax(d2, o2), fmin(d1, o1));
        d1 = fmax(d1, o1);
      }
      const double total64 = a.group_top == 2 && d2 > -__builtin_inf() ? d1 + d2 : d1;
      int better = 0;
#pragma unroll 1
      for (int o = 0; o < a.n_group; ++o) {
        const double other = __shfl(total64, o * lanes);
        better += other > total64 || (other == total64 && o < g);
      }
      in = g < a.n_group && better < a.topk_group;
    }
    const uint64_t kept = __ballot(in);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t half = my.group[i] < 32 ? (uint32_t)kept : (uint32_t)(kept >> 32);
      key[i] &= (uint32_t)__builtin_amdgcn_sbfe((int)half, my.group[i] & 31, 1);  // all ones or zero
    }
  }
  sort_desc(key);
  // lane j receives the j-th largest key and its lane
  uint32_t mine = 0, from = 0;
  auto round = [&](int j) {
    const uint32_t best = wave_max_u32(key[0]);
    const int win = __builtin_ctzll(__ballot(key[0] == best));
    if (lane == j) mine = best, from = win;
    const bool pop = lane == win;
#pragma unroll
    for (int i = 0; i + 1 < VPL; ++i) key[i] = pop ? key[i + 1] : key[i];
    key[VPL - 1] = pop ? 0 : key[VPL - 1];
    return best;
  };
  uint32_t kth = 0, next = 0;
  for (int j = 0; j < a.k; ++j) kth = round(j);
  if (kth == 0) return false;
  int n = a.k;  // candidates
  // whether key o, at or below key m in order, may be above it in 64 bits (0: no expert)
  auto close = [&](uint32_t m, uint32_t o) {
    if (by_logit) return (m & ~kPlace) == (o & ~kPlace);
    const float c = key_to_float(m & ~kPlace);
    return o != 0 && !(c - key_to_float(o & ~kPlace) > kNear * (1.0f + fabsf(c)));
  };
  next = wave_max_u32(key[0]);
  const uint32_t below = (uint32_t)__shfl_down((int)mine, 1);
  int e = (int)(from + kWave * (mine & kPlace));
  if (close(kth, next) || __ballot(lane < a.k - 1 && close(mine, below))) {
    const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)mine);
    if (((first ^ next) & ~kPlace) == 0) even |= equal_row(a, l_lds);
    // too close: every expert that may be among the k is a candidate, and 64 bits rank them
    while (!even && close(kth, next)) {
      if (n == kWave) return false;
      round(n++);
      next = wave_max_u32(key[0]);
    }
    if (even) n = 0;
    const double inv = by_logit || even ? 0.0 : sum64();
    e = (int)(from + kWave * (mine & kPlace));
    double c = -__builtin_inf();
    if (lane < n) c = by_logit ? (double)l_lds[e] : score64(l_lds[e], inv) + (double)a.bias[e];
    int rank = 0;
#pragma unroll 1
    for (int o = 0; o < n; ++o) {
      const double oc = __shfl(c, o);
      const int oe = __builtin_amdgcn_readlane(e, o);
      rank += oc > c || (oc == c && oe < e);
    }
    // lane j takes the candidate of rank j (the ranks of the candidates are a permutation)
    e = __builtin_amdgcn_ds_permute(4 * (lane < n ? rank : lane), e);
    if (even) e = lane;
  }
  // The gates are fp32, as those of moe_route: p's own error and a quotient, 7e-8 in the root mean square, against
  // 2.5e-8 of 64 bits rounded once, which would take another exp in 64 bits and, for softmax, the sum's E of them.
  float p = 0.f;
  if (lane < a.k) p = score(l_lds[e]);
  const float sum = wave_add_f32(p);
  // gates that fp32 does not hold (those of an equal row of -inf are 0)
  if (!(sum > 1e-30f) && !(even && l_lds[0] == -__builtin_inff())) return false;
  if (a.renormalize) p = sum > 0.f ? p / sum : 0.f;
  if (lane < a.k) {
    a.ids[t * a.k + lane] = e;
    a.gates[t * a.k + lane] = p * a.scale;
  }
  return true;
}

// A wave takes tokens a grid apart; the next token's logits are fetched while this one is routed.  At least
// 4 waves to a SIMD (3 above 512 experts): a token is a long chain of dependent steps, and other tokens
// fill its gaps.
constexpr int kRouteGroups = 2048;  // workgroups of a launch at most: two rounds of 4 on each of 256 CUs
template <int VPL, bool SIGMOID, bool GROUPED>
__global__ __launch_bounds__(64 * kRouteWaves, VPL > 8 ? 3 : 4) void route_scored_kernel(RouteScoredArgs a) {
  __shared__ double c_lds[kRouteWaves][64 * VPL];
  __shared__ float l_lds[kRouteWaves][64 * VPL];
  const int lane = wave_lane(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int step = gridDim.x * kRouteWaves;
  int64_t t = (int64_t)blockIdx.x * kRouteWaves + w;
  if (t >= a.T) return;
  float next[VPL];
  auto fetch = [&](int64_t u) {
    const float* row = a.logits + u * a.E;
#pragma unroll
    for (int i = 0; i < VPL; ++i) next[i] = row[min(lane + kWave * i, a.E - 1)];
  };
  fetch(t);
  LaneExperts<VPL> my;
  const int log_g = GROUPED ? 32 - __builtin_clz(a.n_group - 1) : 0;
  const float inv_gs = (float)a.n_group / (float)a.E;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + kWave * i;
    my.bias[i] = e < a.E ? (a.bias ? a.bias[e] : 0.f) : -__builtin_inff();
    // e / gs: (e + 1/2) / gs is at least 1 / (2 gs) from a whole number, far more than fp32 loses
    my.group[i] = GROUPED && e < a.E ? (uint32_t)(((float)e + 0.5f) * inv_gs) << (6 - log_g) : 0;
  }
  for (; t < a.T; t += step) {
    float l[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = next[i];
      l_lds[w][lane + kWave * i] = l[i];
    }
    if (t + step < a.T) fetch(t + step);
    if (!route_token<VPL, SIGMOID, GROUPED>(a, l, my, log_g, t, c_lds[w], l_lds[w]))
      route_token64(a, l_lds[w], t, c_lds[w]);
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- four tokens to a wave, 16 lanes each, for large batches.  A reduction over 16 lanes is four DPP steps and
// serves four tokens at once, where a whole wave for one token takes six and a broadcast.  A lane holds 8 M
// logits, sorted in chunks of eight and merged into its kTop largest keys; what falls out is remembered by its
// largest key.  Where one that was left may be among the k, more are taken, up to 16; where two taken are
// close, their scores are compared again without bits dropped and each with its own error.  A token that is not
// settled then, or whose groups are not, goes through route_token with the whole wave: that costs the wave
// 5 to 10 us (much of it fetching code that is not in the instruction cache), so the bounds are tight here.
template <int CTRL>
__device__ __forceinline__ uint32_t row_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <class Op>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, Op op) {  // the result in all 16 lanes
  v = op(v, row_dpp<0xB1>(v));   // quad_perm [1,0,3,2]
  v = op(v, row_dpp<0x4E>(v));   // quad_perm [2,3,0,1]
  v = op(v, row_dpp<0x141>(v));  // row_half_mirror
  return op(v, row_dpp<0x140>(v));  // row_mirror
}
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  return row_reduce(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ float row_add_f32(float v) {
  return __uint_as_float(row_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// From which batch on, one token / four tokens to a wave in us (top-8 with a bias; graph replays):
//                               E     T = 4096     6144         8192         16384        65536
//   sigmoid, 4 of 8 groups      128   7.4 / 6.8    8.8 / 10.5   10.1 / 8.6   16.7 / 12.5  51.2 / 25.6
//                               256   8.4 / 10.3   10.0 / 12.4  12.5 / 12.2  19.1 / 14.5  59.3 / 34.4
//                               384   8.8 / 11.7   11.7 / 13.2  13.6 / 13.4  22.7 / 18.0  73.4 / 43.9
//                               512   9.4 / 14.2   14.5 / 15.9  15.5 / 16.2  26.4 / 23.2  83.5 / 58.1
//   softmax                     128   6.1 / 6.0    7.2 / 8.9    8.2 / 6.4    12.8 / 10.5  38.1 / 20.4
//                               256   6.8 / 6.4    7.8 / 10.3   9.3 / 7.0    14.2 / 9.4   44.0 / 26.6
//                               384   7.5 / 10.1   9.3 / 8.2    11.3 / 10.5  17.2 / 12.8  50.6 / 31.2
//                               512   8.4 / 7.5    10.6 / 12.7  12.9 / 8.8   19.9 / 16.4  60.9 / 36.8
//   sigmoid                     384   6.4 / 6.6    8.1 / 10.4   9.8 / 10.1   15.0 / 12.7  45.2 / 30.7
// Below 8192 the four-token kernel's time hangs on how many tokens of the batch at hand are close (a wave that has
// one takes 3 to 5 us longer), from there on it wins or loses 1 us at most.
constexpr int kRowsMinT = 8192;
// workgroups of a launch at most (65536 tokens, 128 / 384 experts: with 1024 it took 6 / 9 % longer)
constexpr int kRowsGroups = 2048;
constexpr int kTop = 6, kRowsMaxK = 16, kRowsMaxGroups = 16;

template <int M, bool SIGMOID, bool GROUPED, bool BIASED>
__global__ __launch_bounds__(64 * kRouteWaves, M > 2 ? 3 : 4) void route_rows_kernel(RouteScoredArgs a) {
  constexpr int N = 8 * M, VPL = 2 * M;      // logits of a lane; of a lane of route_token
  constexpr int kRow = 128 * M + 4;          // c of a token in LDS, and a pad: the tokens in different banks
  constexpr int B = N > 16 ? 5 : N > 8 ? 4 : 3;
  constexpr uint32_t kPlace = (1u << B) - 1;
  constexpr uint32_t kOut = 0x007FFFFFu;     // the image of -inf
  // Errors as in route_token, but for the sum's 8 M + 3 additions: S = 4 M + 3 + 1.11 ln E <= 26 u.  Two scores, or two
  // sums of two, of magnitude m are off against each other by at most S + 2.3 u (sigmoid: 8 u) and by u m for the
  // bias: kExact (1 + m).  Dropping B bits lowers c by at most kDrop |c|.
  constexpr float kExact = SIGMOID ? 1.0f / (1 << 19) : 1.0f / (1 << 18), kDrop = 1.0f / (1 << (23 - B));
  __shared__ double lds[kRouteWaves][4 * kRow / 2];
  __shared__ uint32_t chosen[kRouteWaves][4][16];
  __shared__ __align__(16) float bias_lds[128 * M];  // -inf past the last expert
  const int lane = wave_lane(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int q = lane >> 4, E = a.E;
  int r = lane & 15;
  aliased_float* c_lds = reinterpret_cast<aliased_float*>(lds[w]) + q * kRow;
  const int log_g = GROUPED ? 32 - __builtin_clz(a.n_group - 1) : 0, gs = E / a.n_group;
  const int lanes = 16 >> log_g, g = r >> (4 - log_g);  // lanes of a group (log_g <= 4), this lane's group
  // logit 4 j + c of the lane is expert 64 j + 4 r + c
  auto expert = [&](int i) { return 64 * (i >> 2) + 4 * r + (i & 3); };
  for (int e = threadIdx.x; e < 128 * M; e += 64 * kRouteWaves) {
    const float b = e < E ? (BIASED ? a.bias[e] : 0.f) : -__builtin_inff();
    bias_lds[e] = b > -__builtin_inff() ? b : -__builtin_inff();  // a NaN is out of service too
  }
  __syncthreads();
  uint32_t first = 0;  // the first lane of the group of experts 64 j + 4 r .. + 3, four bits each
  const float inv_gs = (float)a.n_group / (float)E;
#pragma unroll
  for (int j = 0; j < 2 * M; ++j)
    if (GROUPED && expert(4 * j) < E)  // as in route_scored_kernel
      first |= ((uint32_t)(((float)expert(4 * j) + 0.5f) * inv_gs) << (4 - log_g)) << (4 * j);
  const int64_t step = (int64_t)gridDim.x * (4 * kRouteWaves);
  int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + w) * 4;
  for (; t0 < a.T; t0 += step) {
    asm volatile("" : "+v"(r));  // what follows from the lane is formed again per token, not held
    const int64_t t = t0 + q;
    const float* row = a.logits + min(t, (int64_t)a.T - 1) * E;
    float l[N];
#pragma unroll
    for (int j = 0; j < 2 * M; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(row + min(64 * j + 4 * r, E - 4));
      l[4 * j] = v.x, l[4 * j + 1] = v.y, l[4 * j + 2] = v.z, l[4 * j + 3] = v.w;
    }
    const float m = largest(l);
    bool redo = !(m < __builtin_inff());
    float lmax = 0.f, inv_sum = 1.f;
    if (!SIGMOID) {
      lmax = key_to_float(row_max_u32(order_key(m)));
      redo |= lmax == -__builtin_inff();
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) z += expert(i) < E ? __expf(l[i] - lmax) : 0.f;
      inv_sum = 1.0f / row_add_f32(z);
    }
    auto score = [&](float v) {
      return SIGMOID ? __builtin_amdgcn_rcpf(1.0f + __expf(-v)) : __expf(v - lmax) * inv_sum;
    };
    // (of a row that is not done again: no c is a NaN, and no c is -0)
    auto image = [](float c) {
      const uint32_t u = __float_as_uint(c);
      return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    };
    uint32_t key[N];  // at or below kOut: out of service
#pragma unroll
    for (int j = 0; j < 2 * M; ++j) {
      f32x4 c = {0.f, 0.f, 0.f, 0.f};
      if (BIASED || GROUPED) {
        const f32x4 b = *reinterpret_cast<const f32x4*>(bias_lds + 64 * j + 4 * r);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = score(l[4 * j + i]) + b[i];
      }
      if (GROUPED) *reinterpret_cast<aliased_f32x4*>(c_lds + 64 * j + 4 * r) = c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float by = BIASED ? c[i] : expert(4 * j + i) < E ? l[4 * j + i] + 0.f : -__builtin_inff();
        key[4 * j + i] = (image(by) & ~kPlace) | (4 * j + i);
      }
    }
    if constexpr (GROUPED) {
      float c1 = -__builtin_inff(), c2 = c1;
      if (g < a.n_group) {
        const aliased_float* cg = c_lds + g * gs;
#pragma unroll 4
        for (int j = r & (lanes - 1); j < gs; j += lanes) {
          const float c = cg[j];
          c2 = __builtin_amdgcn_fmed3f(c1, c2, c);  // c1 >= c2: the second of the three
          c1 = fmaxf(c1, c);
        }
      }
      for (int off = 1; off < lanes; off <<= 1) {
        const float o1 = __shfl_xor(c1, off), o2 = __shfl_xor(c2, off);
        c2 = fmaxf(fmaxf(c2, o2), fminf(c1, o1));
        c1 = fmaxf(c1, o1);
      }
      const float total = a.group_top == 2 && c2 > -__builtin_inff() ? c1 + c2 : c1;
      const float near = kExact * (1.0f + fabsf(c1) + fabsf(total - c1)), hi = total + near, lo = total - near;
      int sure = 0, maybe = -1;  // groups that are better beyond doubt, and that may be (but for itself)
      for (int o = 0; o < a.n_group; ++o) {
        const float other = __shfl(total, 16 * q + o * lanes);
        sure += other > hi;
        maybe += !(other < lo);
      }
      const bool in = g < a.n_group && maybe < a.topk_group;
      redo |= !in && g < a.n_group && total > -__builtin_inff() && sure < a.topk_group;  // as in route_token
      const uint32_t kept = (uint32_t)(__ballot(in) >> (16 * q));
#pragma unroll
      for (int j = 0; j < 2 * M; ++j) {
        const uint32_t on = (uint32_t)__builtin_amdgcn_sbfe((int)kept, first >> (4 * j) & 15, 1);  // all ones or zero
#pragma unroll
        for (int i = 0; i < 4; ++i) key[4 * j + i] &= on;
      }
    }
    // the lane's kTop largest keys in order, and the largest of the others
    uint32_t top[8], lost = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = key[8 * m + i];
      sort_desc(v);
      if (m == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = v[i];
        continue;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lost = max(lost, min(top[i], v[7 - i]));
        top[i] = max(top[i], v[7 - i]);
      }
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) {  // top is bitonic
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & d)) {
            const uint32_t hi = max(top[i], top[i + d]), lo = min(top[i], top[i + d]);
            top[i] = hi, top[i + d] = lo;
          }
      }
    }
    lost = max(lost, top[kTop]);
    uint32_t mine = 0;  // lane j of the row: the j-th largest key
    int pops = 0;
    auto round = [&](int j, uint32_t on) {  // on: all ones, or zero in a row that takes no part
      const uint32_t best = row_max_u32(top[0]);
      // (masks rather than selects: those the compiler turns into indexing of the list)
      const uint32_t pop = (top[0] == best ? 0xFFFFFFFFu : 0u) & on;
      if (r == j) mine = (best & on) | (mine & ~on);
#pragma unroll
      for (int i = 0; i + 1 < kTop; ++i) top[i] = (top[i + 1] & pop) | (top[i] & ~pop);
      top[kTop - 1] &= ~pop;
      pops -= (int)pop;
      if (pop) chosen[w][q][j] = (best & kPlace) | r << B;
    };
    for (int j = 0; j < a.k; ++j) round(j, 0xFFFFFFFFu);
    // whether key o, at or below key m in order, may be above it
    auto close = [&](uint32_t m, uint32_t o) {
      if (!BIASED) return (m & ~kPlace) <= (o & ~kPlace);
      const float c = key_to_float(m & ~kPlace);
      return o > kOut && !(c - key_to_float(o & ~kPlace) > kDrop * fabsf(c) + kExact * (1.0f + fabsf(c)));
    };
    int n = a.k;  // candidates of the row
    uint32_t rest = row_max_u32(max(top[0], lost));
    bool refine = false;
    for (;;) {  // more candidates, up to 16, where one that is left may be among the k
      const bool more = row_max_u32(r == a.k - 1 && close(mine, rest) ? 1u : 0u) && n < 16;
      if (!__ballot(more)) break;
      refine = true;
      round(n, more ? 0xFFFFFFFFu : 0u);
      n += more;
      rest = row_max_u32(max(top[0], lost));
    }
    redo |= r < a.k && mine <= kOut;
    redo |= r == a.k - 1 && close(mine, rest);
    // two lanes with the same key pop together
    redo |= row_reduce((uint32_t)pops, [](uint32_t x, uint32_t y) { return x + y; }) != (uint32_t)n;
    __builtin_amdgcn_wave_barrier();
    const uint32_t pick = r < n ? chosen[w][q][r] : 0;
    const int place = pick & kPlace;
    int e = min(64 * (place >> 2) + 4 * (int)(pick >> B) + (place & 3), E - 1);
    float p = 0.f, le = 0.f;
    if (r < n) {
      le = row[e];
      p = score(le);
    }
    const uint32_t after = row_dpp<0x101>(mine);  // row_shl 1: the next lane's, read with all lanes on
    if (refine || __ballot(r < n - 1 && close(mine, after))) {
      // the candidates in order of their scores without bits dropped, each with its own error
      const float c = BIASED ? p + bias_lds[e] : le;
      float err = 0.f;
      if (BIASED) {
        // S p + p (1.11 x + 1.5), as another's score may be 0 (and p = 0 where le is -inf)
        err = SIGMOID ? p * (1.0f - p) * (fabsf(le) + 2.0f) + 2.0f * p : p * (1.25f * (lmax - le) + (4 * M + 13));
        err = p > 0.f ? err : 0.f;
        err = err * 0x1p-23f + fabsf(c) * 0x1p-24f + 1e-37f;
      }
      int rank = 0;
      bool twin = false;
#pragma unroll 1
      for (int o = 0; o < 16; ++o) {
        const float oc = __shfl(c, 16 * q + o), other = __shfl(err, 16 * q + o);
        const int oe = __shfl(e, 16 * q + o);
        const bool on = o < n && o != r;
        rank += on && (oc > c || (oc == c && oe < e));
        if (BIASED) twin |= on && !(fabsf(oc - c) > err + other);
      }
      redo |= r < n && twin;
      const int to = 4 * (16 * q + (r < n ? rank : r));  // a permutation of the row
      e = __builtin_amdgcn_ds_permute(to, e);
      p = __uint_as_float(__builtin_amdgcn_ds_permute(to, (int)__float_as_uint(p)));
    }
    if (r >= a.k) p = 0.f;
    const float sum = row_add_f32(p);
    redo |= !(sum > 1e-30f);
    uint64_t again = __ballot(redo);
    again |= again >> 8, again |= again >> 4, again |= again >> 2, again |= again >> 1;
    again &= 0x0001000100010001ull;  // one bit per token
    if (t < a.T && r < a.k && !(again >> (16 * q) & 1)) {
      a.ids[t * a.k + r] = e;
      a.gates[t * a.k + r] = (a.renormalize ? p / sum : p) * a.scale;
    }
    if (again) {
      int l0 = lane;
      asm volatile("" : "+v"(l0));
      LaneExperts<VPL> my;
      const int lg = GROUPED ? log_g : 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int x = l0 + kWave * i;
        my.bias[i] = bias_lds[x];
        my.group[i] = GROUPED && x < E ? (uint32_t)(((float)x + 0.5f) * inv_gs) << (6 - lg) : 0;
      }
      float* l_lds = reinterpret_cast<float*>(lds[w] + 64 * VPL);
      for (; again; again &= again - 1) {
        const int64_t u = t0 + (__builtin_ctzll(again) >> 4);
        if (u >= a.T) break;
        __builtin_amdgcn_wave_barrier();
        float lu[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          lu[i] = a.logits[u * E + min(l0 + kWave * i, E - 1)];
          l_lds[l0 + kWave * i] = lu[i];
        }
        if (!route_token<VPL, SIGMOID, GROUPED>(a, lu, my, lg, u, lds[w], l_lds)) route_token64(a, l_lds, u, lds[w]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int VPL, bool SIGMOID, bool GROUPED>
hipError_t start(const RouteScoredArgs& a, hipStream_t s) {
  const int64_t want = ((int64_t)a.T + kRouteWaves - 1) / kRouteWaves;
  route_scored_kernel<VPL, SIGMOID, GROUPED>
      <<<(unsigned)(want < kRouteGroups ? want : kRouteGroups), 64 * kRouteWaves, 0, s>>>(a);
  return hipGetLastError();
}

template <int M, bool SIGMOID, bool GROUPED>
hipError_t start_rows(const RouteScoredArgs& a, hipStream_t s) {
  const int64_t want = ((int64_t)a.T + 4 * kRouteWaves - 1) / (4 * kRouteWaves);
  const unsigned grid = (unsigned)(want < kRowsGroups ? want : kRowsGroups);
  if (a.bias)
    route_rows_kernel<M, SIGMOID, GROUPED, true><<<grid, 64 * kRouteWaves, 0, s>>>(a);
  else
    route_rows_kernel<M, SIGMOID, GROUPED, false><<<grid, 64 * kRouteWaves, 0, s>>>(a);
  return hipGetLastError();
}

template <int M>
hipError_t go_rows(const RouteScoredArgs& a, hipStream_t s) {
  if (a.n_group > 1) return a.sigmoid ? start_rows<M, true, true>(a, s) : start_rows<M, false, true>(a, s);
  return a.sigmoid ? start_rows<M, true, false>(a, s) : start_rows<M, false, false>(a, s);
}

template <int VPL>
hipError_t go(const RouteScoredArgs& a, hipStream_t s) {
  if (a.n_group > 1) return a.sigmoid ? start<VPL, true, true>(a, s) : start<VPL, false, true>(a, s);
  return a.sigmoid ? start<VPL, true, false>(a, s) : start<VPL, false, false>(a, s);
}

}  // namespace

hipError_t launch_route_scored(const RouteScoredArgs& a, hipStream_t s) {
  if (a.T >= kRowsMinT && a.E <= 512 && a.E % 4 == 0 && a.k <= kRowsMaxK && a.n_group <= kRowsMaxGroups &&
      (a.n_group == 1 || a.E / a.n_group % 4 == 0) &&
      reinterpret_cast<uintptr_t>(a.logits) % 16 == 0) {
    if (a.E <= 128) return go_rows<1>(a, s);
    if (a.E <= 256) return go_rows<2>(a, s);
    if (a.E <= 384) return go_rows<3>(a, s);
    return go_rows<4>(a, s);
  }
  const int vpl = (a.E + kWave - 1) / kWave;
  if (vpl <= 1) return go<1>(a, s);
  if (vpl <= 2) return go<2>(a, s);
  if (vpl <= 4) return go<4>(a, s);
  if (vpl <= 6) return go<6>(a, s);
  if (vpl <= 8) return go<8>(a, s);
  return go<16>(a, s);
}

}  // namespace bitmoe
