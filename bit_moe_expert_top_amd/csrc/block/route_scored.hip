// Scored top-k routing: softmax or sigmoid scores over all experts, a bias for the choice,
// group-limited selection, gates from the unbiased scores.  One wavefront per token.
//   p = sigmoid(l) or softmax(l);  c = p + bias
//   a group's score is the sum of its group_top largest c; the topk_group best groups stay
//   the k largest c of the groups that stay (without a bias: the k largest l, the same order)
//   gate = p / sum of the chosen p * scale, or p * scale
// Ties go to the lower group and the lower expert.  An expert whose c is -inf or NaN is taken
// after every other and gets gate 0; a group counts its other experts only.
#include "../common.h"
#include "../route_dev.h"
#include "block_kernels.h"

namespace bitmoe {

namespace {

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

template <int VPL>
__global__ __launch_bounds__(64 * kRouteWaves) void route_scored_kernel(RouteScoredArgs a) {
  __shared__ double lds_c[kRouteWaves][64 * VPL];
  const int lane = wave_lane(), w = threadIdx.x / kWave, E = a.E;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + w; t < a.T; t += (int64_t)gridDim.x * kRouteWaves) {
    const float* row = a.logits + t * E;
    float l[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = row[min(lane + kWave * i, E - 1)];
    double lmax = 0.0, inv_sum = 1.0;
    if (!a.sigmoid) {
      float m = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
      lmax = m;
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + kWave * i < E) z += exp((double)l[i] - lmax);
      inv_sum = 1.0 / wave_sum(z);
    }
    auto score = [&](float v) {
      return a.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - lmax) * inv_sum;
    };
    uint64_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + kWave * i;
      const double c = score(l[i]) + (a.bias ? (double)a.bias[min(e, E - 1)] : 0.0);
      const bool live = c > -__builtin_inf();
      key[i] = e >= E ? 0 : live ? order_key64(a.bias ? c : (double)l[i]) : kKeyDead;
      lds_c[w][e] = live ? c : -__builtin_inf();
    }
    if (a.n_group > 1) {
      const int gs = E / a.n_group;
      double c1 = -__builtin_inf(), c2 = -__builtin_inf();
      if (lane < a.n_group) {
        for (int j = 0; j < gs; ++j) {
          const double c = lds_c[w][lane * gs + j];
          c2 = fmax(c2, fmin(c, c1));
          c1 = fmax(c1, c);
        }
      }
      const double total = a.group_top == 2 && c2 > -__builtin_inf() ? c1 + c2 : c1;
      int better = 0;
      for (int g = 0; g < a.n_group; ++g) {
        const double o = __shfl(total, g);
        better += o > total || (o == total && g < lane);
      }
      const uint64_t kept = __ballot(lane < a.n_group && better < a.topk_group);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + kWave * i;
        if (e < E && !((kept >> (e / gs)) & 1)) key[i] = 0;
      }
    }
    int mine = 0;
    bool mine_live = false;
    for (int j = 0; j < a.k; ++j) {
      uint64_t best = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) best = max_u64(best, key[i]);
      best = wave_max_u64(best);
      int e = E;  // the lowest expert with this key
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == best) e = lane + kWave * i;
      e = wave_min_i32(e);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + kWave * i == e) key[i] = 0;
      if (lane == j) mine = e, mine_live = best > kKeyDead;
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
}

template <int VPL>
hipError_t go(const RouteScoredArgs& a, hipStream_t s) {
  const int64_t want = ((int64_t)a.T + kRouteWaves - 1) / kRouteWaves, cap = 1 << 20;
  route_scored_kernel<VPL><<<(unsigned)(want < cap ? want : cap), 64 * kRouteWaves, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const RouteScoredArgs& a, hipStream_t s) {
  const int vpl = (a.E + kWave - 1) / kWave;
  if (vpl <= 1) return go<1>(a, s);
  if (vpl <= 2) return go<2>(a, s);
  if (vpl <= 4) return go<4>(a, s);
  if (vpl <= 6) return go<6>(a, s);
  if (vpl <= 8) return go<8>(a, s);
  return go<16>(a, s);
}

}  // namespace bitmoe
