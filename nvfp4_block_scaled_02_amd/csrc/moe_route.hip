// Routing to experts for gfx950: softmax or sigmoid scores, a bias that balances the experts, groups of
// experts, top-k and its weights.
//
// For a token with logits l over E experts:
//   score_e = softmax(l)_e (over all E) or 1 / (1 + exp(-l_e));   key_e = score_e + bias_e.
// An expert whose logit or key is -inf is never chosen; a NaN key comes first. Of G groups of E / G
// consecutive experts the top_groups of largest score stay, a group's score being the sum of its
// group_best (1 or 2) largest keys, of those that it has. Of their experts the top_k of largest
// key are chosen, in falling order; without a bias the order is that of the logits. Ties go to the
// lowest index. weight = scale * score, over the chosen experts' sum if renormalized.
//
// Keys and sums are held in 64 bits: what is next to each other in rank is told apart as the
// formula has it, where 32 bits would order by their own rounding. A key is compared as an
// unsigned number of the same order, in two halves.
#include "kernels.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

constexpr int kRouteTopK = (int)kMoeMaxTopK;

// Order of two doubles as unsigned numbers: increasing with the value, NaN above +inf, -inf at 0
// (never chosen).
__device__ __forceinline__ uint64_t order_of(double v) {
  v += 0.0;  // -0 counts as 0
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  if ((b & 0x7FFFFFFFFFFFFFFFull) > 0x7FF0000000000000ull) return ~0ull;
  if (b == 0xFFF0000000000000ull) return 0ull;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  const uint32_t hi = wave_max_u32((uint32_t)(v >> 32));
  const uint32_t lo = wave_max_u32((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// 1 / (1 + exp(-l)) times exp(-m), for m <= 0 with l <= m wherever l < 0 (m = 0: the score itself). A score that
// 64 bits have no room for keeps its share of a sum of its like.
__device__ __forceinline__ double sigmoid(double l, double m) {
  return exp((l < 0.0 ? l : 0.0) - m) / (1.0 + exp(l < 0.0 ? l : -l));
}

// A token per wave: lane l holds experts l, l + 64, ... in kPer registers.
template <int kPer>
__global__ void __launch_bounds__(256) route_kernel(RouteProblem p) {
  __shared__ uint64_t keys[4][64 * kPer];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= p.T) return;
  const float* row = p.logits + t * p.E;
  float l[kPer];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < p.E ? row[e] : -__builtin_inff();
    top = __builtin_fmaxf(top, l[i]);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off, 64));
  // softmax: exp(l - top), and their sum
  double share[kPer], sum = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    share[i] = l[i] == -__builtin_inff() ? 0.0 : p.sigmoid ? sigmoid(l[i], 0.0) : exp((double)l[i] - (double)top);
    sum += share[i];
  }
  sum = p.sigmoid ? 1.0 : wave_sum_f64(sum);
  uint64_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    double k = share[i] / sum;
    if (p.bias && e < p.E) k += (double)p.bias[e];
    key[i] = l[i] == -__builtin_inff() ? 0ull : order_of(k);
  }
  if (p.top_groups < p.groups) {
    // a group per lane
    const int size = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < kPer; ++i) keys[wave][lane + 64 * i] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    uint64_t best = 0ull, second = 0ull;
    if (lane < p.groups)
      for (int j = 0; j < size; ++j) {
        const uint64_t k = keys[wave][lane * size + j];
        second = k > best ? best : k > second ? k : second;
        best = k > best ? k : best;
      }
    auto value = [](uint64_t k) {
      return __builtin_bit_cast(double, (k >> 63) ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
    };
    uint64_t score = best;
    if (p.group_best == 2 && second != 0ull)
      score = best == ~0ull ? best : order_of(value(best) + value(second));
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint64_t o = __shfl(score, g, 64);
      before += o > score || (o == score && g < lane);
    }
    const uint64_t open = __ballot(lane < p.groups && before < p.top_groups);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = (lane + 64 * i) / size;
      if (g >= 64 || !((open >> g) & 1)) key[i] = 0ull;
    }
  }
  if (!p.bias) {  // the order of the logits: shares of different logits can round to the same
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] != 0ull) key[i] = order_of((double)l[i]);
  }
  // lane j: the j-th choice
  int id = -1;
  float chosen = 0.0f;
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = key[i] > best ? key[i] : best;
    best = wave_max_u64(best);
    if (best == 0ull) break;  // nothing left to choose
    int e = -1;
    float le = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e < 0) {
        const uint64_t at = __ballot(key[i] == best);
        if (at != 0) {
          const int first = __builtin_ctzll(at);
          e = 64 * i + first;
          le = __shfl(l[i], first, 64);
          if (lane == first) key[i] = 0ull;
        }
      }
    if (lane == j) {
      id = e;
      chosen = le;
    }
  }
  // weights, in the lanes of the choices
  double m = p.sigmoid ? 0.0 : (double)top;
  if (p.renormalize) {
    float most = id >= 0 ? chosen : -__builtin_inff();
#pragma unroll
    for (int off = kRouteTopK / 2; off >= 1; off >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, off, 64));
    m = p.sigmoid ? (most < 0.0f ? (double)most : 0.0) : (double)most;
  }
  double w = 0.0;
  if (id >= 0) w = p.sigmoid ? sigmoid(chosen, m) : exp((double)chosen - m);
  if (p.renormalize) {
    sum = w;
#pragma unroll
    for (int off = kRouteTopK / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  }
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = id;
    p.weights[t * p.top_k + lane] = id < 0 ? 0.0f : (float)((double)p.scale * (w / sum));
  }
}

}  // namespace

hipError_t launch_moe_route(const RouteProblem& p, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  const dim3 grid((unsigned)((p.T + 3) / 4)), block(256);
  if (p.E <= 64) hipLaunchKernelGGL(route_kernel<1>, grid, block, 0, stream, p);
  else if (p.E <= 128) hipLaunchKernelGGL(route_kernel<2>, grid, block, 0, stream, p);
  else if (p.E <= 256) hipLaunchKernelGGL(route_kernel<4>, grid, block, 0, stream, p);
  else hipLaunchKernelGGL(route_kernel<8>, grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
