// Routing to experts for gfx950: softmax or sigmoid scores, a bias that balances the experts, groups of
// experts, top-k and its weights.
//
// For a token with logits l over E experts:
//   score_e = softmax(l)_e (over all E) or 1 / (1 + exp(-l_e));   key_e = score_e + bias_e.
// An expert whose logit or key is -inf is never chosen; a NaN key comes first. Of G groups of E / G
// consecutive experts the top_groups of largest score stay, a group's score being the sum of its
// group_best (1 or 2) largest keys, of those that it has. Of their experts the top_k of largest
// key are chosen, in falling order. Without a bias the order is that of the logits, of groups too if
// their largest alone counts. Ties go to the lowest index. weight = scale * score, over the chosen experts' sum if renormalized.
//
// Keys and sums are defined in 64 bits: what is next to each other in rank is told apart as the formula
// has it, where 32 bits would order by their own rounding. Computing them so for all experts is
// bound by the 64-bit exponentials and the selection of 64-bit keys (32768 x 256, 73 us for 36 MB). So
// 16 lanes choose for a token by 32-bit keys (route_rows; 23 us), and know when these do not tell: two
// keys next to each other closer than their error bound. Those few are compared as the formula has
// them; what that leaves, some tokens in ten thousand, a whole wave chooses again in 64 bits
// (route_exact).
#include "kernels.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

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

// A choice's weight, in the first 16 lanes of a wave or in each 16: id and logit are the lane's, top the
// largest logit and sum, under softmax, the sum of exp(logit - top) over all experts (not needed if
// renormalized). Where renormalized, exponentials are taken relative to the chosen ones'
// largest: one that 64 bits have no room for keeps its share.
template <bool kSigmoid>
__device__ __forceinline__ void store_choice(const RouteProblem& p, int64_t t, int j, int id, float logit, float top,
                                             double sum) {
  double m = kSigmoid ? 0.0 : (double)top;
  if (p.renormalize) {
    float most = id >= 0 ? logit : -__builtin_inff();
#pragma unroll
    for (int off = kRouteTopK / 2; off >= 1; off >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, off, 64));
    m = kSigmoid ? (most < 0.0f ? (double)most : 0.0) : (double)most;
  }
  double w = 0.0;
  if (id >= 0) w = kSigmoid ? sigmoid(logit, m) : exp((double)logit - m);
  if (p.renormalize) {
    sum = w;
#pragma unroll
    for (int off = kRouteTopK / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  } else if (kSigmoid) {
    sum = 1.0;
  }
  if (j < p.top_k) {
    p.ids[t * p.top_k + j] = id;
    p.weights[t * p.top_k + j] = id < 0 ? 0.0f : (float)((double)p.scale * (w / sum));
  }
}

// A token by a wave, in 64 bits: lane l holds experts l, l + 64, ... in kPer registers; `keys` is the
// wave's.
template <int kPer>
__device__ __forceinline__ void route_exact(const RouteProblem& p, int64_t t, int lane, uint64_t* keys) {
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
  auto by_logit = [&]() {  // the order of the logits: shares of different logits can round to the same
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] != 0ull) key[i] = order_of((double)l[i]);
  };
  if (!p.bias && p.group_best == 1) by_logit();
  if (p.top_groups < p.groups) {
    // a group per lane
    const int size = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < kPer; ++i) keys[lane + 64 * i] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    uint64_t best = 0ull, second = 0ull;
    if (lane < p.groups) {
#pragma unroll 8
      for (int j = 0; j < size; ++j) {
        const uint64_t k = keys[lane * size + j];
        second = k > best ? best : k > second ? k : second;
        best = k > best ? k : best;
      }
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
  if (!p.bias && p.group_best == 2) by_logit();
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
  if (p.sigmoid) store_choice<true>(p, t, lane, id, chosen, top, sum);
  else store_choice<false>(p, t, lane, id, chosen, top, sum);
}
template <int kPer>
__global__ void __launch_bounds__(256) route_exact_kernel(RouteProblem p) {
  __shared__ uint64_t keys[4][64 * kPer];
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t < p.T) route_exact<kPer>(p, t, threadIdx.x & 63, keys[threadIdx.x >> 6]);
}

// ---- 16 lanes to a token -------------------------------------------------------------------
//
// Lane r of a row of 16 holds experts r * per .. r * per + per - 1 (per = E / 16, rounded up), so
// that a group of experts is one or several whole lanes. Of a 32-bit key the lowest bits are the
// expert's place in its lane (from the last one down), so that the largest key of a row and
// the lane that has it name an expert. A round takes the largest key below the round before's,
// which needs no key to be cleared: with v = before - 1 - key, unsigned, keys that are not
// below it wrap around to the largest v.
template <int kCtrl>
__device__ __forceinline__ uint32_t row_lane(uint32_t v) {  // of the row's lanes, all of them there
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  v = min(v, row_lane<0x121>(v));  // row_ror 1, 2, 4, 8
  v = min(v, row_lane<0x122>(v));
  v = min(v, row_lane<0x124>(v));
  return min(v, row_lane<0x128>(v));
}
__device__ __forceinline__ float row_maxf(float v) {
  v = __builtin_fmaxf(v, u2f(row_lane<0x121>(f2u(v))));
  v = __builtin_fmaxf(v, u2f(row_lane<0x122>(f2u(v))));
  v = __builtin_fmaxf(v, u2f(row_lane<0x124>(f2u(v))));
  return __builtin_fmaxf(v, u2f(row_lane<0x128>(f2u(v))));
}
__device__ __forceinline__ float row_sumf(float v) {
  v += u2f(row_lane<0x121>(f2u(v)));
  v += u2f(row_lane<0x122>(f2u(v)));
  v += u2f(row_lane<0x124>(f2u(v)));
  return v + u2f(row_lane<0x128>(f2u(v)));
}
__device__ __forceinline__ double row_sum_f64(double v) {
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
// Keys: a float as an unsigned number of the same order; to name an expert its lowest bits (kPlace) take
// its place. -inf becomes at most kPlace (nothing to choose), the lowest finite value more, +inf and NaN
// at least kOdd.
template <uint32_t kPlace>
struct Key32 {
  static constexpr uint32_t kBase = 0x007FFFFFu - kPlace, kOdd = 0xFF800000u - kBase;
  static __device__ __forceinline__ uint32_t whole(float v) {
    const uint32_t b = f2u(v + 0.0f);  // -0 counts as 0
    return (b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) - kBase;
  }
  static __device__ __forceinline__ uint32_t cut(uint32_t key, uint32_t place) { return (key & ~kPlace) | place; }
  static __device__ __forceinline__ float value(uint32_t key) {
    const uint32_t k = key + kBase;
    return u2f((k >> 31) ? k ^ 0x80000000u : ~k);
  }
};

// kScored: keys are scores with their bias, as 32 bits have them. Else they are the logits, cut by the
// bits of the place alone.
//
// How far such a key is off. Its cut: kPer - 1 last places, with the rounding of the sum with the bias
// below kPer 2^-22 of its value together (cut). A sigmoid s: its
// exponential's argument is off by at most 2.2 * 2^-24 of itself, which moves s by that times
// |l| s (1 - s) < 0.23; the hardware's exponential and reciprocal, a last place each (2^-23), move
// it by s (1 - s) 2^-23 and s 2^-23, the sum between them by s 2^-24: below 2^-22 in all. A share p
// of a softmax with largest share m: likewise |l - top| exp(l - top) < 0.37, below 2^-21 m; all
// shares of a row by the same factor, their sum's (36 additions on the way), within 2^-18. So two
// keys tell their order if they are further apart than cut + 2^-21, or cut + 2^-17 m. Without a
// bias, where shares may be small, a score is good to 2^-16.8 of itself (arguments up to 68), two
// are told apart by 2^-15, and none is trusted below 2^-40 m.
//
// A group's sum with a bias is off by the roundings of its two keys, 2^-24 of each key's own size, and by its
// own, 2^-24 of itself: the keys may be of different signs, and their sum far smaller than what it is off
// by. So each group has an interval of 2^-22 of its keys' sizes together to either side (2^-23, and 2^-24
// where its end is computed), and the kept groups tell if all of theirs lie above all of the others'. Beside that
// 2^-21 to either side for two sigmoids, 2^-17 m for two shares (of two groups' difference, at most 2 m, their
// common factor is 2^-17 m off and the four shares 2^-21 m each).
template <int kPer, bool kScored, bool kSigmoid>
__global__ void __launch_bounds__(256) route_rows_kernel(RouteProblem p, int per, bool whole) {
  constexpr uint32_t kPlace = kPer - 1;
  __shared__ uint64_t keys[4][16 * kPer];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * 16 + 4 * wave, t = t0 + (lane >> 4);
  if (t0 >= p.T) return;
  const bool there = t < p.T;
  const int e0 = r * per, mine = max(min(per, p.E - e0), 0);
  const float* row = p.logits + min(t, p.T - 1) * p.E;
  // this lane's experts of a row of E values (past the last of them: others); whole: they come in fours
  auto load = [&](float (&v)[kPer], const float* from) {
    if (whole) {
#pragma unroll
      for (int c = 0; c < kPer; c += 4) {
        const floatx4 f = *(const floatx4*)(from + (c < mine ? e0 + c : 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c + i] = f[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = from[i < mine ? e0 + i : 0];
    }
  };
  float l[kPer], bias[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) bias[i] = 0.0f;
  if (kScored && p.bias) load(bias, p.bias);
  load(l, row);
#pragma unroll
  for (int i = 0; i < kPer; ++i) l[i] = i < mine ? l[i] : -__builtin_inff();
  typedef Key32<kPlace> Key;
  bool unsure = false;  // of this lane's row
  float top = l[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) top = __builtin_fmaxf(top, l[i]);
  top = row_maxf(top);
  uint32_t key[kPer];
  float most = 0.0f;  // the row's largest score
  if constexpr (kScored) {
    constexpr float kLog2e = 1.44269504f;
    float s[kPer];
    if (kSigmoid) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l[i]));
      most = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * top));
      unsure = top < -40.0f && top > -__builtin_inff();
    } else {
      const float from = top == -__builtin_inff() ? 0.0f : top;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += s[i] = __builtin_amdgcn_exp2f(kLog2e * (l[i] - from));
      most = __builtin_amdgcn_rcpf(row_sumf(sum));
#pragma unroll
      for (int i = 0; i < kPer; ++i) s[i] *= most;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      key[i] = Key::whole(l[i] == -__builtin_inff() ? -__builtin_inff() : s[i] + bias[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = Key::whole(l[i]);
  }
  uint32_t best = key[0], second = 0u;
#pragma unroll
  for (int i = 1; i < kPer; ++i) {
    if (kScored) second = max(second, min(best, key[i]));
    best = max(best, key[i]);
  }
  unsure = unsure || best >= Key::kOdd;  // NaN and +inf go the other way
  // whether a and b, sums of n keys off by `cut` of their value each, may be in another order than theirs
  auto near = [&](float a, float b, float n, float cut) {
    cut *= __builtin_fmaxf(__builtin_fabsf(a), __builtin_fabsf(b));
    if (p.bias) return !(__builtin_fabsf(a - b) > n * (cut + (kSigmoid ? 0x1p-21f : 0x1p-17f * most)));
    return !(__builtin_fabsf(a - b) > n * (cut + 0x1p-15f * a)) || a < 0x1p-40f * most;
  };
  bool open = true;  // this lane's group
  if (p.top_groups < p.groups) {
    const int lanes = 16 / p.groups, group = r / lanes;
    auto merge = [&](uint32_t b, uint32_t s) {
      second = max(max(second, s), min(best, b));
      best = max(best, b);
    };
    if (lanes > 1) merge(row_lane<0xB1>(best), row_lane<0xB1>(second));    // quad_perm [1, 0, 3, 2]
    if (lanes > 2) merge(row_lane<0x4E>(best), row_lane<0x4E>(second));    // quad_perm [2, 3, 0, 1]
    if (lanes > 4) merge(row_lane<0x141>(best), row_lane<0x141>(second));  // row_half_mirror
    if (lanes > 8) merge(row_lane<0x140>(best), row_lane<0x140>(second));  // row_mirror
    const bool some = best > kPlace;
    float score = some ? Key::value(best) : -__builtin_inff(), size = some ? __builtin_fabsf(score) : 0.0f;
    if (kScored && p.group_best == 2 && second > kPlace) {
      score += Key::value(second);
      size += __builtin_fabsf(Key::value(second));
    }
    // a sum beyond what 32 bits hold is not nothing, and may be in another order than others of its like
    unsure = unsure || size == __builtin_inff();
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
      const float o = __shfl(score, (lane & 48) + g * lanes, 64);
      before += o > score || (o == score && g < group);
    }
    open = before < p.top_groups;
    // the worst that stays against the best that does not, where there are such
    const float off = kScored && p.bias ? 0x1p-22f * size + (kSigmoid ? 0x1p-21f : 0x1p-17f * most) : 0.0f;
    const float in = -row_maxf(open ? off - score : -__builtin_inff()), out = row_maxf(open ? -__builtin_inff() : score + off);
    if (kScored && out > -__builtin_inff()) unsure = unsure || (p.bias ? !(in > out) : near(in, out, 2.0f, 0x1p-22f));
  }
  // v = before - 1 - key of each round; a lane whose group is out has nothing
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = open ? ~Key::cut(key[i], kPlace - i) : 0xFFFFFFFFu;
  // A round's key and the lanes that have it: lane j keeps the j-th choice's, all lanes those of the
  // first that is not one.
  uint32_t before = 0u;  // (its first "less 1" is the largest number)
  struct Round {
    uint32_t taken, at;  // 0: nothing was left
  };
  auto round = [&](bool first) {
    uint32_t v = key[0] + before;
#pragma unroll
    for (int i = 1; i < kPer; ++i) v = min(v, key[i] + before);
    const uint32_t least = row_min(v), taken = before - 1u - least;
    const uint32_t at = (uint32_t)(__ballot(v == least) >> (lane & 48)) & 0xFFFFu;
    const bool some = taken > kPlace && (first || least < before);  // (else wrapped around)
    before = some ? taken : 1u;  // (below 1 there is nothing)
    return some ? Round{taken, at} : Round{0u, 0u};
  };
  auto expert_of = [&](const Round& k) {
    return k.at == 0u ? -1 : __builtin_ctz(k.at) * per + (int)(kPlace - (k.taken & kPlace));
  };
  auto near_keys = [&](uint32_t a, uint32_t b) {  // neither is nothing
    return kScored ? near(Key::value(a), Key::value(b), 1.0f, (float)kPer * 0x1p-22f) : ((a ^ b) & ~kPlace) == 0u;
  };
  Round choice = {0u, 0u}, after = {0u, 0u};
  for (int j = 0; j < p.top_k; ++j) {
    const Round k = round(j == 0);
    if (r == j) choice = k;
  }
  after = round(false);
  int id = expert_of(choice);
  const int next = expert_of(after);
  unsure = unsure || (choice.at & (choice.at - 1u)) != 0u || (after.at & (after.at - 1u)) != 0u;
  // Where neighbours among them are near, the formula's own keys of these tell: the logits, or in 64
  // bits a sigmoid and its bias. (Those of a softmax with a bias take a sum over all experts.)
  const uint32_t right = row_lane<0x101>(choice.taken);  // row_shl 1: the next lane's (read with every lane there)
  const uint32_t behind = r == p.top_k - 1 ? after.taken : right;
  const bool lane_close = choice.taken != 0u && behind != 0u && near_keys(choice.taken, behind);
  const uint32_t close_lanes = (uint32_t)(__ballot(lane_close) >> (lane & 48)) & 0xFFFFu;
  const bool close = close_lanes != 0u, edge = (close_lanes >> (p.top_k - 1)) & 1u;
  if (__ballot(close) != 0) {
    if (kScored && !kSigmoid && p.bias) {
      unsure = unsure || close;
    } else {
      // the one after the next one has to be far from it
      const Round third = round(false);
      if (edge && third.taken != 0u) unsure = unsure || near_keys(after.taken, third.taken);
      auto exact = [&](int e) {
        if (e < 0) return -(double)__builtin_inff();
        return p.bias ? sigmoid((double)row[e], 0.0) + (double)p.bias[e] : (double)row[e];
      };
      const double mine64 = exact(id), next64 = exact(next);
      int rank = 0;
      for (int j = 0; j < p.top_k; ++j) {
        const int o = __shfl(id, (lane & 48) + j, 64);
        const double o64 = __shfl(mine64, (lane & 48) + j, 64);
        rank += o64 > mine64 || (o64 == mine64 && o < id);
      }
      // the next one pushes the last out if it comes before it
      rank += next >= 0 && (next64 > mine64 || (next64 == mine64 && next < id));
      int next_rank = 0;
      for (int j = 0; j < p.top_k; ++j) {
        const int o = __shfl(id, (lane & 48) + j, 64);
        const double o64 = __shfl(mine64, (lane & 48) + j, 64);
        next_rank += o64 > next64 || (o64 == next64 && o < next);
      }
      if (id < 0) rank = kRouteTopK;
      int sorted = -1;
      for (int j = 0; j < p.top_k; ++j) {
        const int o = __shfl(id, (lane & 48) + j, 64), k = __shfl(rank, (lane & 48) + j, 64);
        if (k == r) sorted = o;
      }
      if (next >= 0 && next_rank == r) sorted = next;
      if (close) id = r < p.top_k ? sorted : -1;
    }
  }
  double sum = 0.0;
  if (!kSigmoid && !p.renormalize) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (l[i] != -__builtin_inff()) sum += exp((double)l[i] - (double)top);
    sum = row_sum_f64(sum);
  }
  const uint64_t again = __ballot(unsure && there);
  const bool sure = ((again >> (lane & 48)) & 0xFFFFull) == 0;
  // (a row that is not sure computes what it does not store)
  store_choice<kSigmoid>(p, t, sure && there ? r : kRouteTopK, id, id >= 0 ? row[id] : 0.0f, top, sum);
  for (int g = 0; g < 4; ++g)
    if ((again >> (16 * g)) & 0xFFFFull) route_exact<kPer / 4>(p, t0 + g, lane, keys[wave]);
}

}  // namespace

// Sixteen lanes take a token wherever a group of experts is whole lanes of them.
bool route_by_rows(const RouteProblem& p) {
  return p.top_groups >= p.groups || (p.groups <= 16 && 16 % p.groups == 0 && p.E % 16 == 0);
}

template <int kPer, bool kScored>
void launch_rows(const RouteProblem& p, int per, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 15) / 16)), block(256);
  const bool whole = per % 4 == 0 && p.E % 4 == 0 && (uintptr_t)p.logits % 16 == 0 && (uintptr_t)p.bias % 16 == 0;
  if (p.sigmoid) hipLaunchKernelGGL((route_rows_kernel<kPer, kScored, true>), grid, block, 0, stream, p, per, whole);
  else hipLaunchKernelGGL((route_rows_kernel<kPer, kScored, false>), grid, block, 0, stream, p, per, whole);
}
template <int kPer>
void launch_rows(const RouteProblem& p, int per, hipStream_t stream) {
  if (p.bias || (p.top_groups < p.groups && p.group_best == 2)) launch_rows<kPer, true>(p, per, stream);
  else launch_rows<kPer, false>(p, per, stream);
}

hipError_t launch_moe_route(const RouteProblem& p, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  if (route_by_rows(p)) {
    // (without groups, fours wherever they fit)
    const int least = (p.E + 15) / 16, per = p.top_groups < p.groups ? least : (least + 3) / 4 * 4;
    if (per <= 4) launch_rows<4>(p, per, stream);
    else if (per <= 8) launch_rows<8>(p, per, stream);
    else if (per <= 16) launch_rows<16>(p, per, stream);
    else launch_rows<32>(p, per, stream);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((p.T + 3) / 4)), block(256);
  if (p.E <= 64) hipLaunchKernelGGL(route_exact_kernel<1>, grid, block, 0, stream, p);
  else if (p.E <= 128) hipLaunchKernelGGL(route_exact_kernel<2>, grid, block, 0, stream, p);
  else if (p.E <= 256) hipLaunchKernelGGL(route_exact_kernel<4>, grid, block, 0, stream, p);
  else hipLaunchKernelGGL(route_exact_kernel<8>, grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
