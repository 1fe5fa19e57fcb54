// A mixture-of-experts layer for a few tokens on gfx950, with MXFP4 expert weights and bf16
// activations: the router's product, and the routed experts' gated feed-forward.
//
// For token t with logits l_t over E experts: the top_k experts of largest logit (ties to
// the lowest index) with softmax weights g, taken over all E or over the chosen ones; then
//   h_tj = silu(Wg_e x_t) * (Wu_e x_t),  e = the j-th chosen expert, silu(z) = z / (1 + exp(-z))
//   out_t = sum_j g_tj (W2_e h_tj).
// W13 holds the gate rows Wg and then the up rows Wu of each expert, [E, 2I, H]; W2 is
// [E, H, I]; both MXFP4 along their last axis.
#include <type_traits>

#include "gemm_common.hpp"
#include "moe_offsets.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kMoeTokens = 64;   // tokens planned together
constexpr int kMoeExperts = (int)kMoeMaxExperts;
constexpr int kMoeTopK = (int)kMoeMaxTopK;
constexpr int kMoeSlots = kMoeTokens * kMoeTopK;

// ---- the router's product --------------------------------------------------------------
//
// logits[t, e] = sum_h x[t, h] w[e, h], summed in fp64 (products of bf16 values are exact
// there) and rounded once to fp32: two experts whose logits differ by more than that rounding
// are never exchanged by the order of the summation. A wave takes kE experts and kT tokens,
// its lanes eight elements of H each in turn; every element is converted once per wave.
template <int kE, int kT>
__global__ void __launch_bounds__(256) moe_router_kernel(const u32x4* __restrict__ x,
                                                         const u32x4* __restrict__ w,
                                                         float* __restrict__ logits, int64_t T,
                                                         int64_t E, int64_t H8) {
  const int lane = threadIdx.x & 63;
  const int64_t e0 = ((int64_t)blockIdx.y * 4 + (threadIdx.x >> 6)) * kE;
  const int64_t t0 = (int64_t)blockIdx.x * kT;
  if (e0 >= E) return;
  double acc[kE][kT] = {};
  u32x4 wv[kE], xv[kT], wn[kE], xn[kT];  // this turn's, and the next one's in flight
  auto load = [&](u32x4 (&a)[kE], u32x4 (&b)[kT], int64_t i) {
#pragma unroll
    for (int e = 0; e < kE; ++e) a[e] = w[min(e0 + e, E - 1) * H8 + i];
#pragma unroll
    for (int t = 0; t < kT; ++t) b[t] = x[min(t0 + t, T - 1) * H8 + i];
  };
  if (lane < H8) load(wv, xv, lane);
  for (int64_t i = lane; i < H8; i += 64) {
    load(wn, xn, min(i + 64, H8 - 1));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      auto element = [&](const u32x4& v) {
        const uint32_t word = v[j >> 1];
        return (double)u2f(j & 1 ? word & 0xFFFF0000u : word << 16);
      };
      double wd[kE];
#pragma unroll
      for (int e = 0; e < kE; ++e) wd[e] = element(wv[e]);
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const double xd = element(xv[t]);
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e][t] = __builtin_fma(xd, wd[e], acc[e][t]);
      }
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) wv[e] = wn[e];
#pragma unroll
    for (int t = 0; t < kT; ++t) xv[t] = xn[t];
  }
#pragma unroll
  for (int e = 0; e < kE; ++e)
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      double v = acc[e][t];
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
      if (lane == 0 && t0 + t < T && e0 + e < E) logits[(t0 + t) * E + e0 + e] = (float)v;
    }
}

// ---- the plan: who goes where ------------------------------------------------------------
//
// Tokens are planned in chunks of 64. A chunk's plan lists the experts that any of its
// tokens reached and, for each, its slots (slot = token-within-chunk * top_k + j).
struct MoePlan {
  int active;                      // experts reached
  int expert[kMoeExperts];         // their indices, increasing
  int first[kMoeExperts + 1];      // their first entry in slot[]
  int tile[kMoeExperts];           // and their first tile of h
  int slot[kMoeSlots];
};

// h, between the two products, is held in two bf16 parts that add up to it within 2^-16 of its
// value, far below the rounding of the layer's output: the matrix instruction takes bf16, and h
// rounded to it once was as much of the layer's error as the output's own rounding (relative to
// 64 bits 2.3e-3 against 1.65e-3). The two parts are two columns of the instruction: a tile is
// 8 slots of one expert, column 2n the n-th one's upper parts, 2n + 1 the lower, in the order in
// which the second product's lanes take it, [tile][16-byte chunk of I][column][16 bytes], so that
// a load reads the columns' chunks side by side. (With a row per slot its loads, an access for
// every lane, bounded that product: 64 tokens 81 us against 75.)
__device__ __forceinline__ uint8_t* h_tiles(const MoeProblem& p) {
  const int64_t tokens = min(p.T, (int64_t)kMoeTokens);
  return (uint8_t*)p.h + (int64_t)blockIdx.z * moe_tiles(tokens * p.top_k, p.E) * (32 * p.I);
}

// Order of two logits as an unsigned key: increasing with the value, NaN above +inf, and
// -inf at 0 (never chosen). key_logit is its inverse.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = f2u(l + 0.0f);  // -0 counts as 0
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if (b == 0xFF800000u) return 0u;
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) { return u2f((k >> 31) ? k ^ 0x80000000u : ~k); }

// The top_k of one token by one wave. Lane l holds experts l, l + 64, ... in kPer registers; each
// round takes the largest key, the lowest index among equals. A row of fewer than top_k experts
// that can be chosen ends in slots of id -1 and weight 0. Lane j < top_k returns the j-th choice.
struct Choice {
  int id;
  float weight;
};
template <int kPer>
__device__ __forceinline__ Choice moe_topk_of(const float* __restrict__ row, int E, int top_k, bool renormalize,
                                              int lane) {
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 64 * i < E ? logit_key(row[lane + 64 * i]) : 0u;
  Choice mine = {-1, 0.0f};
  float top = 0.0f, sum = 0.0f;
  for (int j = 0; j < top_k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = max(best, key[i]);
    const uint32_t k = wave_max_u32(best);
    if (k == 0u) break;  // nothing left to choose
    if (j == 0) {
      top = key_logit(k);
      if (!renormalize) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (key[i] != 0u) s += expf(key_logit(key[i]) - top);
        sum = wave_sum(s);
      }
    }
    int e = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e < 0) {
        const uint64_t at = __ballot(key[i] == k);
        if (at != 0) {
          const int first = __builtin_ctzll(at);
          e = 64 * i + first;
          if (lane == first) key[i] = 0u;
        }
      }
    if (lane == j) mine = Choice{e, key_logit(k)};
  }
  // the choices' exponentials at once, in the lanes that hold them
  mine.weight = mine.id < 0 ? 0.0f : expf(mine.weight - top);
  if (renormalize) sum = wave_sum(mine.weight);
  if (mine.id >= 0) mine.weight /= sum;
  return mine;
}
__device__ __forceinline__ Choice moe_topk(const float* __restrict__ row, int E, int top_k, bool renormalize,
                                           int lane) {
  static_assert(kMoeExperts <= 512, "eight registers of 64 experts");
  if (E <= 64) return moe_topk_of<1>(row, E, top_k, renormalize, lane);
  if (E <= 128) return moe_topk_of<2>(row, E, top_k, renormalize, lane);
  return moe_topk_of<8>(row, E, top_k, renormalize, lane);
}
// The choices of a token whose routing the caller gives, likewise. An index that is no expert's is
// none. One that the token has already is taken into its first slot, with its weight: an
// expert's slots are of different tokens (which is what bounds them).
__device__ __forceinline__ Choice moe_given(const MoeProblem& p, int64_t t, int lane) {
  Choice mine = {-1, 0.0f};
  if (lane < p.top_k) mine = Choice{p.given_ids[t * p.top_k + lane], p.given_weights[t * p.top_k + lane]};
  if (mine.id < 0 || mine.id >= p.E) mine = Choice{-1, 0.0f};
  bool repeated = false;
  float sum = mine.weight;
  for (int j = 0; j < p.top_k; ++j) {
    const int id = __builtin_amdgcn_readlane(mine.id, j);
    const float weight = u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(mine.weight), j));
    if (id != mine.id || id < 0) continue;
    if (j < lane) repeated = true;
    if (j > lane) sum += weight;
  }
  return repeated ? Choice{-1, 0.0f} : Choice{mine.id, sum};
}

// Who routes the tokens of a kernel: the plan that is made already, the kernel itself, the caller.
enum class Routing { kPlanned, kOwn, kGiven };
template <Routing kRouting>
__device__ __forceinline__ Choice choices_of(const MoeProblem& p, int64_t t, int lane) {
  if constexpr (kRouting == Routing::kGiven) return moe_given(p, t, lane);
  else return moe_topk(p.logits + t * p.E, p.E, p.top_k, p.renormalize, lane);
}
template <Routing kRouting>
__device__ __forceinline__ void route_token(const MoeProblem& p, int64_t t, int lane, int* chosen) {
  const Choice c = choices_of<kRouting>(p, t, lane);
  if (lane < p.top_k) {
    if (chosen) chosen[lane] = c.id;
    p.ids[t * p.top_k + lane] = c.id;
    p.weights[t * p.top_k + lane] = c.weight;
  }
}

// The routing of many tokens, a token per wave, over the whole chip: in the plan's one workgroup
// the selection is bound by its instructions (a layer of 64 tokens, 8 of 128 experts, 182 us
// against 178; 8 of 256 experts 84 against 73; up to 32 tokens and for few experts alike).
__global__ void __launch_bounds__(256) moe_route_kernel(MoeProblem p) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t < p.T) route_token<Routing::kOwn>(p, t, threadIdx.x & 63, nullptr);
}

// One workgroup per chunk. kOwn: it routes the tokens itself, one per wave (at most 16); kGiven: it
// takes the caller's routing, up to four tokens per wave.
template <Routing kRouting>
__global__ void __launch_bounds__(1024) moe_plan_kernel(MoeProblem p) {
  __shared__ int count[kMoeExperts];
  __shared__ int place[kMoeExperts];
  __shared__ int chosen[kMoeSlots];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kMoeTokens;
  const int nt = (int)min(p.T - t0, (int64_t)kMoeTokens);
  const int n = nt * p.top_k;
  MoePlan* plan = (MoePlan*)p.plan + blockIdx.x;
  for (int e = threadIdx.x; e < p.E; e += 1024) count[e] = 0;
  if constexpr (kRouting == Routing::kOwn) {
    if (wave < nt) route_token<kRouting>(p, t0 + wave, lane, chosen + wave * p.top_k);
  } else if constexpr (kRouting == Routing::kGiven) {
    for (int t = wave; t < nt; t += 16) route_token<kRouting>(p, t0 + t, lane, chosen + t * p.top_k);
  } else {
    for (int i = threadIdx.x; i < n; i += 1024) chosen[i] = p.ids[t0 * p.top_k + i];
  }
  __syncthreads();
  const int s = threadIdx.x;  // n <= 1024
  const int e = s < n ? chosen[s] : -1;
  if (e >= 0) atomicAdd(&count[e], 1);
  __syncthreads();
  if (wave == 0) {
    int active = 0, first = 0, tile = 0;
    for (int b = 0; b < p.E; b += 64) {
      const int c = b + lane < p.E ? count[b + lane] : 0;
      const uint64_t on = __ballot(c > 0);
      const int rank = active + __popcll(on & ((1ull << lane) - 1ull));
      int sum = c;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(sum, off, 64);
        if (lane >= off) sum += o;
      }
      const int ct = (c + kTileSlots - 1) / kTileSlots;
      int tiles = ct;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(tiles, off, 64);
        if (lane >= off) tiles += o;
      }
      if (b + lane < p.E) place[b + lane] = first + sum - c;
      if (c > 0) {
        plan->expert[rank] = b + lane;
        plan->first[rank] = first + sum - c;
        plan->tile[rank] = tile + tiles - ct;
      }
      active += __popcll(on);
      first += __shfl(sum, 63, 64);
      tile += __shfl(tiles, 63, 64);
    }
    if (lane == 0) {
      plan->active = active;
      plan->first[active] = first;
    }
  }
  __syncthreads();
  // the order of an expert's slots does not enter any result: each slot is its own column
  if (e >= 0) plan->slot[atomicAdd(&place[e], 1)] = s;
}

// ---- the experts' products --------------------------------------------------------------
//
// v_mfma_f32_16x16x32_bf16 with 16 weight rows as its A operand and 16 slots as columns. K
// goes by units of 512 elements (16 blocks). In the matrix instruction a lane (q, r) =
// (lane / 16, lane % 16) stands for row r, so that neighbouring lanes are different rows; a
// load made in that order takes a cache access for every lane (measured: it bounded these
// kernels, not memory). So the weights are loaded in the order of memory, four lanes to the 64
// bytes of blocks 4g .. 4g + 3 of a row, and handed over to lane (q, r), which gets block 4g + q
// of row r, by lane permutes through the LDS crossbar. Its four dwords go into four MFMAs,
// eight elements each; the activations follow the same order of K. The scaled conversion to
// bf16 gives a weight's value exactly.
struct WeightUnit {  // as loaded
  u32x4 codes[4];
  uint32_t scales;
};

// Where 16 rows start (the same for the whole wave), and this lane's share of them.
struct WeightRows {
  const uint8_t *codes, *scales;
};
struct WeightLane {
  uint32_t codes, scales;
  __device__ __forceinline__ WeightLane(int nb, int lane)
      : codes(weight_code_at(lane, nb)), scales(weight_scale_at(lane, nb)) {}
};
__device__ __forceinline__ void load_unit(WeightUnit& w, const WeightRows& rows, const WeightLane& at, int u,
                                          int nb, int lane) {
  const int b0 = unit_start(u, nb);
  const uint8_t* codes = rows.codes + 16 * (int64_t)b0;
  const uint8_t* scales = rows.scales + b0;
  if (nb >= kUnit) {
#pragma unroll
    for (int g = 0; g < 4; ++g) w.codes[g] = *(const u32x4*)&codes[at.codes + 64u * (uint32_t)g];
    __builtin_memcpy(&w.scales, &scales[at.scales], 4);  // at any alignment
  } else {
    w.scales = 0u;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      w.codes[g] = *(const u32x4*)&codes[short_code_at(lane, g, nb)];
      w.scales |= (uint32_t)scales[short_scale_at(lane, g, nb)] << (8 * g);
    }
  }
}
// Codes and scale bytes of blocks that are not unit u's (unit_cut): zero.
__device__ __forceinline__ void clear_unit(WeightUnit& w, int u, int nb, int lane) {
  const int b0 = unit_start(u, nb), part = lane & 3;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    if (!unit_has(u, b0 + 4 * g + part, nb)) w.codes[g] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!unit_has(u, b0 + 4 * part + i, nb)) w.scales &= ~(0xFFu << (8 * i));
}

// A unit's activations of 16 columns: lane (q, r) holds, of column r, elements 8j .. 8j + 7 of
// block 4g + q in x[4 g + j]. load_acts: the column starts at byte `at` of the window and its
// 16-byte chunks are `stride` bytes apart. What a short row has no blocks for is read from
// beyond it (zeros past the window) and cleared. Lanes of columns that are not there (`have`
// false) load nothing: a column's results depend on its own activations alone.
struct ActUnit {
  u32x4 x[kUnit];
};
template <int kStride>
__device__ __forceinline__ void load_acts(ActUnit& a, __amdgpu_buffer_rsrc_t window, bool have, uint32_t at,
                                          int u, int nb, int q) {
  if (!have) return;
  at += act_first(kStride, u, nb, q);
#pragma unroll
  for (int i = 0; i < kUnit; ++i)
    a.x[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
        window, (int)(at + act_step(kStride, i)), 0, 0));
}
__device__ __forceinline__ void clear_acts(ActUnit& a, int u, int nb, int q) {
  const int b0 = unit_start(u, nb);
#pragma unroll
  for (int i = 0; i < kUnit; ++i)
    if (!unit_has(u, b0 + 4 * (i >> 2) + q, nb)) a.x[i] = u32x4{0u, 0u, 0u, 0u};
}

__device__ __forceinline__ uint32_t from_lane(int lane, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * lane, (int)v);
}

// Eight codes under a scale, as bf16.
__device__ __forceinline__ bf16x8_t decode8_bf16(uint32_t c, float sc) {
  const u32x4 o = {
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3))};
  return __builtin_bit_cast(bf16x8_t, o);
}

// acc[f][t] += the unit of weights w[f] times tile t's activations: fetch(i, t) gives entry i of
// an ActUnit of this lane's column.
template <int kF, int kT, typename Fetch>
__device__ __forceinline__ void multiply_unit(floatx4 (&acc)[kF][kT], const WeightUnit (&w)[kF], int lane,
                                              const Fetch& fetch) {
  const int q = lane >> 4, r = lane & 15;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    u32x4 x[4][kT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < kT; ++t) x[j][t] = fetch(4 * g + j, t);
    uint32_t c[kF][4];
    float sc[kF];
#pragma unroll
    for (int f = 0; f < kF; ++f) {
      const uint32_t bytes = from_lane(4 * r + g, w[f].scales);
      sc[f] = u2f(((bytes >> (8 * q)) & 0xFFu) << 23);
      const uint32_t c0 = w[f].codes[g].x, c1 = w[f].codes[g].y, c2 = w[f].codes[g].z, c3 = w[f].codes[g].w;
      c[f][0] = from_lane(4 * r + q, c0);
      c[f][1] = from_lane(4 * r + q, c1);
      c[f][2] = from_lane(4 * r + q, c2);
      c[f][3] = from_lane(4 * r + q, c3);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int f = 0; f < kF; ++f) {
        const bf16x8_t wv = decode8_bf16(c[f][j], sc[f]);
#pragma unroll
        for (int t = 0; t < kT; ++t)
          acc[f][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8_t, x[j][t]),
                                                              acc[f][t], 0, 0, 0);
      }
    }
    // (without a fence the decodes of all groups are moved ahead of the MFMAs, into registers
    // that are not there)
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The same in two steps, for several tiles in turn: the unit decoded, then each tile's products.
struct DecodedUnit {
  bf16x8_t w[kUnit];
};
__device__ __forceinline__ void decode_unit(DecodedUnit& d, const WeightUnit& w, int lane) {
  const int q = lane >> 4, r = lane & 15;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t bytes = from_lane(4 * r + g, w.scales);
    const float sc = u2f(((bytes >> (8 * q)) & 0xFFu) << 23);
    const uint32_t c0 = w.codes[g].x, c1 = w.codes[g].y, c2 = w.codes[g].z, c3 = w.codes[g].w;
    d.w[4 * g] = decode8_bf16(from_lane(4 * r + q, c0), sc);
    d.w[4 * g + 1] = decode8_bf16(from_lane(4 * r + q, c1), sc);
    d.w[4 * g + 2] = decode8_bf16(from_lane(4 * r + q, c2), sc);
    d.w[4 * g + 3] = decode8_bf16(from_lane(4 * r + q, c3), sc);
  }
}
template <typename Fetch>
__device__ __forceinline__ void multiply_decoded(floatx4& acc, const DecodedUnit& d, const Fetch& fetch) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(d.w[i], __builtin_bit_cast(bf16x8_t, fetch(i)), acc, 0, 0, 0);
}

constexpr int kTiles = kMoeTokens / 16;
constexpr int kGateWaves = 4;

// One expert's part of a launch.
struct ExpertSlots {
  int64_t expert;
  const int* slots;
  int n;
  uint8_t* h;  // its first tile
};
__device__ __forceinline__ bool expert_slots(const MoeProblem& p, ExpertSlots& s) {
  const MoePlan* plan = (const MoePlan*)p.plan + blockIdx.z;
  const int a = blockIdx.y;
  s.expert = __builtin_amdgcn_readfirstlane(plan->expert[a]);  // (of no meaning past the active ones, but in the buffer)
  s.slots = plan->slot + plan->first[a];
  s.n = plan->first[a + 1] - plan->first[a];
  s.h = h_tiles(p) + (int64_t)plan->tile[a] * (32 * p.I);
  return a < plan->active;
}

// The same without a plan made before, for one to four tokens: every workgroup routes all of
// them, a token per wave, and orders their at most 64 slots in a wave's lanes; the first one
// writes the plan for the second product. (One token: a launch and its 5 us less, for 2 us
// in each workgroup.) With so few tokens an expert has one tile of h.
constexpr int kInlineTokens = 4;
static_assert(kInlineTokens * kMoeTopK <= 64 && kInlineTokens <= kGateWaves, "a slot per lane, a token per wave");
static_assert(kInlineTokens <= kTileSlots, "a tile per expert");
struct InlinePlan {
  int id[64];
  float weight[64];
  int slot[kInlineTokens];
};
template <Routing kRouting>
__device__ __forceinline__ bool expert_slots(const MoeProblem& p, ExpertSlots& s, InlinePlan& ip, int wave,
                                             int lane) {
  const int T = (int)p.T, n = T * p.top_k;
  if (wave < T) {
    const Choice c = choices_of<kRouting>(p, wave, lane);
    if (lane < p.top_k) {
      ip.id[wave * p.top_k + lane] = c.id;
      ip.weight[wave * p.top_k + lane] = c.weight;
    }
  }
  __syncthreads();
  const int id = lane < n ? ip.id[lane] : -1;
  // of this lane's expert: its slots before this one; in all, slots and experts of lower index
  int before = 0, slots_below = 0, experts_below = 0;
  uint64_t firsts = 0;  // lanes that are their expert's first slot
  for (int i = 0; i < n; ++i) {
    const int o = __builtin_amdgcn_readlane(id, i);
    if (o < 0) continue;
    before += o == id && i < lane;
    slots_below += o < id;
  }
  firsts = __ballot(id >= 0 && before == 0);
  for (uint64_t f = firsts; f != 0; f &= f - 1) experts_below += __builtin_amdgcn_readlane(id, __builtin_ctzll(f)) < id;
  const int active = __popcll(firsts), a = blockIdx.y;
  if (blockIdx.x == 0 && a == 0 && wave == 0) {
    MoePlan* plan = (MoePlan*)p.plan;
    if (lane < n) {
      p.ids[lane] = id;
      p.weights[lane] = ip.weight[lane];
    }
    if (id >= 0) plan->slot[slots_below + before] = lane;
    if (id >= 0 && before == 0) {
      plan->expert[experts_below] = id;
      plan->first[experts_below] = slots_below;
      plan->tile[experts_below] = experts_below;
    }
    const int chosen = __popcll(__ballot(id >= 0));
    if (lane == 0) {
      plan->active = active;
      plan->first[active] = chosen;
    }
  }
  if (a >= active) return false;
  const uint64_t mine = __ballot(id >= 0 && experts_below == a);
  s.expert = __builtin_amdgcn_readlane(id, __builtin_ctzll(mine));
  s.n = __popcll(mine);
  if (wave == 0 && id >= 0 && experts_below == a) ip.slot[before] = lane;
  __syncthreads();
  s.slots = ip.slot;
  s.h = h_tiles(p) + (int64_t)a * (32 * p.I);
  return true;
}
template <Routing kRouting>
__device__ __forceinline__ bool find_slots(const MoeProblem& p, ExpertSlots& s, int wave, int lane) {
  if constexpr (kRouting != Routing::kPlanned) {
    __shared__ InlinePlan ip;
    return expert_slots<kRouting>(p, s, ip, wave, lane);
  } else {
    return expert_slots(p, s);
  }
}

// 16 gate rows from row i of an expert on, and their up rows.
struct GateRows {
  WeightRows gate, up;
  __device__ __forceinline__ GateRows(const MoeProblem& p, int64_t expert, int64_t i) {
    const int64_t row = expert * 2 * p.I + i;
    gate = WeightRows{p.w13_packed + row * (p.H >> 1), p.w13_scales + row * (p.H >> 5)};
    up = WeightRows{gate.codes + p.I * (p.H >> 1), gate.scales + p.I * (p.H >> 5)};
  }
  __device__ __forceinline__ void load(WeightUnit (&w)[2], const WeightLane& at, int u, int nb, int lane) const {
    load_unit(w[0], gate, at, u, nb, lane);
    load_unit(w[1], up, at, u, nb, lane);
  }
};

// h = silu(g) * u of four rows, i .. i + 3 (i a multiple of 4), of an expert's n-th slot: the upper half
// of its 32 bits (cut, so that it overflows with h alone) and the rest, rounded. An infinite h has
// no rest; a NaN's may be anything.
__device__ __forceinline__ void store_h(const MoeProblem& p, const ExpertSlots& s, int n, int64_t i,
                                        const floatx4 g, const floatx4 u) {
  uint32_t b[4];
  float rest[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float v = g[j] / (1.0f + expf(-g[j])) * u[j];
    b[j] = f2u(v);
    rest[j] = (b[j] & 0x7FFFFFFFu) == 0x7F800000u ? 0.0f : v - u2f(b[j] & 0xFFFF0000u);
  }
  uint8_t* at = s.h + h_at(n, i, p.I);
  *(u32x2*)at = u32x2{(b[0] >> 16) | (b[1] & 0xFFFF0000u), (b[2] >> 16) | (b[3] & 0xFFFF0000u)};
  *(u32x2*)(at + 16) = bf16x4_rne(rest[0], rest[1], rest[2], rest[3]);
}

// The products of a slot's two parts, added in both lanes (quad_perm [1, 0, 3, 2]).
__device__ __forceinline__ floatx4 add_parts(floatx4 v) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] += u2f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f2u(v[j]), 0xB1, 0xF, 0xF, false));
  return v;
}

// h[slot, i] = silu(gate) * up, few experts reached: 16 gate rows and their up rows per
// workgroup, whose waves take units of K in turn, a unit's weights and activations in flight at
// once, and meet in LDS.
template <Routing kRouting>
__global__ void __launch_bounds__(64 * kGateWaves, 2) moe_gate_up_split_kernel(MoeProblem p) {
  constexpr int NW = kGateWaves;
  __shared__ floatx4 part[NW][2][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ExpertSlots s;
  if (!find_slots<kRouting>(p, s, wave, lane)) return;
  const int q = lane >> 4, r = lane & 15;
  const int64_t i0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.z * kMoeTokens;
  const int nb = (int)(p.H >> 5), nu = (nb + kUnit - 1) / kUnit;
  const GateRows rows(p, s.expert, i0);
  const WeightLane at(nb, lane);
  const int64_t tokens = min(p.T - t0, (int64_t)kMoeTokens);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + t0 * p.H, (uint32_t)(tokens * p.H * 2));
  for (int c0 = 0; c0 < s.n; c0 += 16) {
    const int slot = s.slots[min(c0 + r, s.n - 1)];
    const uint32_t row = (uint32_t)(slot / p.top_k) * (uint32_t)(p.H * 2);
    WeightUnit w[2];
    ActUnit x = {};
    floatx4 acc[2][1];
    acc[0][0] = acc[1][0] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = wave; u < nu; u += NW) {
      rows.load(w, at, u, nb, lane);
      load_acts<16>(x, rx, c0 + r < s.n, row, u, nb, q);
      __builtin_amdgcn_sched_barrier(0);
      if (unit_cut(u, nb)) {
        clear_unit(w[0], u, nb, lane);
        clear_unit(w[1], u, nb, lane);
        clear_acts(x, u, nb, q);
      }
      multiply_unit<2, 1>(acc, w, lane, [&](int i, int) { return x.x[i]; });
    }
    __syncthreads();
    part[wave][0][lane] = acc[0][0];
    part[wave][1][lane] = acc[1][0];
    __syncthreads();
    if (wave == 0 && c0 + r < s.n) {
      floatx4 g = acc[0][0], v = acc[1][0];
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        g += part[w][0][lane];
        v += part[w][1][lane];
      }
      store_h(p, s, c0 + r, i0 + 4 * q, g, v);
    }
  }
}

// The same for many experts: 64 gate rows and their up rows per workgroup, 16 + 16 per wave,
// each wave over the whole of K, with the activations of a unit staged in LDS for all of them
// (direct loads of one slot's 1 KiB per instruction). Chunk c (16 bytes) of row s sits at slot
// c ^ (s % 16), so that the 16 columns of a fragment read are in distinct banks.
// One barrier per unit: behind it the unit is readable, and the buffer of the unit before
// takes the next. kT tiles of 16 slots from slot c0 on; a single buffer is filled between two
// barriers.
template <int kT, int kBufs>
__device__ __forceinline__ void gate_up_tiles(const MoeProblem& p, const ExpertSlots& s, const GateRows& rows,
                                              bool mine, int64_t t0, int64_t i0, int c0, int wave,
                                              int lane, uint8_t* lds) {
  constexpr int kBytes = kT * 16 * 1024;
  const int q = lane >> 4, r = lane & 15;
  const int nb = (int)(p.H >> 5), nu = (nb + kUnit - 1) / kUnit;
  const int64_t tokens = min(p.T - t0, (int64_t)kMoeTokens);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + t0 * p.H, (uint32_t)(tokens * p.H * 2));
  uint32_t row0[kT];  // where the activations of this lane's columns start
#pragma unroll
  for (int t = 0; t < kT; ++t)
    row0[t] = (uint32_t)(s.slots[min(c0 + 16 * t + r, s.n - 1)] / p.top_k) * (uint32_t)(p.H * 2);
  auto stage = [&](int u, int buf) {
    const uint32_t from = stage_soff(u, nb);
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int k = 0; k < 16 / kGateWaves; ++k) {
        const int row = kGateWaves * k + wave;  // of tile t
        if (c0 + 16 * t + row >= s.n) continue;
        const uint32_t start = (uint32_t)__builtin_amdgcn_readlane((int)row0[t], row);
        buffer_load_lds16(rx, lds + buf * kBytes + (16 * t + row) * 1024, stage_voff(start, lane ^ row, u, nb), from);
      }
  };
  const WeightLane at(nb, lane);
  WeightUnit cur[2], nxt[2];
  if (mine) rows.load(cur, at, 0, nb, lane);
  stage(0, 0);
  floatx4 acc[2][kT];
#pragma unroll
  for (int t = 0; t < kT; ++t) acc[0][t] = acc[1][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int u = 0; u < nu; ++u) {
    const int buf = kBufs == 2 ? u & 1 : 0;
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    if (u + 1 < nu) {
      if (mine) rows.load(nxt, at, u + 1, nb, lane);
      if (kBufs == 2) stage(u + 1, buf ^ 1);
    }
    if (mine) {
      if (unit_cut(u, nb)) {
        clear_unit(cur[0], u, nb, lane);
        clear_unit(cur[1], u, nb, lane);
      }
      multiply_unit<2, kT>(acc, cur, lane, [&](int i, int t) {
        const int chunk = 16 * (i >> 2) + 4 * q + (i & 3);  // of block 4 (i / 4) + q, its 16 bytes i % 4
        return *(const u32x4*)&lds[buf * kBytes + (16 * t + r) * 1024 + 16 * (chunk ^ r)];
      });
    }
    if (kBufs == 1 && u + 1 < nu) {
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      stage(u + 1, 0);
    }
    cur[0] = nxt[0];
    cur[1] = nxt[1];
  }
  if (!mine) return;
#pragma unroll
  for (int t = 0; t < kT; ++t)
    if (c0 + 16 * t + r < s.n) store_h(p, s, c0 + 16 * t + r, i0 + 4 * q, acc[0][t], acc[1][t]);
}

// kFew: half the LDS and three workgroups per compute unit, so that more of them start at once.
// For up to 16 tokens (an expert has at most as many slots as there are tokens; 24 layers and
// numbers, two workgroups against three: 2% less on average, from 8% less to 8% more as the last
// workgroups fall), and where a workgroup is short, below 8 units of K, and experts have at most 8
// slots on average (an expert of more than 16 takes them 32 at a time, with registers that spill).
// The layer, two workgroups against three: 64 tokens, 4 of 32 experts, I 1440, with 5, 7, 8 and 8
// units (H 2560, 3584, 3616, 4096) 77 / 71, 95 / 89, 109 / 106, 102 / 98; 8 of 128, I 1024, with 5, 7, 7, 8
// and 8 (2560, 3328, 3584, 3616, 4096) 132 / 132, 166 / 167, 170 / 174, 197 / 206, 187 / 193; 6 of 64, I 1408,
// with 5, 7, 8 and 8 (2560, 3584, 3616, 4064) 113 / 111, 140 / 140, 162 / 168, 174 / 180; and with more slots,
// 2 of 8, 4096 x 4096, 93 / 101, 4 of 64, 4096 x 1024, 105 / 115.
template <Routing kRouting, bool kFew>
__global__ void __launch_bounds__(64 * kGateWaves, kFew ? 3 : 2) moe_gate_up_kernel(MoeProblem p) {
  __shared__ __align__(16) uint8_t lds[(kFew ? 2 : kTiles) * 16 * 1024];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ExpertSlots s;
  if (!find_slots<kRouting>(p, s, wave, lane)) return;
  const int64_t i0 = (int64_t)blockIdx.x * (16 * kGateWaves) + 16 * wave, t0 = (int64_t)blockIdx.z * kMoeTokens;
  const bool mine = i0 < p.I;  // I % 32 == 0: a wave's 16 rows are all there or none
  const GateRows rows(p, s.expert, mine ? i0 : 0);
  if (kRouting != Routing::kPlanned || s.n <= 16) {
    gate_up_tiles<1, 2>(p, s, rows, mine, t0, i0, 0, wave, lane, lds);
  } else if constexpr (kFew) {
    for (int c0 = 0; c0 < s.n; c0 += 32) {
      if (c0 > 0) __syncthreads();
      gate_up_tiles<2, 1>(p, s, rows, mine, t0, i0, c0, wave, lane, lds);
    }
  } else if (s.n <= 32) {
    gate_up_tiles<2, 2>(p, s, rows, mine, t0, i0, 0, wave, lane, lds);
  } else {
    gate_up_tiles<4, 1>(p, s, rows, mine, t0, i0, 0, wave, lane, lds);
  }
}

// out[t, o] for 16 rows of W2 and one to four tokens: the workgroup's waves take (expert, unit of
// K) pairs in turn, a pair's weights and h in flight at once, and add the weighted results to
// their own fp32 sums by token in LDS; the waves' sums are added in a fixed order. (One token,
// 6 of 64 experts, 2048 x 1408: 6.5 us, of which the weights' 9.2 MB are 1.6.)
__global__ void __launch_bounds__(1024) moe_down_kernel(MoeProblem p) {
  constexpr int NW = 16, kSlots = kInlineTokens * kMoeTopK;
  __shared__ floatx4 sums[NW][kInlineTokens][4];
  __shared__ int s_expert[kSlots];
  __shared__ int s_first[kSlots + 1];
  __shared__ int s_slot[kSlots];
  __shared__ float s_weight[kSlots];  // by slot (a load at its use would wait for all loads before it)
  const MoePlan* plan = (const MoePlan*)p.plan;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int64_t o0 = (int64_t)blockIdx.x * 16;
  const int nb = (int)(p.I >> 5), nu = (nb + kUnit - 1) / kUnit;
  const int nt = (int)p.T, n = nt * p.top_k;
  const int active = plan->active;
  // the plan's lists, as long as they can be (past the active experts: of no meaning)
  if (threadIdx.x < n) {
    s_expert[threadIdx.x] = plan->expert[threadIdx.x];
    s_slot[threadIdx.x] = plan->slot[threadIdx.x];
    s_weight[threadIdx.x] = p.weights[threadIdx.x];
  }
  if (threadIdx.x <= n) s_first[threadIdx.x] = plan->first[threadIdx.x];
  for (int i = threadIdx.x; i < NW * nt * 4; i += 64 * NW)
    sums[i / (nt * 4)][i % (nt * 4) >> 2][i & 3] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  const uint8_t* h = h_tiles(p);  // a tile for each expert
  const WeightLane lane_at(nb, lane);
  // pair (a, u): unit u of the a-th expert; a wave's next is NW units on
  struct Pair {
    int a, u;
  };
  auto next = [&](Pair k) {
    k.u += NW;
    while (k.u >= nu) {
      k.u -= nu;
      ++k.a;
    }
    return k;
  };
  WeightUnit w[1];
  ActUnit x = {};
  for (Pair at = next(Pair{0, wave - NW}); at.a < active; at = next(at)) {
    const int s0 = __builtin_amdgcn_readfirstlane(s_first[at.a]);
    const int ns = __builtin_amdgcn_readfirstlane(s_first[at.a + 1]) - s0, u = at.u;
    load_acts<256>(x, make_rsrc(h + (int64_t)at.a * (32 * p.I), (uint32_t)(32 * p.I)), (r >> 1) < ns,
                   16u * (uint32_t)r, u, nb, q);
    const int64_t row = (int64_t)__builtin_amdgcn_readfirstlane(s_expert[at.a]) * p.H + o0;
    load_unit(w[0], WeightRows{p.w2_packed + row * (p.I >> 1), p.w2_scales + row * nb}, lane_at, u, nb, lane);
    __builtin_amdgcn_sched_barrier(0);
    if (unit_cut(u, nb)) {
      clear_unit(w[0], u, nb, lane);
      clear_acts(x, u, nb, q);
    }
    floatx4 acc[1][1];
    acc[0][0] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    multiply_unit<1, 1>(acc, w, lane, [&](int i, int) { return x.x[i]; });
    const floatx4 y = add_parts(acc[0][0]);
    if ((r & 1) == 0 && (r >> 1) < ns) {
      const int slot = s_slot[s0 + (r >> 1)];
      sums[wave][slot / p.top_k][q] += s_weight[slot] * y;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * 4; i += 64 * NW) {
    const int t = i >> 2, o = i & 3;
    floatx4 v = sums[0][t][o];
#pragma unroll
    for (int j = 1; j < NW; ++j) v += sums[j][t][o];
    *(u32x2*)&p.out[t * p.H + o0 + 4 * o] = bf16x4_rne(v[0], v[1], v[2], v[3]);
  }
}

// The same for more tokens: 64 rows of W2 per workgroup, 16 per wave, so that a unit of h, staged
// in LDS, serves four times the weights (with 16 rows the reads of h take the cache as long as
// the weights take memory: 64 tokens, 8 of 128 experts, 4096 x 1024, 75 us). A workgroup takes
// one of `groups` shares of the (expert, unit of K) pairs and writes its fp32 sums by token,
// which moe_combine_kernel adds. Loads run two items ahead, into three sets of registers: with
// one ahead a unit's multiplications were all the time its successor's loads had (74 us; now
// 59, the weights at 4.8 TB/s, and 5 for the sums). An expert of more than 8 slots has several
// tiles of h, multiplied one after the other with a unit that is permuted and decoded once
// (against once a tile, the layer: 64 tokens, 8 of 8 experts, 4096 x 4096, 161 -> 137 us; 2 of 8,
// 4096 x 14336, 266 -> 244), their sums in registers to the expert's end (against adding every unit to
// the tokens' sums: 138 -> 127, 240 -> 228).
constexpr int kSumPitch = 68;  // floats of a token's 64 sums: 16 columns in distinct banks

__global__ void __launch_bounds__(256, 2) moe_down_wide_kernel(MoeProblem p) {
  constexpr int kBytes = kUnit * 1024;
  __shared__ __align__(16) uint8_t lds[3 * kBytes];  // a unit's first tiles in turn, its others
  __shared__ __align__(16) float sums[kMoeTokens * kSumPitch];
  __shared__ int s_expert[kMoeExperts];
  __shared__ int s_first[kMoeExperts + 1];
  __shared__ int s_tile[kMoeExperts];
  __shared__ int s_slot[kMoeSlots];
  __shared__ float s_weight[kMoeSlots];  // by slot (a load at its use would wait for all loads before it)
  const MoePlan* plan = (const MoePlan*)p.plan + blockIdx.z;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  // H % 32 == 0: a wave's 16 rows are all there or none (then it computes the first 16 again)
  const bool mine = (int64_t)blockIdx.x * 64 + 16 * wave < p.H;
  const int64_t o0 = mine ? (int64_t)blockIdx.x * 64 + 16 * wave : 0;
  const int nb = (int)(p.I >> 5), nu = (nb + kUnit - 1) / kUnit;
  const int64_t t0 = (int64_t)blockIdx.z * kMoeTokens;
  const int nt = (int)min(p.T - t0, (int64_t)kMoeTokens);
  const int n = nt * p.top_k, most = min(n, p.E);
  const int active = plan->active;
  for (int i = threadIdx.x; i < most; i += 256) {
    s_expert[i] = plan->expert[i];
    s_tile[i] = plan->tile[i];
  }
  for (int i = threadIdx.x; i <= most; i += 256) s_first[i] = plan->first[i];
  for (int i = threadIdx.x; i < n; i += 256) {
    s_slot[i] = plan->slot[i];
    s_weight[i] = p.weights[t0 * p.top_k + i];
  }
  for (int i = threadIdx.x; i < nt * kSumPitch; i += 256) sums[i] = 0.0f;
  __syncthreads();
  const uint8_t* h = h_tiles(p);
  const WeightLane lane_at(nb, lane);
  // this group's pairs, [begin, end) in the order of (expert, unit)
  const int64_t pairs = (int64_t)active * nu;
  const int begin = (int)(pairs * blockIdx.y / gridDim.y), end = (int)(pairs * (blockIdx.y + 1) / gridDim.y);
  // an item: unit u of expert a, which has so many slots
  struct Item {
    int a, u, slots;
  };
  const int a_end = end > 0 ? (end - 1) / nu : 0, a_begin = begin / nu;
  auto u_end = [&](int a) { return a == a_end ? end - a * nu : nu; };
  auto slots_of = [&](int a) {
    return __builtin_amdgcn_readfirstlane(s_first[a + 1]) - __builtin_amdgcn_readfirstlane(s_first[a]);
  };
  auto next = [&](Item k) {
    if (++k.u < u_end(k.a)) return k;
    k.u = 0;
    if (++k.a <= a_end) k.slots = slots_of(k.a);
    return k;
  };
  // a lane's share of a unit of h's tile c: through registers, for a load that goes to LDS by itself would
  // make every read of LDS wait for all loads in flight
  struct HShare {
    u32x4 v[kUnit / 4];
  };
  auto fetch = [&](HShare& s, const Item& k, int c) {
    const int64_t tile = __builtin_amdgcn_readfirstlane(s_tile[k.a]) + c;
    const __amdgpu_buffer_rsrc_t rh = make_rsrc(h + tile * (32 * p.I), (uint32_t)(32 * p.I));
#pragma unroll
    for (int j = 0; j < kUnit / 4; ++j) {
      const int b = 4 * j + wave;  // 1 KiB: a block's four chunks of 16 columns
      s.v[j] = __builtin_amdgcn_raw_buffer_load_b128(rh, (int)h_voff(lane, c, k.slots, k.u, b, nb), h_soff(k.u, b, nb), 0);
    }
  };
  auto stage = [&](const HShare& s, int buf) {
#pragma unroll
    for (int j = 0; j < kUnit / 4; ++j) *(u32x4*)&lds[buf * kBytes + (4 * j + wave) * 1024 + 16 * lane] = s.v[j];
  };
  auto load = [&](WeightUnit& w, const Item& k) {
    const int64_t row = (int64_t)__builtin_amdgcn_readfirstlane(s_expert[k.a]) * p.H + o0;
    load_unit(w, WeightRows{p.w2_packed + row * (p.I >> 1), p.w2_scales + row * nb}, lane_at, k.u, nb, lane);
  };
  if (begin < end) {
    // turn i multiplies item i, puts h of item i + 1 into LDS and loads item i + 2 (past the last
    // item the present one again), h before the weights, which are not waited for with it. Tiles of
    // h past the item's first go through a buffer of their own against the same weights.
    Item at = {a_begin, begin - a_begin * nu, slots_of(a_begin)}, then = next(at);
    auto there = [&](const Item& k) { return k.a <= a_end ? k : at; };
    WeightUnit w0, w1, w2;
    HShare hs, others;
    fetch(hs, at, 0);
    load(w0, at);
    stage(hs, 0);
    fetch(hs, there(then), 0);
    load(w1, there(then));
    constexpr int kMost = kMoeTokens / kTileSlots;  // an expert's tiles: a token's slots are of different experts
    floatx4 acc[kMost];
#pragma unroll
    for (int c = 0; c < kMost; ++c) acc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    auto meet = [&]() {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    };
    auto h_of = [&](int buf, int i) {
      const int chunk = 16 * (i >> 2) + 4 * q + (i & 3);
      return *(const u32x4*)&lds[buf * kBytes + (chunk * 16 + r) * 16];
    };
    auto add = [&](int c) {  // the item's tile c to its tokens' sums
      const int s0 = __builtin_amdgcn_readfirstlane(s_first[at.a]);
      const floatx4 y = add_parts(acc[c]);
      if ((r & 1) == 0 && kTileSlots * c + (r >> 1) < at.slots) {
        const int slot = s_slot[s0 + kTileSlots * c + (r >> 1)];
        *(floatx4*)&sums[(slot / p.top_k) * kSumPitch + 16 * wave + 4 * q] += s_weight[slot] * y;
      }
      acc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    auto turn = [&](WeightUnit& now, int buf, WeightUnit& fill) {
      meet();  // item i's h is in LDS, and everyone is done with item i - 1's
      const Item after = then.a <= a_end ? next(then) : then;
      const int tiles = (at.slots + kTileSlots - 1) / kTileSlots;
      stage(hs, buf ^ 1);
      if (tiles > 1) fetch(others, at, 1);
      fetch(hs, there(after), 0);
      load(fill, there(after));
      __builtin_amdgcn_sched_barrier(0);
      if (unit_cut(at.u, nb)) clear_unit(now, at.u, nb, lane);
      DecodedUnit d;
      decode_unit(d, now, lane);
      const bool last = at.u + 1 == u_end(at.a);
      multiply_decoded(acc[0], d, [&](int i) { return h_of(buf, i); });
      if (last) add(0);
#pragma unroll
      for (int c = 1; c < kMost; ++c) {
        if (c >= tiles) break;
        if (c > 1) meet();
        stage(others, 2);
        meet();
        if (c + 1 < tiles) fetch(others, at, c + 1);
        multiply_decoded(acc[c], d, [&](int i) { return h_of(2, i); });
        if (last) add(c);
      }
      at = then;
      then = after;
      return at.a <= a_end;
    };
    while (turn(w0, 0, w2) && turn(w1, 1, w0) && turn(w2, 0, w1) &&
           turn(w0, 1, w2) && turn(w1, 0, w0) && turn(w2, 1, w1)) {
    }
  }
  if (!mine) return;
  // a wave's own columns
  for (int i = lane; i < nt * 4; i += 64) {
    const int t = i >> 2, o = i & 3;
    const floatx4 v = *(const floatx4*)&sums[t * kSumPitch + 16 * wave + 4 * o];
    *(floatx4*)&p.partial[(((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * min(p.T, (int64_t)kMoeTokens) + t) * p.H + o0 + 4 * o] = v;
  }
}

// out = the sum of the groups' sums, in their order. (Added by the last share to finish instead, a
// launch less, they cost more: every wave's fence writes the level-2 cache back, and the
// second product took 140 us against 63 + 5 with 64 tokens, 68 against 18 + 5 with 12.)
constexpr int kMostGroups = 16;
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeProblem p, int groups) {
  const int64_t o = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4, t = blockIdx.x;
  if (o >= p.H) return;
  const int64_t tokens = min(p.T, (int64_t)kMoeTokens);
  const float* from = p.partial + (t / kMoeTokens * groups * tokens + t % kMoeTokens) * p.H + o;
  floatx4 part[kMostGroups];  // all in flight at once
#pragma unroll
  for (int g = 0; g < kMostGroups; ++g) part[g] = *(const floatx4*)&from[(int64_t)min(g, groups - 1) * tokens * p.H];
  floatx4 v = part[0];
#pragma unroll
  for (int g = 1; g < kMostGroups; ++g)
    if (g < groups) v += part[g];
  *(u32x2*)&p.out[t * p.H + o] = bf16x4_rne(v[0], v[1], v[2], v[3]);
}

}  // namespace

int64_t moe_plan_bytes(int64_t T) {
  return (T + kMoeTokens - 1) / kMoeTokens * (int64_t)sizeof(MoePlan);
}

int64_t moe_h_bytes(int64_t T, int64_t E, int64_t I, int64_t top_k) {
  const int64_t tokens = T < kMoeTokens ? T : kMoeTokens;
  return (T + kMoeTokens - 1) / kMoeTokens * moe_tiles(tokens * top_k, E) * (32 * I);
}

// Shares of the second product's pairs: two workgroups per compute unit (for an MI355X's 256, since the
// size of the workspace is asked for without a device), at most kMostGroups (16
// against 8: 64 tokens of 256 experts of 1024 x 512 in 73 us against 91; 32: another 3 less there,
// 1 to 2 more elsewhere). 0: the kernel without shares, for up to four tokens (five layers of 16
// to 256 experts, both sides in turn: at 2 and 4 tokens shares are slower in eight of ten, by up
// to 5 us, at 5 and 8 faster in six, by up to 9).
int moe_groups(int64_t T, int64_t H) {
  if (T <= kInlineTokens) return 0;
  const int64_t wide = (H + 63) / 64 * ((T + kMoeTokens - 1) / kMoeTokens), groups = 512 / wide;
  return (int)(groups < 1 ? 1 : groups > kMostGroups ? kMostGroups : groups);
}

int64_t moe_partial_bytes(int64_t T, int64_t H) {
  const int64_t tokens = T < kMoeTokens ? T : kMoeTokens;
  return (T + kMoeTokens - 1) / kMoeTokens * tokens * moe_groups(T, H) * H * 4;
}

hipError_t launch_moe_router(const void* x, const void* w, int64_t T, int64_t E, int64_t H,
                             void* logits, hipStream_t stream) {
  // one or two tokens: an expert per wave, the most waves; more: blocks of 2 experts x 4 tokens
  if (T <= 2) {
    hipLaunchKernelGGL((moe_router_kernel<1, 1>), dim3((unsigned)T, (unsigned)((E + 3) / 4)), dim3(256), 0,
                       stream, (const u32x4*)x, (const u32x4*)w, (float*)logits, T, E, H / 8);
  } else {
    hipLaunchKernelGGL((moe_router_kernel<2, 4>), dim3((unsigned)((T + 3) / 4), (unsigned)((E + 7) / 8)),
                       dim3(256), 0, stream, (const u32x4*)x, (const u32x4*)w, (float*)logits, T, E, H / 8);
  }
  return hipGetLastError();
}

MoeForm moe_form(int64_t T, int64_t E, int64_t H, int64_t I, int64_t top_k) {
  const int64_t chunks = (T + kMoeTokens - 1) / kMoeTokens, slots = (T < kMoeTokens ? T : kMoeTokens) * top_k;
  const int64_t most = slots < E ? slots : E;  // experts a chunk can reach
  MoeForm f;
  f.routing = T <= kInlineTokens ? 0 : T <= 16 ? 1 : 2;
  // Workgroups of 64 rows, whose waves take all units of K one after the other, where there is one
  // for each of an MI355X's 256 compute units, with more than 8 units two; else of 16 rows with K over
  // the waves. (The layer, 16 rows against 64: 4 tokens, 8 of 256 experts, 1024 x 512, 31 us
  // against 24, 256 workgroups of 64 rows; 3 tokens, 6 of 64, 2048 x 1408, 38 against 34, 396; but
  // 4 tokens, 2 of 16, 6144 x 2048, 39 against 50, 256; 1 token, 8 of 128, 4096 x 1024, 20 against 28, 128.)
  const int64_t units = (H / 32 + kUnit - 1) / kUnit;
  f.staged = (I + 63) / 64 * most * chunks >= (units <= 8 ? 256 : 512);
  f.few = f.staged && (T <= 16 || (units < 8 && slots <= 8 * E));
  f.groups = moe_groups(T, H);
  return f;
}

hipError_t launch_moe(const MoeProblem& p, hipStream_t stream) {
  const unsigned chunks = (unsigned)((p.T + kMoeTokens - 1) / kMoeTokens);
  const int64_t slots = (p.T < kMoeTokens ? p.T : kMoeTokens) * p.top_k;
  const unsigned most = (unsigned)(slots < p.E ? slots : p.E);  // experts a chunk can reach
  const MoeForm f = moe_form(p.T, p.E, p.H, p.I, p.top_k);
  const bool in_line = f.routing == 0;
  hipError_t e;
  if (!in_line) {
    if (p.given_ids != nullptr) {
      hipLaunchKernelGGL(moe_plan_kernel<Routing::kGiven>, dim3(chunks), dim3(1024), 0, stream, p);
    } else if (f.routing == 1) {
      hipLaunchKernelGGL(moe_plan_kernel<Routing::kOwn>, dim3(1), dim3(1024), 0, stream, p);
    } else {
      hipLaunchKernelGGL(moe_route_kernel, dim3((unsigned)((p.T + 3) / 4)), dim3(256), 0, stream, p);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(moe_plan_kernel<Routing::kPlanned>, dim3(chunks), dim3(1024), 0, stream, p);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 wide((unsigned)((p.I + 63) / 64), most, chunks), narrow((unsigned)(p.I / 16), most, chunks);
  const dim3 block(64 * kGateWaves);
  const bool given = p.given_ids != nullptr;
  if (f.staged) {
    if (in_line && given) hipLaunchKernelGGL((moe_gate_up_kernel<Routing::kGiven, true>), wide, block, 0, stream, p);
    else if (in_line) hipLaunchKernelGGL((moe_gate_up_kernel<Routing::kOwn, true>), wide, block, 0, stream, p);
    else if (f.few) hipLaunchKernelGGL((moe_gate_up_kernel<Routing::kPlanned, true>), wide, block, 0, stream, p);
    else hipLaunchKernelGGL((moe_gate_up_kernel<Routing::kPlanned, false>), wide, block, 0, stream, p);
  } else {
    if (in_line && given) hipLaunchKernelGGL(moe_gate_up_split_kernel<Routing::kGiven>, narrow, block, 0, stream, p);
    else if (in_line) hipLaunchKernelGGL(moe_gate_up_split_kernel<Routing::kOwn>, narrow, block, 0, stream, p);
    else hipLaunchKernelGGL(moe_gate_up_split_kernel<Routing::kPlanned>, narrow, block, 0, stream, p);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int groups = f.groups;
  if (groups == 0) {
    hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(p.H / 16)), dim3(1024), 0, stream, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(moe_down_wide_kernel, dim3((unsigned)((p.H + 63) / 64), groups, chunks), dim3(256), 0, stream, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)p.T, (unsigned)((p.H + 1023) / 1024)), dim3(256), 0, stream, p, groups);
  return hipGetLastError();
}

}  // namespace nvfp4
