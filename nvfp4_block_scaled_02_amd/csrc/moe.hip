// A mixture-of-experts layer for a few tokens on gfx950, with MXFP4 expert weights and bf16
// activations: the router's product, and the routed experts' gated feed-forward.
//
// For token t with logits l_t over E experts: the top_k experts of largest logit (ties to
// the lowest index) with softmax weights g, taken over all E or over the chosen ones; then
//   h_tj = silu(Wg_e x_t) * (Wu_e x_t),  e = the j-th chosen expert, silu(z) = z / (1 + exp(-z))
//   out_t = sum_j g_tj (W2_e h_tj).
// W13 holds the gate rows Wg and then the up rows Wu of each expert, [E, 2I, H]; W2 is
// [E, H, I]; both MXFP4 along their last axis.
#include "gemm_common.hpp"

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
// logits[t, e] = sum_h x[t, h] w[e, h], each product exact in fp32 (8 x 8 significant bits)
// and the sum kept in fp64, rounded once to fp32: two experts whose logits differ by more
// than that rounding are never exchanged by the order of the summation. One wave per
// expert and group of kTT tokens.
template <int kTT>
__global__ void __launch_bounds__(256) moe_router_kernel(const u32x4* __restrict__ x,
                                                         const u32x4* __restrict__ w,
                                                         float* __restrict__ logits, int64_t T,
                                                         int64_t E, int64_t H8) {
  const int lane = threadIdx.x & 63;
  const int64_t e = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t0 = (int64_t)blockIdx.y * kTT;
  if (e >= E) return;
  double acc[kTT] = {};
  for (int64_t i = lane; i < H8; i += 64) {
    const u32x4 wv = w[e * H8 + i];
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      const u32x4 xv = x[min(t0 + t, T - 1) * H8 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[t] += (double)(u2f(xv[j] << 16) * u2f(wv[j] << 16));
        acc[t] += (double)(u2f(xv[j] & 0xFFFF0000u) * u2f(wv[j] & 0xFFFF0000u));
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off, 64);
    if (lane == 0 && t0 + t < T) logits[(t0 + t) * E + e] = (float)acc[t];
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
  int slot[kMoeSlots];
};

// Order of two logits as an unsigned key: increasing with the value, NaN above +inf, and
// -inf at 0 (never chosen).
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = f2u(l + 0.0f);  // -0 counts as 0
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if (b == 0xFF800000u) return 0u;
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

// The top_k of one token by one wave. Lane l holds experts l, l + 64, ...; each round takes
// the largest key, the lowest index among equals. A row of fewer than top_k experts that
// can be chosen ends in slots of id -1 and weight 0.
__device__ __forceinline__ void moe_topk(const float* __restrict__ row, int E, int top_k,
                                         bool renormalize, int lane, int* ids, float* weights) {
  constexpr int kPer = kMoeExperts / 64;
  float l[kPer];
  uint32_t key[kPer];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? row[e] : -__builtin_inff();
    key[i] = logit_key(l[i]);
    top = l[i] != l[i] ? l[i] : (top != top ? top : __builtin_fmaxf(top, l[i]));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float o = __shfl_xor(top, off, 64);
    top = o != o ? o : (top != top ? top : __builtin_fmaxf(top, o));
  }
  float sum = 0.0f;
  if (!renormalize) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] != 0u) sum += expf(l[i] - top);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  }
  int my_id = -1;        // lane j keeps the j-th choice
  float my_w = 0.0f;
  for (int j = 0; j < top_k; ++j) {
    uint32_t bk = 0u;
    int be = 0x7FFFFFFF;
    float bl = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] > bk) {
        bk = key[i];
        be = lane + 64 * i;
        bl = l[i];
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint32_t ok = (uint32_t)__shfl_xor((int)bk, off, 64);
      const int oe = __shfl_xor(be, off, 64);
      const float ol = __shfl_xor(bl, off, 64);
      if (ok > bk || (ok == bk && oe < be)) {
        bk = ok;
        be = oe;
        bl = ol;
      }
    }
    if (bk == 0u) break;  // nothing left to choose (uniform over the wave)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 64 * i == be) key[i] = 0u;
    const float p = expf(bl - top);
    if (renormalize) sum += p;
    if (lane == j) {
      my_id = be;
      my_w = p;
    }
  }
  if (lane < top_k) {
    ids[lane] = my_id;
    weights[lane] = my_id < 0 ? 0.0f : my_w / sum;
  }
}

// One workgroup per chunk.
__global__ void __launch_bounds__(1024) moe_plan_kernel(MoeProblem p) {
  __shared__ int count[kMoeExperts];
  __shared__ int place[kMoeExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kMoeTokens;
  const int nt = (int)min(p.T - t0, (int64_t)kMoeTokens);
  const int n = nt * p.top_k;
  MoePlan* plan = (MoePlan*)p.plan + blockIdx.x;
  int* ids = p.ids + t0 * p.top_k;
  float* weights = p.weights + t0 * p.top_k;
  for (int e = threadIdx.x; e < p.E; e += 1024) count[e] = 0;
  for (int t = wave; t < nt; t += 16)
    moe_topk(p.logits + (t0 + t) * p.E, p.E, p.top_k, p.renormalize, lane, ids + t * p.top_k,
             weights + t * p.top_k);
  __threadfence_block();
  __syncthreads();
  const int s = threadIdx.x;  // n <= 1024
  const int e = s < n ? ids[s] : -1;
  if (e >= 0) atomicAdd(&count[e], 1);
  __syncthreads();
  if (wave == 0) {
    int active = 0, first = 0;
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
      if (b + lane < p.E) place[b + lane] = first + sum - c;
      if (c > 0) {
        plan->expert[rank] = b + lane;
        plan->first[rank] = first + sum - c;
      }
      active += __popcll(on);
      first += __shfl(sum, 63, 64);
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
// v_mfma_f32_16x16x32_bf16 with 16 weight rows as its A operand and 16 slots as columns.
// A lane (q, r) = (lane / 16, lane % 16) takes the 32 elements of block 4 g + q of row r
// (one 16-byte load, one scale byte) and feeds them to four MFMAs, eight elements each; the
// activations follow the same order of K. The scaled conversion to bf16 gives a weight's
// value exactly.
struct W4Block {
  u32x4 codes;
  uint32_t byte;
};
__device__ __forceinline__ W4Block load_block(const uint8_t* codes, const uint8_t* scales,
                                              int64_t b, int64_t nb) {
  W4Block w;
  if (b < nb) {
    w.codes = __builtin_nontemporal_load((const u32x4*)&codes[16 * b]);
    w.byte = scales[b];
  } else {
    w.codes = u32x4{0u, 0u, 0u, 0u};
    w.byte = 0u;
  }
  return w;
}
__device__ __forceinline__ bf16x8_t decode_part(const W4Block& w, int s) {
  const float sc = u2f(w.byte << 23);
  const uint32_t c = w.codes[s];
  const u32x4 o = {
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3))};
  return __builtin_bit_cast(bf16x8_t, o);
}
__device__ __forceinline__ u32x4 load_x(const uint16_t* row, int64_t b, int64_t nb, int s) {
  return b < nb ? *(const u32x4*)&row[32 * b + 8 * s] : u32x4{0u, 0u, 0u, 0u};
}

// h[slot, i] = silu(gate) * up for 16 gate rows and their 16 up rows of one expert and up
// to 64 slots: four waves split K and meet in LDS.
__global__ void __launch_bounds__(256) moe_gate_up_kernel(MoeProblem p) {
  constexpr int NW = 4, kTiles = kMoeTokens / 16;
  __shared__ floatx4 part[NW][2][64];
  const MoePlan* plan = (const MoePlan*)p.plan + blockIdx.z;
  const int a = blockIdx.y;
  if (a >= plan->active) return;
  const int64_t e = plan->expert[a];
  const int s0 = plan->first[a], ns = plan->first[a + 1] - s0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, r = lane & 15;
  const int64_t i0 = (int64_t)blockIdx.x * 16;
  const int64_t nb = p.H >> 5;
  const int64_t t0 = (int64_t)blockIdx.z * kMoeTokens;
  const int64_t grow = e * 2 * p.I + i0 + r, urow = grow + p.I;
  const uint8_t* gc = p.w13_packed + grow * (p.H >> 1);
  const uint8_t* uc = p.w13_packed + urow * (p.H >> 1);
  const uint8_t* gs = p.w13_scales + grow * nb;
  const uint8_t* us = p.w13_scales + urow * nb;
  for (int c0 = 0; c0 < ns; c0 += 16) {
    const int slot = plan->slot[s0 + min(c0 + r, ns - 1)];
    const uint16_t* xr = p.x + (t0 + slot / p.top_k) * p.H;
    floatx4 g = {0.0f, 0.0f, 0.0f, 0.0f}, u = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t b0 = 4 * wave; b0 < nb; b0 += 4 * NW) {
      const W4Block gw = load_block(gc, gs, b0 + q, nb), uw = load_block(uc, us, b0 + q, nb);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bf16x8_t xv = __builtin_bit_cast(bf16x8_t, load_x(xr, b0 + q, nb, s));
        g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode_part(gw, s), xv, g, 0, 0, 0);
        u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode_part(uw, s), xv, u, 0, 0, 0);
      }
    }
    __syncthreads();
    part[wave][0][lane] = g;
    part[wave][1][lane] = u;
    __syncthreads();
    if (wave == 0 && c0 + r < ns) {
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        g += part[w][0][lane];
        u += part[w][1][lane];
      }
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = g[i] / (1.0f + expf(-g[i])) * u[i];
      // h is rounded to bf16, the type of the activations that the next product takes
      *(u32x2*)&p.h[(t0 * p.top_k + slot) * p.I + i0 + 4 * q] = bf16x4_rne(v[0], v[1], v[2], v[3]);
    }
  }
  (void)kTiles;
}

// out[t, o] for 16 rows of W2 and one chunk of tokens: the workgroup's waves take (expert,
// K) parts in turn and each adds its weighted results to its own fp32 sums by token; the
// waves' sums are added in a fixed order.
__global__ void __launch_bounds__(512) moe_down_kernel(MoeProblem p) {
  constexpr int NW = 8;
  __shared__ float sums[NW][kMoeTokens][16];
  const MoePlan* plan = (const MoePlan*)p.plan + blockIdx.z;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, r = lane & 15;
  const int64_t o0 = (int64_t)blockIdx.x * 16;
  const int64_t nb = p.I >> 5;
  const int64_t t0 = (int64_t)blockIdx.z * kMoeTokens;
  const int nt = (int)min(p.T - t0, (int64_t)kMoeTokens);
  for (int i = threadIdx.x; i < NW * kMoeTokens * 16; i += 64 * NW) (&sums[0][0][0])[i] = 0.0f;
  __syncthreads();
  const int active = plan->active;
  for (int a = wave; a < active; a += NW) {
    const int64_t e = plan->expert[a];
    const int s0 = plan->first[a], ns = plan->first[a + 1] - s0;
    const int64_t row = e * p.H + o0 + r;
    const uint8_t* wc = p.w2_packed + row * (p.I >> 1);
    const uint8_t* ws = p.w2_scales + row * nb;
    for (int c0 = 0; c0 < ns; c0 += 16) {
      const int slot = plan->slot[s0 + min(c0 + r, ns - 1)];
      const uint16_t* hr = p.h + (t0 * p.top_k + slot) * p.I;
      floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int64_t b0 = 0; b0 < nb; b0 += 4) {
        const W4Block w = load_block(wc, ws, b0 + q, nb);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              decode_part(w, s), __builtin_bit_cast(bf16x8_t, load_x(hr, b0 + q, nb, s)), acc, 0, 0, 0);
      }
      if (c0 + r < ns) {
        const float g = p.weights[t0 * p.top_k + slot];
        float* to = &sums[wave][slot / p.top_k][4 * q];
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] += g * acc[i];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * 16; i += 64 * NW) {
    const int t = i >> 4, o = i & 15;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += sums[w][t][o];
    p.out[(t0 + t) * p.H + o0 + o] = (uint16_t)bf16x2_rne(v, 0.0f);
  }
}

}  // namespace

int64_t moe_plan_bytes(int64_t T) {
  return (T + kMoeTokens - 1) / kMoeTokens * (int64_t)sizeof(MoePlan);
}

hipError_t launch_moe_router(const void* x, const void* w, int64_t T, int64_t E, int64_t H,
                             void* logits, hipStream_t stream) {
  constexpr int kTT = 4;
  const dim3 grid((unsigned)((E + 3) / 4), (unsigned)((T + kTT - 1) / kTT));
  hipLaunchKernelGGL((moe_router_kernel<kTT>), grid, dim3(256), 0, stream, (const u32x4*)x,
                     (const u32x4*)w, (float*)logits, T, E, H / 8);
  return hipGetLastError();
}

hipError_t launch_moe(const MoeProblem& p, hipStream_t stream) {
  const unsigned chunks = (unsigned)((p.T + kMoeTokens - 1) / kMoeTokens);
  const int64_t slots = (p.T < kMoeTokens ? p.T : kMoeTokens) * p.top_k;
  const unsigned most = (unsigned)(slots < p.E ? slots : p.E);  // experts a chunk can reach
  hipLaunchKernelGGL(moe_plan_kernel, dim3(chunks), dim3(1024), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_gate_up_kernel, dim3((unsigned)(p.I / 16), most, chunks), dim3(256), 0,
                     stream, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(p.H / 16), 1, chunks), dim3(512), 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
