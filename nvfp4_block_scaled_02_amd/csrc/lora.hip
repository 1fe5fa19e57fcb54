// Low-rank adapters of many requests beside a shared projection, for gfx950.
//
// For row t with adapter a = adapters[t] in [0, L):
//   v_t = s_a * A_a x_t  (R sums over K),   out_t = bf16(y_t + B_a v_t);
// any other row keeps y_t. x [T, K], A [L, R, K], B [L, N, R], y and out [T, N], all bf16.
//
// Two kernels: v, fp32, in kSplits parts over K, and its product with B. Both work on 16 rows at
// a time with v_mfma_f32_16x16x32_bf16: the adapter's rows are its A operand, 16 rows of
// activations its columns, so that a result column belongs to one row alone. Rows come in any
// order: a workgroup lists the distinct adapters of its rows, takes them one after the other
// and keeps of each result the columns whose adapter it is. Where there are few rows the
// adapters are dealt out to several workgroups (grid z) instead.
//
// v enters the second product in two bf16 parts that add up to it within 2^-16 of its value
// (rounded to one it would be off by as much as the output's own rounding).
#include "gemm_common.hpp"
#include "lora_offsets.hpp"

namespace nvfp4 {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ floatx4 mfma(const u32x4 a, const u32x4 b, const floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                 c, 0, 0, 0);
}

// The adapter of a lane's row (lane % 16), -1 where it has none.
__device__ __forceinline__ int adapter_of(const LoraProblem& p, int64_t t) {
  const int a = t < p.T ? p.adapters[t] : -1;
  return a >= 0 && a < p.L ? a : -1;
}

// Calls f(adapter) for the distinct adapters of lanes 0..15 that are this workgroup's: the
// i-th where i % gridDim.z == blockIdx.z.
template <typename F>
__device__ __forceinline__ void for_adapters(int adapter, const F& f) {
  uint64_t left = __ballot(adapter >= 0) & 0xFFFFull;
  for (unsigned i = 0; left != 0; ++i) {
    const int a = __builtin_amdgcn_readlane(adapter, __builtin_ctzll(left));
    left &= ~__ballot(adapter == a);
    if (i % gridDim.z == blockIdx.z) f(a);
  }
}

// v[split][t][r] of 16 rows: a workgroup's four waves take steps of 32 elements of K in turn,
// and the splits (grid y) between them.
template <int kTiles>
__global__ void __launch_bounds__(256) lora_down_kernel(LoraProblem p) {
  __shared__ floatx4 part[3][kTiles][64];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * 16, t = t0 + r;
  const int adapter = adapter_of(p, t);
  const int chunks = (int)(p.K >> 3), steps = (chunks + 3) / 4;
  const int begin = lora_split_begin(steps, blockIdx.y, gridDim.y), end = lora_split_begin(steps, blockIdx.y + 1, gridDim.y);
  const u32x4* x = (const u32x4*)p.x + min(t, p.T - 1) * chunks;
  for_adapters(adapter, [&](int a) {
    const u32x4* w = (const u32x4*)p.a + (int64_t)a * p.R * chunks;
    floatx4 acc[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = begin + wave; s < end; s += 4) {
      const int c = 4 * s + q;
      const bool in = c < chunks;
      const u32x4 none = {0u, 0u, 0u, 0u};
      const u32x4 xv = in ? x[c] : none;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const u32x4 wv = in ? w[(int64_t)min(16 * i + r, p.R - 1) * chunks + c] : none;
        acc[i] = mfma(wv, xv, acc[i]);
      }
    }
    __syncthreads();
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) part[wave - 1][i][lane] = acc[i];
    }
    __syncthreads();
    if (wave == 0 && adapter == a) {
      float* v = p.down + ((int64_t)blockIdx.y * p.T + t) * p.R;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        if (16 * i + 4 * q >= p.R) break;  // R % 8 == 0: four rows are all there or none
        *(floatx4*)&v[16 * i + 4 * q] = acc[i] + part[0][i][lane] + part[1][i][lane] + part[2][i][lane];
      }
    }
  });
}

// A value in two bf16 parts: the upper half of its 32 bits (cut, so that it overflows with the
// value alone), and the rest, rounded. An infinity has no rest.
__device__ __forceinline__ void two_parts(const float (&v)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b0 = f2u(v[2 * j]), b1 = f2u(v[2 * j + 1]);
    const float r0 = (b0 & 0x7FFFFFFFu) == 0x7F800000u ? 0.0f : v[2 * j] - u2f(b0 & 0xFFFF0000u);
    const float r1 = (b1 & 0x7FFFFFFFu) == 0x7F800000u ? 0.0f : v[2 * j + 1] - u2f(b1 & 0xFFFF0000u);
    hi[j] = (b0 >> 16) | (b1 & 0xFFFF0000u);
    lo[j] = bf16x2_rne(r0, r1);
  }
}

// out = y + B v of 16 rows. A wave takes 64 columns of the output at a time, as four fragments of
// 16 rows of B such that a lane's results are 16 consecutive columns. v's two parts follow one
// another along the matrix instruction's K: chunk c (8 elements) of 2R is chunk c % (R / 8) of R,
// of the upper part first.
template <int kSteps>
__global__ void __launch_bounds__(256) lora_up_kernel(LoraProblem p, int splits) {
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * 16 + r;
  const int64_t n0 = ((int64_t)blockIdx.y * 4 + wave) * 64;
  if (n0 >= p.N) return;
  const int adapter = adapter_of(p, t);
  const int R8 = p.R >> 3;
  floatx4 sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  for_adapters(adapter, [&](int a) {
    const float s = p.scales ? p.scales[a] : 1.0f;
    const u32x4* w = (const u32x4*)p.b + (int64_t)a * p.N * R8;
    floatx4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int c = 4 * k + q, at = c % R8;
      const bool in = c < 2 * R8;
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (in && adapter == a) {
        for (int j = 0; j < splits; ++j) {
          const floatx4* d = (const floatx4*)&p.down[((int64_t)j * p.T + t) * p.R + 8 * at];
          const floatx4 d0 = d[0], d1 = d[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] += d0[i];
            v[4 + i] += d1[i];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= s;
      u32x4 hi, lo;
      two_parts(v, hi, lo);
      const u32x4 part = c < R8 ? hi : lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t n = min(n0 + lora_column(r, i), p.N - 1);
        const u32x4 wv = in ? w[n * R8 + at] : u32x4{0u, 0u, 0u, 0u};
        acc[i] = mfma(wv, part, acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (adapter == a) sum[i] = acc[i];
  });
  // a lane's row and its 16 columns; of an adapter that is another workgroup's: nothing
  if (t >= p.T) return;
  bool mine = false;
  for_adapters(adapter, [&](int a) { mine = mine || adapter == a; });
  if (adapter < 0) mine = blockIdx.z == 0;
  if (!mine) return;
  const uint16_t* y = p.y + t * p.N;
  uint16_t* out = p.out + t * p.N;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + 16 * q + 4 * i + j;
      if (n < p.N) out[n] = adapter < 0 ? y[n] : (uint16_t)bf16x2_rne(u2f((uint32_t)y[n] << 16) + sum[i][j], 0.0f);
    }
  }
}

}  // namespace

int64_t lora_down_bytes(int64_t T, int64_t K, int64_t R) { return lora_splits(T, K) * T * R * 4; }

hipError_t launch_lora(const LoraProblem& p, hipStream_t stream) {
  if (p.T == 0 || p.N == 0) return hipSuccess;
  const unsigned tiles = (unsigned)((p.T + 15) / 16), splits = (unsigned)lora_splits(p.T, p.K), z = (unsigned)lora_deal(p.T);
  const dim3 down(tiles, splits, z), up(tiles, (unsigned)((p.N + 255) / 256), z);
  switch ((p.R + 15) / 16) {
#define NVFP4_LORA_CASE(n)                                                                          \
  case n:                                                                                           \
    hipLaunchKernelGGL((lora_down_kernel<n>), down, dim3(256), 0, stream, p);                       \
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;                                \
    hipLaunchKernelGGL((lora_up_kernel<n>), up, dim3(256), 0, stream, p, (int)splits);              \
    break;
    NVFP4_LORA_CASE(1)
    NVFP4_LORA_CASE(2)
    NVFP4_LORA_CASE(3)
    NVFP4_LORA_CASE(4)
    NVFP4_LORA_CASE(5)
    NVFP4_LORA_CASE(6)
    NVFP4_LORA_CASE(7)
    NVFP4_LORA_CASE(8)
#undef NVFP4_LORA_CASE
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
