// The residual and the norms around a transformer block's branch, in one pass, for gfx950.
//
// For a row m of group g (its sequence), with the residual stream x, a branch's output y and
// norm(v) = v / sqrt(mean(v^2) + eps) or (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps):
//   z = y, or norm(y) * post;   h = bf16(x + c * gate_g * z)
//   n = norm(h) * weight + bias;   n = n * (1 + scale_g) + shift_g
//   out = bf16(n), or that value as the library's quantizers store it, byte for byte.
// The second norm takes h as it is stored.
//
// Memory-bound: x and y are read and h and out written once (8 bytes per element with a bf16
// result). A row stays in registers, 8 elements (16 bytes) per thread and chunk, its sums in
// fp32. What a sum in fp32 misses of the mean, up to 2^-18 of the values, would stay in every element
// of a row far from zero: it is what is left of the mean after it is taken away, summed along with the
// squares. A row of equal values has exactly their mean (its sum, up to 2^15 values of 8 bits, and
// its quotient are exact), and nothing is left.
#include "quant_common.hpp"
#include "quant_mx.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

// Sums over the threads of a row: a wave's in the vector unit, the waves' in LDS. Two buffers in
// turn: a buffer is written again only behind the next sum's barrier.
template <int kThreads>
struct RowSum {
  float (*part)[2 * (kThreads / 64)];
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = wave_sum(v);
    if constexpr (kThreads == 64) return v;
    float* p = part[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
    __syncthreads();
    v = p[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) v += p[w];
    return v;
  }
  __device__ __forceinline__ void both(float& a, float& b) {
    constexpr int kWaves = kThreads / 64;
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (kThreads == 64) return;
    float* p = part[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      p[threadIdx.x >> 6] = a;
      p[kWaves + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = p[0];
    b = p[kWaves];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      a += p[w];
      b += p[kWaves + w];
    }
  }
  __device__ __forceinline__ float max(float v) {  // of values >= 0
    v = u2f(wave_max_u32(f2u(v)));
    if constexpr (kThreads == 64) return v;
    float* p = part[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
    __syncthreads();
    v = p[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) v = __builtin_fmaxf(v, p[w]);
    return v;
  }
};

// v = norm(v) over the row's H elements, of which this thread holds its chunks.
template <int kThreads, int kChunks, bool kLayer>
__device__ __forceinline__ void normalize(float (&v)[kChunks][8], RowSum<kThreads>& sum, int thread, int chunks,
                                          float H, float rH, float eps) {
  float left = 0.0f, squares = 0.0f;
  if constexpr (kLayer) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[c][i];  // (chunks past the row hold zeros)
    const float mean = sum(s) / H;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = thread + kThreads * c < chunks ? v[c][i] - mean : 0.0f;
        left += v[c][i];
      }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) squares = __builtin_fmaf(v[c][i], v[c][i], squares);
  float off = 0.0f;  // of the mean
  if constexpr (kLayer) {
    sum.both(left, squares);
    off = left * rH;
    squares = __builtin_fmaxf(__builtin_fmaf(-off, left, squares), 0.0f);  // about the mean
  } else {
    squares = sum(squares);
  }
  const float r = 1.0f / sqrtf(squares * rH + eps);
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = (kLayer ? v[c][i] - off : v[c][i]) * r;
}

// kThreads threads per row (64: four rows per workgroup), kChunks chunks of 8 elements each.
template <int kThreads, int kChunks, bool kLayer>
__global__ void __launch_bounds__(kThreads == 64 ? 256 : kThreads) norm_kernel(NormProblem p) {
  constexpr int kRows = kThreads == 64 ? 4 : 1;
  __shared__ float part[2][2 * (kThreads / 64)];
  RowSum<kThreads> sum{part};
  const int thread = kThreads == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int chunks = (int)(p.H >> 3);
  const float H = (float)p.H, rH = 1.0f / H;
  const QuantScale qs = p.format == NVFP4_NORM_NVFP4 ? quant_scale(p.gs, 6.0f * p.gs, 1.0f / (6.0f * p.gs), p.gs_dev)
                                                      : QuantScale{1.0f, 6.0f, 1.0f};
  for (int64_t row = (int64_t)blockIdx.x * kRows + (kRows > 1 ? threadIdx.x >> 6 : 0); row < p.M;
       row += (int64_t)gridDim.x * kRows) {
    const int64_t at = row * chunks;
    u32x4 xv[kChunks], yv[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = thread + kThreads * c;
      xv[c] = yv[c] = u32x4{0u, 0u, 0u, 0u};
      if (i < chunks) {
        xv[c] = ((const u32x4*)p.x)[at + i];
        if (p.y) yv[c] = ((const u32x4*)p.y)[at + i];
      }
    }
    // the row's group; none: its vectors read as zero
    int64_t group = p.rows ? p.rows[row] : p.groups == 1 ? 0 : row / (p.M / p.groups);
    const bool grouped = group >= 0 && group < p.groups;
    if (!grouped) group = 0;
    const int64_t group_at = group * chunks;
    float v[kChunks][8];
    if (p.y) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) unpack_bf16x8(yv[c], v[c]);
      if (p.post) normalize<kThreads, kChunks, kLayer>(v, sum, thread, chunks, H, rH, p.eps);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i = thread + kThreads * c;
        if (i < chunks) {
          float f[8];
          if (p.post) {
            unpack_bf16x8(((const u32x4*)p.post)[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] *= f[j];
          }
          if (p.gate) {
            unpack_bf16x8(((const u32x4*)p.gate)[group_at + i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] *= f[j];
          }
          unpack_bf16x8(xv[c], f);
          u32x4 o;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = bf16x2_rne(__builtin_fmaf(p.residual_scale, v[c][2 * j], f[2 * j]),
                              __builtin_fmaf(p.residual_scale, v[c][2 * j + 1], f[2 * j + 1]));
          if (p.gate && !grouped) o = xv[c];
          ((u32x4*)p.h)[at + i] = o;
          xv[c] = o;
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) unpack_bf16x8(xv[c], v[c]);
    normalize<kThreads, kChunks, kLayer>(v, sum, thread, chunks, H, rH, p.eps);
    u32x4 n[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = thread + kThreads * c;
      n[c] = u32x4{0u, 0u, 0u, 0u};
      if (i < chunks) {
        float f[8];
        if (p.weight) {
          unpack_bf16x8(((const u32x4*)p.weight)[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] *= f[j];
        }
        if (p.bias) {
          unpack_bf16x8(((const u32x4*)p.bias)[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] += f[j];
        }
        if (p.scale && grouped) {
          unpack_bf16x8(((const u32x4*)p.scale)[group_at + i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] = __builtin_fmaf(v[c][j], f[j], v[c][j]);
        }
        if (p.shift && grouped) {
          unpack_bf16x8(((const u32x4*)p.shift)[group_at + i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] += f[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) n[c][j] = bf16x2_rne(v[c][2 * j], v[c][2 * j + 1]);
      }
    }
    // The lanes of a block are together in the row or past it: its length is a multiple of
    // the block's.
    if (p.format == NVFP4_NORM_BF16) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i = thread + kThreads * c;
        if (i < chunks) ((u32x4*)p.out)[at + i] = n[c];
      }
    } else if (p.format == NVFP4_NORM_MXFP4) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i = thread + kThreads * c;
        const Mx4Codes q = mx4_encode_quad(n[c]);
        if (i < chunks) {
          ((uint32_t*)p.out)[at + i] = q.word;
          if ((i & 3) == 0) ((uint8_t*)p.scales)[(at + i) >> 2] = (uint8_t)q.byte;
        }
      }
    } else if (p.format == NVFP4_NORM_MXFP8) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i = thread + kThreads * c;
        const Mx8Codes q = mx8_encode_quad<false>(n[c]);
        if (i < chunks) {
          ((u32x2*)p.out)[at + i] = q.words;
          if ((i & 3) == 0) ((uint8_t*)p.scales)[(at + i) >> 2] = (uint8_t)q.byte;
        }
      }
    } else if (p.format == NVFP4_NORM_NVFP4) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i = thread + kThreads * c;
        float f[8];
        unpack_bf16x8(n[c], f);
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = __builtin_fmaxf(a, __builtin_fabsf(f[j]));
        // partner lane's partial maximum (DPP quad_perm [1, 0, 3, 2]: lane ^ 1)
        const float o = u2f((uint32_t)__builtin_amdgcn_mov_dpp((int)f2u(a), 0xB1, 0xF, 0xF, false));
        const BlockScale bs = block_scale(__builtin_fmaxf(a, o), qs.den, qs.rden, qs.gs);
        const uint32_t word = __any(bs.code == kE4M3MaxCode) ? encode_half<true>(f, bs) : encode_half<false>(f, bs);
        if (i < chunks) {
          ((uint32_t*)p.out)[at + i] = word;
          if ((i & 1) == 0) ((uint8_t*)p.scales)[(at + i) >> 1] = (uint8_t)bs.code;
        }
      }
    } else {
      float a = 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) a = amax8(n[c], a);
      const RowScale rs = row_scale(sum.max(a), (float*)p.scales, row, thread);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i = thread + kThreads * c;
        if (i < chunks) ((u32x2*)p.out)[at + i] = encode8(n[c], rs.s, rs.r, rs.corrected);
      }
    }
  }
}

template <int kThreads, int kChunks>
hipError_t launch(const NormProblem& p, hipStream_t stream) {
  constexpr int64_t kMost = 1 << 20;  // workgroups (a launch has fewer than 2^32 threads)
  const int64_t want = kThreads == 64 ? (p.M + 3) / 4 : p.M;
  const dim3 grid((unsigned)(want < kMost ? want : kMost)), block(kThreads == 64 ? 256 : kThreads);
  if (p.kind == NVFP4_NORM_LAYER)
    hipLaunchKernelGGL((norm_kernel<kThreads, kChunks, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((norm_kernel<kThreads, kChunks, false>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_norm(const NormProblem& p, hipStream_t stream, const LaunchInfo& dev) {
  if (p.M == 0) return hipSuccess;
  const int64_t chunks = p.H >> 3;
  // Threads to a row: as few as hold it in four chunks each, so that many rows are under way (16384 x
  // 2048: 256 threads 53 us, 512 65; 16384 x 8192 at 5.3 TB/s either way). With no more rows than compute
  // units, widths of two chunks to 256 threads take one each (64 x 4096: 4.5 us, 512 threads 4.0). Other
  // widths do not, though they would gain as well (in a graph, 64 x 1024: 3.2 us, 128 threads 2.7; 64 x
  // 8192: 4.7, 1024 threads 3.7).
  if (chunks > 256 && chunks <= 512 && p.M <= dev.num_cus) return launch<512, 1>(p, stream);
  if (chunks <= 64) return launch<64, 1>(p, stream);
  if (chunks <= 128) return launch<64, 2>(p, stream);
  if (chunks <= 256) return launch<256, 1>(p, stream);
  if (chunks <= 512) return launch<256, 2>(p, stream);
  if (chunks <= 768) return launch<256, 3>(p, stream);
  if (chunks <= 1024) return launch<256, 4>(p, stream);
  if (chunks <= 2048) return launch<512, 4>(p, stream);
  return launch<1024, 4>(p, stream);
}

}  // namespace nvfp4
