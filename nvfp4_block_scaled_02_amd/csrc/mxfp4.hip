// MXFP4 path for gfx950: quantize (bf16 -> E2M1 codes with one E8M0 scale per 32 elements),
// dequantize, and the product of two MXFP4 operands on the block-scaled MFMA.
//
// MXFP4 is the 4-bit member of the Open Compute Project's microscaling formats: E2M1
// elements in 32-element blocks that share one power-of-two scale. A block's shared
// exponent is e = floor(log2(amax)) - 2 (2 = the exponent of the largest E2M1 value,
// 6 = 1.5 * 2^2) clamped to [-127, 127], stored as the byte e + 127; an all-zero block
// takes byte 0, and a block that holds a NaN or an infinity takes byte 0xFF, the scale
// format's NaN, so that it reads back as NaN. Elements are the E2M1 value nearest to
// x / 2^e, ties to the even code, saturating at 6, sign copied.
#include "gemm_common.hpp"

namespace nvfp4 {

namespace {

typedef int v8i_t __attribute__((ext_vector_type(8)));

// Scale byte of a block from the largest bf16 magnitude pattern in it (sign bits cleared):
// the exponent field less 2, zero for zero and subnormal maxima (whose floor(log2) is at
// most -127), 0xFF for infinities and NaN.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax16) {
  const int field = (int)(amax16 >> 7);
  return field == 0xFF ? 0xFFu : (uint32_t)max(field - 2, 0);
}

// The scale of byte b as the binary32 operand of gfx950's scaled conversions, which take
// its exponent field alone: field 0 stands for 2^-127 and field 255 for NaN.
__device__ __forceinline__ float mx4_scale_operand(uint32_t b) { return u2f(b << 23); }

// ---- quantize ----------------------------------------------------------------------
//
// Memory-bound: 2 B read, 1/2 + 1/32 B written per element. Four lanes share a block:
// lane 4i+q loads elements [8q, 8q+8) of block i (16 bytes, so that a wave's load reads
// 1 KiB of consecutive bytes). The block's maximum is taken on the bf16 bit patterns (for
// magnitudes their integer order is the order of the values), and each lane converts its
// elements with the scaled conversion from bf16 (x / 2^e, nearest even, saturating: equal
// to the rule above for every bf16 value and scale), 4 bytes of codes per lane.
template <int UNROLL>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const u32x4* __restrict__ x,
                                                           uint32_t* __restrict__ packed,
                                                           uint8_t* __restrict__ scales,
                                                           int64_t nlanes) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x * UNROLL;
  for (int64_t base = (int64_t)blockIdx.x * blockDim.x * UNROLL + threadIdx.x; base < nlanes;
       base += stride) {
    u32x4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t li = base + (int64_t)u * blockDim.x;
      v[u] = li < nlanes ? __builtin_nontemporal_load(&x[li]) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t li = base + (int64_t)u * blockDim.x;
      uint32_t a = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a = max(a, v[u][i] & 0x7FFFu);
        a = max(a, (v[u][i] >> 16) & 0x7FFFu);
      }
      // quad maximum (DPP quad_perm [1,0,3,2], then [2,3,0,1]); nlanes is a multiple of 4,
      // so the lanes of a quad are in or out of range together
      a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, false));
      a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, false));
      const uint32_t byte = mx4_scale_byte(a);
      const float s = mx4_scale_operand(byte);
      // each pair through an integer of its own: __builtin_bit_cast of a vector's element
      // takes the first element whatever the index (this toolchain)
      const uint32_t x0 = v[u].x, x1 = v[u].y, x2 = v[u].z, x3 = v[u].w;
      uint32_t w = 0u;
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x0), s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x1), s, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x2), s, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x3), s, 3);
      if (byte == 0xFFu) w = 0u;  // a NaN block's codes are not read: any fixed value
      if (li < nlanes) {
        __builtin_nontemporal_store(w, &packed[li]);
        if ((li & 3) == 0) scales[li >> 2] = (uint8_t)byte;
      }
    }
  }
}

// ---- dequantize ----------------------------------------------------------------------
//
// Memory-bound the other way: a lane reads 8 codes (4 bytes) and its block's scale byte
// and stores 8 bf16 values (16 bytes). E2M1 times a power of two is exact in bf16 (also
// among its subnormals); only 2^126 and 2^127 times 4 and 6 exceed its range, and become
// infinities.
template <int UNROLL>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint32_t* __restrict__ packed,
                                                             const uint8_t* __restrict__ scales,
                                                             u32x4* __restrict__ out,
                                                             int64_t nlanes) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x * UNROLL;
  for (int64_t base = (int64_t)blockIdx.x * blockDim.x * UNROLL + threadIdx.x; base < nlanes;
       base += stride) {
    uint32_t c[UNROLL], b[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t li = base + (int64_t)u * blockDim.x;
      c[u] = li < nlanes ? packed[li] : 0u;
      b[u] = li < nlanes ? scales[li >> 2] : 0u;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t li = base + (int64_t)u * blockDim.x;
      const float s = mx4_scale_operand(b[u]);
      u32x4 o;
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], s, 3));
      if (li < nlanes) __builtin_nontemporal_store(o, &out[li]);
    }
  }
}

// ---- GEMM ----------------------------------------------------------------------------
//
// out[M, N] (bf16) = A_hat[M, K] W_hat[N, K]^T. v_mfma_scale_f32_32x32x64_f8f6f4 takes
// E2M1 operands and E8M0 scales as stored: over a 64-element step, lane (h, r) =
// (lane / 32, lane % 32) of an operand holds the 32 elements of row r's block h (16
// bytes) and that block's scale byte. The weights are its A operand, so that a lane's
// results are four neighbouring columns of one output row.
__global__ void __launch_bounds__(256) gemm_mx4_simple_kernel(GemmProblem p) {
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int h = lane >> 5, r32 = lane & 31;
  const int64_t tiles_n = (p.N + 63) / 64;
  const int64_t m0 = (blockIdx.x / tiles_n) * 64 + 32 * (wave >> 1);
  const int64_t n0 = (blockIdx.x % tiles_n) * 64 + 32 * (wave & 1);
  // rows past the end read the last row; their results are not stored
  const int64_t m = min(m0 + r32, p.M - 1), n = min(n0 + r32, p.N - 1);
  const int64_t nb = p.K >> 5;
  const uint8_t* xa = p.a_packed + m * (p.K >> 1);
  const uint8_t* wa = p.w_packed + n * (p.K >> 1);
  const uint8_t* xs = p.a_scales + m * nb;
  const uint8_t* ws = p.w_scales + n * nb;
  floatx16 acc[1][1];
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[0][0][v] = 0.0f;
  for (int64_t b = 0; b < nb; b += 2) {
    const bool in = b + h < nb;  // an odd last block: the other half multiplies zeros
    const int64_t at = in ? b + h : b;
    const u32x4 xc = *(const u32x4*)&xa[16 * at], wc = *(const u32x4*)&wa[16 * at];
    const int xb = in ? xs[at] : 0, wb = in ? ws[at] : 0;
    const v8i_t xv = {in ? (int)xc.x : 0, in ? (int)xc.y : 0, in ? (int)xc.z : 0, in ? (int)xc.w : 0, 0, 0, 0, 0};
    const v8i_t wv = {in ? (int)wc.x : 0, in ? (int)wc.y : 0, in ? (int)wc.z : 0, in ? (int)wc.w : 0, 0, 0, 0, 0};
    acc[0][0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, xv, acc[0][0], 4, 4, 0, wb, 0, xb);
  }
  store_tile<1, 1>(acc, p, Alpha{1.0f, 0}, m0, n0, lane);
}

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int64_t M, int64_t K, void* packed, void* scales,
                               hipStream_t stream, const LaunchInfo& dev) {
  const int64_t nlanes = M * K / 8;
  if (nlanes == 0) return hipSuccess;
  constexpr int kThreads = 256, kUnroll = 2;
  const int64_t want = (nlanes + (int64_t)kThreads * kUnroll - 1) / ((int64_t)kThreads * kUnroll);
  const int64_t cap = (int64_t)dev.num_cus * 32;
  hipLaunchKernelGGL((mx4_quantize_kernel<kUnroll>), dim3((unsigned)(want < cap ? want : cap)),
                     dim3(kThreads), 0, stream, (const u32x4*)x, (uint32_t*)packed,
                     (uint8_t*)scales, nlanes);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const void* packed, const void* scales, int64_t M, int64_t K,
                                 void* out, hipStream_t stream, const LaunchInfo& dev) {
  const int64_t nlanes = M * K / 8;
  if (nlanes == 0) return hipSuccess;
  constexpr int kThreads = 256, kUnroll = 2;
  const int64_t want = (nlanes + (int64_t)kThreads * kUnroll - 1) / ((int64_t)kThreads * kUnroll);
  const int64_t cap = (int64_t)dev.num_cus * 32;
  hipLaunchKernelGGL((mx4_dequantize_kernel<kUnroll>), dim3((unsigned)(want < cap ? want : cap)),
                     dim3(kThreads), 0, stream, (const uint32_t*)packed, (const uint8_t*)scales,
                     (u32x4*)out, nlanes);
  return hipGetLastError();
}

hipError_t launch_mx4_gemm(const GemmProblem& p, hipStream_t stream, const LaunchInfo& dev) {
  (void)dev;
  const int64_t tiles = ((p.M + 63) / 64) * ((p.N + 63) / 64);
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(gemm_mx4_simple_kernel, dim3((unsigned)tiles), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
