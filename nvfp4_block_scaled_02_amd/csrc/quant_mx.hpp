// Device helpers of the MXFP4, MXFP8 and rowwise FP8 quantizers, shared with the kernels that quantize
// what they have just computed: a lane holds 8 consecutive elements (16 bytes of bf16).
#pragma once

#include "gemm_common.hpp"

namespace nvfp4 {
namespace {

// ---- MXFP4 ----

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

// Four lanes share a block: lane 4i+q holds elements [8q, 8q+8) of block i. The block's
// maximum is taken on the bf16 bit patterns (for magnitudes their integer order is the order
// of the values), and each lane converts its elements with the scaled conversion from bf16
// (x / 2^e, nearest even, saturating: equal to the rule above for every bf16 value and
// scale) into 4 bytes of codes.
struct Mx4Codes {
  uint32_t word, byte;
};
__device__ __forceinline__ Mx4Codes mx4_encode_quad(const u32x4 v) {
  uint32_t a = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a = max(a, v[i] & 0x7FFFu);
    a = max(a, (v[i] >> 16) & 0x7FFFu);
  }
  // quad maximum: DPP quad_perm [1,0,3,2], then [2,3,0,1]
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, false));
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, false));
  const uint32_t byte = mx4_scale_byte(a);
  const float s = mx4_scale_operand(byte);
  // each pair through an integer of its own: __builtin_bit_cast of a vector's element takes
  // the first element whatever the index (this toolchain)
  const uint32_t x0 = v.x, x1 = v.y, x2 = v.z, x3 = v.w;
  uint32_t w = 0u;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x0), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x1), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x2), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x3), s, 3);
  return Mx4Codes{byte == 0xFFu ? 0u : w, byte};  // a NaN block's codes are 0
}

// ---- MXFP8 ----

__device__ __forceinline__ void mx_unpack_bf16x8(const u32x4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = u2f(w[i] << 16);
    f[2 * i + 1] = u2f(w[i] & 0xFFFF0000u);
  }
}

// x / 2^e clamped to the element type's finite range, [-448, 448] or [-57344, 57344]
// (sign of zero kept): the conversion below then never overflows, and the clamp is the
// format's saturation.
template <bool kE5M2>
__device__ __forceinline__ float mx_scaled(float x, int e) {
  constexpr float lim = kE5M2 ? kE5M2Max : kE4M3Max;
  return __builtin_fminf(__builtin_fmaxf(__builtin_ldexpf(x, -e), -lim), lim);
}

// Shared exponent of a block from its amax (>= 0): floor(log2(amax)) - emax (8 for E4M3,
// 15 for E5M2) from the binary32 exponent field, clamped to [-127, 127]; zero and
// binary32-subnormal maxima (floor(log2) <= -127) give -127.
template <bool kE5M2>
__device__ __forceinline__ int mx_shared_exponent(float amax) {
  const int eb = (int)(f2u(amax) >> 23);
  return eb == 0 ? -127 : max(eb - (kE5M2 ? 142 : 135), -127);
}

// Four elements y0..y3 (already scaled and clamped) into the element type's bytes
// 0..3 of a word (round to nearest even).
template <bool kE5M2>
__device__ __forceinline__ uint32_t mx_convert4(float y0, float y1, float y2, float y3) {
  if constexpr (kE5M2) {
    const uint32_t w = __builtin_amdgcn_cvt_pk_bf8_f32(y0, y1, 0, false);
    return __builtin_amdgcn_cvt_pk_bf8_f32(y2, y3, w, true);
  } else {
    const uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(y0, y1, 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(y2, y3, w, true);
  }
}

// Four lanes share a 32-element block: lane 4i+q holds elements [8q, 8q+8) of block i. The block
// amax is the maximum over the quad (two DPP lane swaps), each lane converts its 8 elements
// with the gfx950 fp8 conversion (round to nearest even).
struct Mx8Codes {
  u32x2 words;
  uint32_t byte;
};
template <bool kE5M2>
__device__ __forceinline__ Mx8Codes mx8_encode_quad(const u32x4 v) {
  float f[8];
  mx_unpack_bf16x8(v, f);
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = __builtin_fmaxf(a, __builtin_fabsf(f[i]));
  // quad maximum: lanes 4i..4i+3 (DPP quad_perm [1,0,3,2], then [2,3,0,1])
  a = __builtin_fmaxf(a, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, a), 0xB1, 0xF, 0xF, false)));
  a = __builtin_fmaxf(a, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, a), 0x4E, 0xF, 0xF, false)));
  const int e = mx_shared_exponent<kE5M2>(a);
  const uint32_t w0 = mx_convert4<kE5M2>(mx_scaled<kE5M2>(f[0], e), mx_scaled<kE5M2>(f[1], e),
                                         mx_scaled<kE5M2>(f[2], e), mx_scaled<kE5M2>(f[3], e));
  const uint32_t w1 = mx_convert4<kE5M2>(mx_scaled<kE5M2>(f[4], e), mx_scaled<kE5M2>(f[5], e),
                                         mx_scaled<kE5M2>(f[6], e), mx_scaled<kE5M2>(f[7], e));
  return Mx8Codes{u32x2{w0, w1}, (uint32_t)(e + 127)};
}

// ---- rowwise FP8 ----

// 8 elements of a row (one bf16x8 word) to 8 E4M3 codes under the row's scale.
__device__ __forceinline__ u32x2 encode8(const u32x4 v, float s, float r, bool corrected) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = u2f(w[i] << 16), x1 = u2f(w[i] & 0xFFFF0000u);
    y[2 * i] = corrected ? div_by_scale_unclamped(x0, s, r) : x0 / s;
    y[2 * i + 1] = corrected ? div_by_scale_unclamped(x1, s, r) : x1 / s;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(y[i], -kE4M3Max, kE4M3Max);
  uint32_t c0 = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  c0 = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c0, true);
  uint32_t c1 = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  c1 = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], c1, true);
  return u32x2{c0, c1};
}

__device__ __forceinline__ float amax8(const u32x4 v, float a) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a = __builtin_fmaxf(a, __builtin_fabsf(u2f(w[i] << 16)));
    a = __builtin_fmaxf(a, __builtin_fabsf(u2f(w[i] & 0xFFFF0000u)));
  }
  return a;
}

// Row scale s = RN(amax / 448) (1 for an all-zero row), stored by lane 0.
struct RowScale {
  float s, r;
  bool corrected;
};
__device__ __forceinline__ RowScale row_scale(float amax, float* scales, int64_t row, int lane) {
  RowScale rs;
  rs.s = amax > 0.0f ? amax / kE4M3Max : 1.0f;  // IEEE division
  if (lane == 0) scales[row] = rs.s;
  rs.r = 1.0f / rs.s;
  rs.corrected = rs.s >= 0x1p-60f;  // wave-uniform
  return rs;
}

}  // namespace
}  // namespace nvfp4
