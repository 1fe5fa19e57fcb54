// Internal launch interface between the C ABI (api.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

struct LaunchInfo {
  int num_cus;  // compute units of the current device
  int device;   // its index
};

// rows * row_bytes < 2^31 (a tile's 32-bit buffer offsets), for rows, row_bytes >= 0,
// evaluated without forming the product (which can exceed int64 for shapes the size
// checks accept, such as one row of 2^61 elements).
inline bool fits_i31(int64_t rows, int64_t row_bytes) {
  return row_bytes <= 0 || rows <= ((((int64_t)1) << 31) - 1) / row_bytes;
}

// gs_dev non-null: the global scale is read on the device from *gs_dev (clamped into
// [2^-90, 2^90], NaN read as 1) and `gs` is ignored.
hipError_t launch_quantize(const void* x, int64_t M, int64_t K, float gs, void* packed,
                           void* scales, hipStream_t stream, const LaunchInfo& dev,
                           const float* gs_dev = nullptr);

// The epilogue scale a_global * w_global as m * 2^e. When RN(a_global * w_global) is a
// normal binary32 (every realistic pair) m is that product and e = 0. Global scales in
// [2^-90, 2^90] can also multiply to anything in [2^-180, 2^180], where a single fp32
// alpha would be subnormal (precision lost) or infinite; then m is the rounded product of
// the two frexp mantissas, in [0.25, 1), e the sum of their exponents, and the epilogue
// applies 2^e with ldexp after the multiply by m.
struct Alpha {
  float m;
  int e;
};
__host__ __device__ inline Alpha split_alpha(float a, float w) {
  const float prod = a * w;
  if (prod >= 0x1p-126f && prod <= 0x1.fffffep127f) return Alpha{prod, 0};
  int ea = 0, ew = 0;
  const float ma = frexpf(a, &ea);
  const float mw = frexpf(w, &ew);
  return Alpha{ma * mw, ea + ew};
}

struct GemmProblem {
  const uint8_t* a_packed;
  const uint8_t* a_scales;
  const uint8_t* w_packed;
  const uint8_t* w_scales;
  uint16_t* out;
  int64_t M, N, K;
  float alpha;  // split_alpha(a_global, w_global): alpha * 2^alpha_exp
  // Device-resident global scales (both set, or both null): the kernel then reads both,
  // clamps each as the quantizer clamps a device-resident scale, and splits their product
  // with split_alpha; alpha and alpha_exp are unused.
  const float* a_gs_dev;
  const float* w_gs_dev;
  int alpha_exp = 0;
};

hipError_t launch_gemm(const GemmProblem& p, hipStream_t stream, const LaunchInfo& dev);

// The fused linear for short activations: the split-K GEMM quantizes its own bf16
// activations (bit-identical to launch_quantize) and, when ws_packed is set, the
// workgroups of the first weight-row tile store the codes and scales there. The GEMM
// problem's a_packed / a_scales are unused.
struct FusedQuant {
  const void* x;          // bf16 activations [M, K]
  float gs, den, rden;    // host global scale, RN(6 gs), RN(1 / RN(6 gs))
  const float* gs_dev;    // device-resident global scale instead (then gs/den/rden unused)
  uint8_t* ws_packed;     // [M, K/2] codes out, or null
  uint8_t* ws_scales;     // [M, K/16] scales out
};
bool linear_fused(int64_t M, int64_t N, int64_t K, bool aligned, int64_t cus);
hipError_t launch_linear_fused(const GemmProblem& p, const FusedQuant& fq, hipStream_t stream,
                               int64_t cus);

// The kernel launch_gemm picks for a shape (values of nvfp4_gemm_kernel in nvfp4.h), and
// the split-K workgroup shape (32a weight rows x 32b activation rows) when it splits.
struct SplitShape { int a, b; };
struct GemmPlan {
  int kernel;
  SplitShape split;
};
GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, bool aligned, int64_t cus,
                   bool allow_gemv16 = true);

// Weight rows per workgroup of the 16-row kernels (NVFP4 and W4A16): a multiple of 4 up
// to 16, the fewest that keep the grid within one workgroup per compute unit.
inline int gemv16_rows(int64_t N, int64_t cus) {
  const int64_t r = 4 * ((N + 4 * cus - 1) / (4 * cus));
  return (int)(r < 4 ? 4 : r > 16 ? 16 : r);
}

struct W4A16Problem {
  const uint16_t* x;  // bf16 [M, K]
  const uint8_t* w_packed;
  const uint8_t* w_scales;
  uint16_t* out;
  int64_t M, N, K;
  float alpha;  // the weights' global scale
};

// W4A16 kernels, in the order of the plan codes: split-K (short activations), the 288 x 192
// tile, the 256 x 256 tile, the tiles with their waves along N: 224 x 256, 128 x 256,
// 96 x 256, 128 x 128 and 64 x 128, and the 16-row kernel (at most 16 activation rows).
enum class W4A16Kernel {
  kSplitK = 0, kFit = 1, kTile256 = 2, kWide = 3, kWide128x256 = 4, kWide96x256 = 5,
  kWide128x128 = 6, kWide64x128 = 7, kGemv16 = 8
};
W4A16Kernel plan_gemm_w4a16(int64_t M, int64_t N, int64_t K, int64_t num_cus, bool aligned);
hipError_t launch_gemm_w4a16(const W4A16Problem& p, hipStream_t stream, const LaunchInfo& dev);

// MXFP8: codes/scales use GemmProblem's a_packed/a_scales/w_packed/w_scales (one byte
// per element, one E8M0 byte per 32 elements); alpha is 1. Elements are E4M3 or E5M2,
// each operand its own.
enum class MxElement { kE4M3 = 0, kE5M2 = 1 };
hipError_t launch_mx_quantize(const void* x, int64_t M, int64_t K, void* codes, void* scales,
                              hipStream_t stream, const LaunchInfo& dev, MxElement elem);
hipError_t launch_mx_gemm(const GemmProblem& p, hipStream_t stream, const LaunchInfo& dev,
                          MxElement a_elem, MxElement w_elem);
// Rowwise FP8: codes as above, scales fp32 [rows] (GemmProblem's a_scales/w_scales point
// to fp32 arrays); alpha unused.
hipError_t launch_fp8r_quantize(const void* x, int64_t M, int64_t K, void* codes, void* scales,
                                hipStream_t stream, const LaunchInfo& dev);
hipError_t launch_fp8r_gemm(const GemmProblem& p, hipStream_t stream, const LaunchInfo& dev);
hipError_t launch_mx_selftest_e4m3_exhaustive(unsigned long long* count, uint32_t* first,
                                              hipStream_t stream);
hipError_t launch_mx_selftest_e5m2_exhaustive(unsigned long long* count, uint32_t* first,
                                              hipStream_t stream);

// MXFP4: packed codes and E8M0 scale bytes in GemmProblem's a_packed/a_scales/w_packed/
// w_scales (two elements per byte, one scale byte per 32 elements).
hipError_t launch_mx4_quantize(const void* x, int64_t M, int64_t K, void* packed, void* scales,
                               hipStream_t stream, const LaunchInfo& dev);
hipError_t launch_mx4_dequantize(const void* packed, const void* scales, int64_t M, int64_t K,
                                 void* out, hipStream_t stream, const LaunchInfo& dev);
hipError_t launch_mx4_gemm(const GemmProblem& p, hipStream_t stream, const LaunchInfo& dev);
// The kernel launch_mx4_gemm picks (a value of nvfp4_mxfp4_kernel).
int plan_mx4_gemm(int64_t M, int64_t N, int64_t K, int64_t cus);
// The form of that kernel it launches: output tiles of m x n, and of the kernel for few rows its
// waves, of the others their stage buffers.
struct Mx4Form {
  int kernel, m, n, depth;
};
Mx4Form mx4_form(int64_t M, int64_t N, int64_t K, int64_t cus);
// The linear in one launch, for a few rows: the product's kernel quantizes the bf16
// activations x itself (and stores the codes and scales).
bool mx4_linear_fused(int64_t M, int64_t N, int64_t K, int64_t cus);
hipError_t launch_mx4_linear_fused(const GemmProblem& p, const void* x, void* packed, void* scales,
                                   hipStream_t stream);

// Mixture of experts (moe.hip): T tokens of width H, E experts of inner width I.
struct MoeProblem {
  const uint16_t* x;        // bf16 [T, H]
  const float* logits;      // fp32 [T, E]
  const uint8_t* w13_packed;
  const uint8_t* w13_scales;
  const uint8_t* w2_packed;
  const uint8_t* w2_scales;
  uint16_t* out;            // bf16 [T, H]
  int* ids;                 // [T, top_k]
  float* weights;           // [T, top_k]
  void* plan;               // moe_plan_bytes(T)
  uint8_t* h;               // moe_h_bytes(T, E, I, top_k): silu(gate) * up, two bf16 parts, in tiles
  float* partial;           // moe_partial_bytes(T, H)
  int64_t T, H, I;
  int E, top_k;
  bool renormalize;
  const int* given_ids;         // [T, top_k], or null: the logits are routed
  const float* given_weights;  // [T, top_k]
};
constexpr int64_t kMoeMaxExperts = 512, kMoeMaxTopK = 16, kMoeMaxTokens = (int64_t)1 << 21;
int64_t moe_plan_bytes(int64_t T);
int64_t moe_h_bytes(int64_t T, int64_t E, int64_t I, int64_t top_k);
int64_t moe_partial_bytes(int64_t T, int64_t H);
hipError_t launch_moe_router(const void* x, const void* w, int64_t T, int64_t E, int64_t H,
                             void* logits, hipStream_t stream);
hipError_t launch_moe(const MoeProblem& p, hipStream_t stream);
// The kernels launch_moe launches: who routes (0: every workgroup of the first product, 1: the plan, 2: a
// kernel of its own), whether the first product stages activations (64 rows per workgroup), of
// that the form of three workgroups per compute unit, and the second product's shares (0: the
// kernel without).
struct MoeForm {
  int routing;
  bool staged, few;
  int groups;
};
MoeForm moe_form(int64_t T, int64_t E, int64_t H, int64_t I, int64_t top_k);

// Routing to experts (moe_route.hip): logits fp32 [T, E], bias fp32 [E] or null.
struct RouteProblem {
  const float* logits;
  const float* bias;
  int* ids;        // [T, top_k]
  float* weights;  // [T, top_k]
  int64_t T;
  int E, top_k, groups, top_groups, group_best;
  bool sigmoid, renormalize;
  float scale;
};
constexpr int64_t kRouteMaxGroups = 64;
hipError_t launch_moe_route(const RouteProblem& p, hipStream_t stream);

// Low-rank adapters (lora.hip): out = y + scales[a] * B_a (A_a x), a = adapters[row].
struct LoraProblem {
  const uint16_t* y;    // bf16 [T, N]
  const uint16_t* x;    // bf16 [T, K]
  const uint16_t* a;    // bf16 [L, R, K]
  const uint16_t* b;    // bf16 [L, N, R]
  const int* adapters;  // [T]; outside [0, L): none
  const float* scales;  // [L], or null: 1
  uint16_t* out;        // bf16 [T, N]; may be y
  uint16_t* down;       // lora_down_bytes(T, N, K, R): A x, three bf16 parts
  int64_t T, N, K, L;
  int R;
};
constexpr int64_t kLoraMaxRank = 128;
int64_t lora_down_bytes(int64_t T, int64_t N, int64_t K, int64_t R);
hipError_t launch_lora(const LoraProblem& p, hipStream_t stream);

// The fused residual and norm (norm.hip). Null pointers: that part is left out.
struct NormProblem {
  const uint16_t* x;     // bf16 [M, H], the residual stream
  const uint16_t* y;     // bf16 [M, H], a branch's output
  const uint16_t* post;  // bf16 [H], the weight of the norm of y
  const uint16_t* gate;  // bf16 [groups, H]
  const uint16_t* weight;
  const uint16_t* bias;   // bf16 [H], of the norm of h
  const uint16_t* scale;  // bf16 [groups, H]
  const uint16_t* shift;  // bf16 [groups, H]
  const int* rows;        // [M], a row's group; null: M / groups rows each
  uint16_t* h;            // bf16 [M, H]; may be x
  void* out;
  void* scales;
  int64_t M, H, groups;
  float residual_scale, eps;
  int kind, format;  // nvfp4_norm_kind, nvfp4_norm_format
  float gs;          // NVFP4: the global scale
  const float* gs_dev;
};
constexpr int64_t kNormMaxWidth = 32768;
hipError_t launch_add_norm(const NormProblem& p, hipStream_t stream, const LaunchInfo& dev);

hipError_t launch_amax(const void* x, int64_t n, float* out, hipStream_t stream,
                       const LaunchInfo& dev);
// amax of x, then in place the global scale from it: RN(amax / 2688) clamped into
// [2^-90, 2^90], 1 for amax == 0.
hipError_t launch_calibrate(const void* x, int64_t n, float* gs, hipStream_t stream,
                            const LaunchInfo& dev);

// self-test support
hipError_t launch_selftest_encode(const float* y, uint8_t* hw, uint8_t* sw, int64_t n,
                                  hipStream_t stream);
hipError_t launch_selftest_encode_exhaustive(unsigned long long* count, uint32_t* first,
                                             hipStream_t stream);
hipError_t launch_selftest_division(unsigned long long* count, uint32_t* first,
                                    hipStream_t stream);
hipError_t launch_selftest_scale(const float* amax, float gs, uint8_t* code, float* d, int64_t n,
                                 hipStream_t stream);
hipError_t launch_selftest_bf16_exhaustive(unsigned long long* count, uint32_t* first,
                                           hipStream_t stream);
hipError_t launch_selftest_decode(const uint8_t* packed, const uint8_t* scales, uint16_t* hw,
                                  uint16_t* sw, int64_t nbytes, hipStream_t stream);

}  // namespace nvfp4
