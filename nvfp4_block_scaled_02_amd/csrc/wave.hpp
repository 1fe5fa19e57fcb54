// Reductions over a wave of 64 lanes.
#pragma once

#include "codec.hpp"

namespace nvfp4 {
namespace {

// Reductions over a wave in the vector unit (data-parallel primitives: a shift within rows of
// 16 lanes, then broadcasts across rows); the result is uniform.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_or_zero<0x111, 0xF>(v));  // row_shr 1, 2, 4, 8
  v = max(v, dpp_or_zero<0x112, 0xF>(v));
  v = max(v, dpp_or_zero<0x114, 0xF>(v));
  v = max(v, dpp_or_zero<0x118, 0xF>(v));
  v = max(v, dpp_or_zero<0x142, 0xA>(v));  // row_bcast 15 into rows 1 and 3
  v = max(v, dpp_or_zero<0x143, 0xC>(v));  // row_bcast 31 into rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += u2f(dpp_or_zero<0x111, 0xF>(f2u(v)));
  v += u2f(dpp_or_zero<0x112, 0xF>(f2u(v)));
  v += u2f(dpp_or_zero<0x114, 0xF>(f2u(v)));
  v += u2f(dpp_or_zero<0x118, 0xF>(f2u(v)));
  v += u2f(dpp_or_zero<0x142, 0xA>(f2u(v)));
  v += u2f(dpp_or_zero<0x143, 0xC>(f2u(v)));
  return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(v), 63));
}

}  // namespace
}  // namespace nvfp4
