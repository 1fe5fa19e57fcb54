// How the low-rank adapters' kernels (lora.hip) divide their work: functions of sizes and lane numbers
// alone, which compile for the host as well.
#pragma once

#include "codec.hpp"

namespace nvfp4 {
namespace {

// First step of K (32 elements) of split i of n.
NVFP4_HD int lora_split_begin(int steps, int i, int n) { return (int)((int64_t)steps * i / n); }

// Column of the output, within a wave's 64, of row r (0..15) of its fragment i (0..3) of B: a lane's results
// of fragment i are rows 4q .. 4q + 3, columns 16q + 4i .. + 3.
NVFP4_HD int lora_column(int r, int i) { return 16 * (r >> 2) + 4 * i + (r & 3); }

// Parts of K: as many as bring the first product's workgroups to 256, at least 8 steps each.
NVFP4_HD int64_t lora_splits(int64_t T, int64_t K) {
  const int64_t tiles = (T + 15) / 16, most = (K + 255) / 256, want = (256 + tiles - 1) / (tiles > 0 ? tiles : 1);
  return want < 1 ? 1 : want > most ? most : want;
}

// Workgroups that share the distinct adapters of 16 rows.
NVFP4_HD int64_t lora_deal(int64_t T) { return T <= 256 ? (T < 16 ? (T > 0 ? T : 1) : 16) : 1; }

}  // namespace
}  // namespace nvfp4
