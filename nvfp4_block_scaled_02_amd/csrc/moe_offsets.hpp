// Where the mixture-of-experts kernels (moe.hip) read their operands and keep h: functions of sizes
// and lane numbers alone, which compile for the host as well, so that a test can evaluate every
// access of a shape against its buffers' ends.
#pragma once

#include "gemm_common.hpp"

namespace nvfp4 {
namespace {

// ---- units of K ----
//
// K goes by units of 16 blocks (512 elements). Unit u of a row of nb blocks starts at block max(min(16 u,
// nb - 16), 0), so that its 16 scale bytes lie in the row. Blocks before 16 u were the unit
// before's; a row of fewer than 16 blocks is one unit, and has no blocks past nb.
constexpr int kUnit = 16;  // blocks
NVFP4_HD int unit_start(int u, int nb) {
  const int s = kUnit * u < nb - kUnit ? kUnit * u : nb - kUnit;
  return s > 0 ? s : 0;
}
NVFP4_HD bool unit_cut(int u, int nb) { return kUnit * u + kUnit > nb; }
// Whether block b (of the row) is one that unit u multiplies.
NVFP4_HD bool unit_has(int u, int b, int nb) { return b >= kUnit * u && b < nb; }

// ---- weights: a unit of 16 rows ----
//
// Lane l reads row l / 4, of every four blocks the block l % 4, and of the 16 scale bytes the dword l % 4:
// offsets from block unit_start of the first row. Codes of blocks 4g .. 4g + 3 lie 64 g on. Rows of
// fewer than 16 blocks: the last block and byte for those that a row has not.
NVFP4_HD uint32_t weight_code_at(int lane, int nb) {
  return (uint32_t)(lane >> 2) * (16u * (uint32_t)nb) + 16u * (uint32_t)(lane & 3);
}
NVFP4_HD uint32_t weight_scale_at(int lane, int nb) {
  return (uint32_t)(lane >> 2) * (uint32_t)nb + 4u * (uint32_t)(lane & 3);
}
NVFP4_HD uint32_t short_code_at(int lane, int g, int nb) {
  const int b = 4 * g + (lane & 3);
  return 16u * ((uint32_t)(lane >> 2) * (uint32_t)nb + (uint32_t)(b < nb - 1 ? b : nb - 1));
}
// Byte i of the dword.
NVFP4_HD uint32_t short_scale_at(int lane, int i, int nb) {
  const int b = 4 * (lane & 3) + i;
  return (uint32_t)(lane >> 2) * (uint32_t)nb + (uint32_t)(b < nb - 1 ? b : nb - 1);
}

// ---- activations ----
//
// Straight into registers: entry i (0..15) of a lane of quarter q, of a column whose 16-byte chunks are
// `stride` bytes apart: act_first + act_step bytes from the column's start.
NVFP4_HD uint32_t act_first(int stride, int u, int nb, int q) {
  return (uint32_t)(4 * stride) * (uint32_t)(unit_start(u, nb) + q);
}
NVFP4_HD uint32_t act_step(int stride, int i) { return (uint32_t)stride * (uint32_t)(16 * (i >> 2) + (i & 3)); }

// Staged in LDS: a lane's chunk (0..63) of a unit of the row at byte `start`. Per-lane offset (blocks
// that are not the unit's lie past any window), and the scalar one that is added to it.
NVFP4_HD uint32_t stage_voff(uint32_t start, int chunk, int u, int nb) {
  return (start + 16u * (uint32_t)chunk) | (unit_has(u, unit_start(u, nb) + (chunk >> 2), nb) ? 0u : 0x80000000u);
}
NVFP4_HD uint32_t stage_soff(int u, int nb) { return (uint32_t)unit_start(u, nb) * 64u; }

// ---- h ----
//
// Tiles of 8 slots of one expert, column 2n the n-th slot's upper parts, 2n + 1 its lower: [tile][16-byte
// chunk of I][column][16 bytes].
constexpr int kTileSlots = 8;
// Tiles that so many slots can need: one per expert reached and one more per 8 slots.
NVFP4_HD int64_t moe_tiles(int64_t slots, int64_t E) { return (slots < E ? slots : E) + slots / kTileSlots; }
// An expert's n-th slot's element i, upper part, from the expert's first tile; the lower lies 16 bytes on.
NVFP4_HD int64_t h_at(int n, int64_t i, int64_t I) {
  return (int64_t)(n / kTileSlots) * (32 * I) + ((i >> 3) * 16 + 2 * (n % kTileSlots)) * 16 + 2 * (i & 7);
}
// A lane's 16 bytes of block b (0..15) of unit u of tile c of an expert with so many slots: per-lane offset
// (columns that are not there and blocks that are not the unit's lie past any window), scalar offset.
NVFP4_HD uint32_t h_voff(int lane, int c, int slots, int u, int b, int nb) {
  const bool there = kTileSlots * c + ((lane & 15) >> 1) < slots && unit_has(u, unit_start(u, nb) + b, nb);
  return 16u * (uint32_t)lane | (there ? 0u : 0x80000000u);
}
NVFP4_HD int h_soff(int u, int b, int nb) { return (unit_start(u, nb) + b) * 1024; }

}  // namespace
}  // namespace nvfp4
