// Where the MXFP4 product's kernels read their operands (mxfp4.hip): functions of sizes and
// lane numbers alone, which compile for the host as well, so that a test can evaluate every
// read of a shape against its operands' ends.
#pragma once

#include "gemm_common.hpp"

namespace nvfp4 {
namespace {

// A part of K of the tiled kernels: nst stages of 8 blocks (256 elements) from stage s0 on, of
// which nb blocks are the row's (the last part may have fewer than 8 nst).
struct Mx4Part {
  int nst, s0, nb;
};
NVFP4_HD Mx4Part mx4_part(int row_blocks, int parts, int part) {
  const int nst = ((row_blocks + 7) / 8 + parts - 1) / parts;
  const int s0 = part * nst, left = row_blocks - 8 * s0;
  return Mx4Part{nst, s0, left < 8 * nst ? left : 8 * nst};
}

// Parts that the scale reads below allow: every read starts inside its row. (One part of a
// shorter row reads its scales byte by byte.)
NVFP4_HD bool mx4_parts_ok(int row_blocks, int parts) {
  return parts == 1 ? row_blocks >= 16 : row_blocks > 16 * parts;
}

// A code load of the tiled kernels: lane l of a wave reads, of row `row` of its operand's
// window, chunk mx4_chunk(l, row) of the stage's 128 bytes. The position in the row that the
// scalar offset adds is stage * 128, so a chunk past the part's blocks has to lie past the
// window by the mask alone.
NVFP4_HD int mx4_chunk(int lane, int row) { return (lane & 7) ^ x_swz(row & 31); }
NVFP4_HD uint32_t mx4_code_voff(int row, int chunk, uint32_t pitch) {
  return (uint32_t)row * pitch + 16u * (uint32_t)chunk;
}
NVFP4_HD uint32_t mx4_code_mask(int stage, int chunk, int nb) {
  return stage * 8 + chunk >= nb ? 0x80000000u : 0u;
}

// First byte, in the row, of the 16 scale bytes that quarter (0..3) of group grp of a part
// reads. A quarter that the part's end cuts is read from 16 bytes before that end; one past it
// is read there too and not used.
NVFP4_HD int mx4_scale_at(const Mx4Part& k, int grp, int quarter) {
  const int at = 64 * grp + 16 * quarter, last = k.nb - 16;
  return 8 * k.s0 + (at < last ? at : last);
}

// The kernel for few rows: lane (q, r) reads blocks 2q + i (i = 0, 1) of group g (8 blocks) of
// a row at per-lane offset row * pitch + 32 q + 16 i, scalar offset 128 g.
NVFP4_HD uint32_t mx4_rows_voff(int row, int q, int i, int g, int row_blocks, uint32_t pitch) {
  const uint32_t past = 8 * g + 2 * q + i < row_blocks ? 0u : 0x80000000u;
  return ((uint32_t)row * pitch + 32u * (uint32_t)q + 16u * (uint32_t)i) | past;
}

}  // namespace
}  // namespace nvfp4
