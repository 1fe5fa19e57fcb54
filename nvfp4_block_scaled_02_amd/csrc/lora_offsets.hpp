// How the low-rank adapters' kernels (lora.hip) divide their work: functions of sizes and lane numbers
// alone, which compile for the host as well.
#pragma once

#include "codec.hpp"

namespace nvfp4 {
namespace {

// Column of the output, within a wave's 64, of row r (0..15) of its fragment i (0..3) of B: a lane's results
// of fragment i are rows 4q .. 4q + 3, columns 16q + 4i .. + 3.
NVFP4_HD int lora_column(int r, int i) { return 16 * (r >> 2) + 4 * i + (r & 3); }

// The three parts of v along the matrix instruction's K. Steps (four chunks of 8 elements) of the upper and
// the middle parts: chunk c of 2R is chunk c % (R / 8) of the upper parts, then of the middle. Whether step
// k multiplies the same rows of B as step k - R / 32: where R is a multiple of 32. The lower parts begin a
// step of their own.
NVFP4_HD bool lora_halves(int R) { return R % 32 == 0; }
NVFP4_HD int lora_steps(int R) { return (R + 15) / 16; }
// v of a tile of 16 rows: chunks of [upper R, middle R, lower R], of each chunk all rows. How many times 16 bytes.
NVFP4_HD constexpr int lora_tile_chunks(int R) { return 3 * (R / 8) * 16; }
// Chunk that lanes 16 q and on take in step k, `steps` being lora_steps(R); -1: none.
NVFP4_HD int lora_chunk(int k, int q, int steps, int R) {
  const int lower = 4 * (k - steps) + q;
  if (k < steps) return 4 * k + q < R / 4 ? 4 * k + q : -1;
  return lower < R / 8 ? R / 4 + lower : -1;
}

// Staging a unit of kC chunks (16 bytes each) of a row: the k-th load of 64 lanes takes rows
// k * 64 / kC and on, lane l the chunk that its slot l % kC holds of row k * 64 / kC + l / kC. Per-lane
// offset from row `first` of the operand on (chunks past the row lie past any window); the unit
// itself is in the scalar offset.
template <int kC>
NVFP4_HD uint32_t lora_stage_voff(int lane, int k, int first, uint32_t pitch, int unit, int chunks) {
  const int row = k * (64 / kC) + lane / kC, chunk = (lane % kC) ^ (row & 15);
  return ((uint32_t)(first + row) * pitch + 16u * (uint32_t)chunk) | (unit * kC + chunk < chunks ? 0u : 0x80000000u);
}

// Which of n neighbours a workgroup takes: consecutive workgroups go to the 8 XCDs in turn, and each XCD
// gets neighbours, which mostly share an adapter, for its own level-2 cache. (The first n % 8 XCDs
// have one more.)
NVFP4_HD int64_t lora_neighbour(int64_t i, int64_t n) {
  const int64_t xcd = i % 8, each = n / 8, more = n % 8;
  return xcd * each + (xcd < more ? xcd : more) + i / 8;
}

// The first product's workgroup i of n: its tile of rows and its first rank, `ranks` of them. The parts of a
// tile's ranks are neighbours, so that x comes from memory for one of them.
struct LoraPart {
  int64_t tile;
  int rank;
};
NVFP4_HD LoraPart lora_part(uint32_t i, uint32_t n, int R, int ranks) {
  const uint32_t parts = (uint32_t)((R + ranks - 1) / ranks), at = (uint32_t)lora_neighbour(i, n);
  return LoraPart{(int64_t)(at / parts), (int)(at % parts) * ranks};
}

// What a launch takes, by sizes alone (how many adapters the rows have is not known).
//
// The first product in the second's kernel: up to 32 ranks, where repeating it for every 512 columns costs
// less than a second launch (graph of 17 rows of their own adapters, K 4096, N 4096, 8.0 us against
// 9.8; but 48 rows 16.2 against 10.8). One fragment of ranks per workgroup up to 48 ranks (2000 rows of
// rank 48 14.6 against 17.1 for two) and where that makes no more than 128 workgroups (450 rows of rank
// 64 12.1, 12.5; 600 13.5, 12.3); two above, or for many rows all at once (1999 rows of rank 64 20.1,
// 18.9, 38.5 for all; 8192 36.7, 35.3, 34.1; 16384 of rank 128 131, 128, 85). Tiles whose adapters are
// dealt out, up to 1024 workgroups: 48 rows of rank 16 48.7, dealt to 16 11.9. The second product's
// workgroups: 512, two to a compute unit, of up to 16 tiles each (both products, 8192 rows of rank 64 into
// 4096: 8 tiles 69.6, 12 76.2, 16 66.4, 24 79.6).
//
// The form of the first product: within the second's kernel, with one or two fragments of 16 ranks
// per tile of rows, or for many rows at once.
enum class LoraDown { kFused, kNarrow, kPair, kWide };
struct LoraForm {
  LoraDown down;
  int deal;      // its workgroups that share the distinct adapters of a tile of 16 rows
  int up_deal;   // the second product's
  int up_tiles;  // tiles of 16 rows per workgroup of the second product
  bool passing;  // whether its y and out leave the caches alone (32 MB of y on)
};
NVFP4_HD int64_t lora_clamp(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }
NVFP4_HD LoraForm lora_form(int64_t T, int64_t N, int64_t K, int64_t R) {
  const int64_t tiles = (T + 15) / 16, slices = (N + 511) / 512, parts = (R + 15) / 16, most = T < 16 ? T : 16;
  LoraForm f;
  if (tiles < 1 || slices < 1) return LoraForm{LoraDown::kFused, 1, 1, 1, false};
  if (R <= 32 && (tiles * slices <= 16 || (slices == 1 && tiles <= 64)))
    return LoraForm{LoraDown::kFused, (int)lora_clamp(256 / (tiles * slices), 1, most), 1, 1, false};
  f.down = R <= 48 || tiles * parts <= 128 ? LoraDown::kNarrow : T <= 4096 ? LoraDown::kPair : LoraDown::kWide;
  f.deal = f.down == LoraDown::kWide ? 1 : (int)lora_clamp(1024 / (tiles * parts), 1, most);
  const int64_t work = tiles * ((N + 255) / 256);
  f.up_deal = (int)lora_clamp(512 / work, 1, most);
  f.up_tiles = (int)lora_clamp((work + 511) / 512, 1, 16);
  f.passing = T * N >= (int64_t)1 << 24;
  return f;
}

}  // namespace
}  // namespace nvfp4
