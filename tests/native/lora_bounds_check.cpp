// The division of the low-rank adapters' work (csrc/lora_offsets.hpp), evaluated on the host: every load
// of a stage reads its own chunk of its own row or nothing, a stage holds every chunk of its rows
// once, output columns and neighbours are permutations, and a launch's grid and tiles lie within what
// the kernels and the device take. Prints "<family> checks N violations V".
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "lora_offsets.hpp"

using namespace nvfp4;

static long long checks, bad;
static void expect(bool ok, const char* what, long long a, long long b, long long c) {
  ++checks;
  if (!ok && bad++ < 10) fprintf(stderr, "%s: %lld %lld %lld\n", what, a, b, c);
}
static void family(const char* name) {
  printf("%s checks %lld violations %lld\n", name, checks, bad);
  checks = bad = 0;
}

// `rows` rows of K elements, staged as `tile` (a multiple of 16) of them, units of kC chunks.
template <int kC>
static void staged(int rows, int tile, int64_t K) {
  const uint32_t pitch = (uint32_t)(K * 2), window = (uint32_t)rows * pitch;
  const int chunks = (int)(K / 8), units = (chunks + kC - 1) / kC;
  std::vector<char> seen((size_t)rows * chunks, 0);
  const int shown[3] = {0, units - 1, units + 1};  // (the last: past the row, as a stage ahead may be)
  for (int s = 0; s < 3; ++s) {
    const int u = shown[s];
    if (s == 1 && u == 0) continue;
    std::vector<char> slot((size_t)tile * kC, 0);
    for (int k = 0; k < tile * kC / 64; ++k)
      for (int lane = 0; lane < 64; ++lane) {
        const int row = k * (64 / kC) + lane / kC, c = (lane % kC) ^ (row & 15);
        slot[(size_t)row * kC + lane % kC] += 1;
        const uint32_t voff = lora_stage_voff<kC>(lane, k, 0, pitch, u, chunks);
        const bool there = row < rows && u * kC + c < chunks;
        expect((voff < window) == there, "in range", k, lane, u);
        if (voff >= window) continue;
        const int64_t at = (int64_t)voff + (int64_t)u * (16 * kC);
        expect(at == (int64_t)row * pitch + 16 * (u * kC + c) && at + 16 <= (int64_t)window, "address", k, lane, at);
        if (there) seen[(size_t)row * chunks + u * kC + c] += 1;
      }
    for (size_t i = 0; i < slot.size(); ++i) expect(slot[i] == 1, "slot", (long long)i, u, slot[i]);
    for (int r = 0; r < rows; ++r)
      for (int c = u * kC; c < (u + 1) * kC && c < chunks; ++c) expect(seen[(size_t)r * chunks + c] == 1, "chunk", r, c, u);
  }
}

int main() {
  for (int64_t K : {8, 16, 72, 120, 128, 136, 256, 264, 520, 1000, 4096, 4104, 1 << 20})
    for (int rows : {1, 3, 15, 16}) {
      staged<16>(rows, 16, K);
      staged<32>(rows, 16, K);
      staged<16>(rows, 32, K);
      if (K <= 4104) staged<16>(4 * rows, 64, K);
    }
  family("staged");

  std::vector<int> columns(64, 0);
  for (int r = 0; r < 16; ++r)
    for (int i = 0; i < 4; ++i) {
      const int c = lora_column(r, i);
      expect(c >= 0 && c < 64, "column", r, i, c);
      if (c >= 0 && c < 64) ++columns[c];
      // what a lane stores: rows 4q .. 4q + 3 of fragment i, columns 16q + 4i on
      expect(c == 16 * (r / 4) + 4 * i + r % 4, "order", r, i, c);
    }
  for (int c = 0; c < 64; ++c) expect(columns[c] == 1, "once", c, columns[c], 0);
  family("columns");

  for (int64_t n : {1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 1000, 4099}) {
    std::vector<int> at(n, 0);
    for (int64_t i = 0; i < n; ++i) {
      const int64_t k = lora_neighbour(i, n);
      expect(k >= 0 && k < n, "neighbour", i, n, k);
      if (k >= 0 && k < n) ++at[k];
    }
    for (int64_t i = 0; i < n; ++i) expect(at[i] == 1, "once", i, n, at[i]);
  }
  // the first product's workgroups: every part of every tile once
  for (int tiles : {1, 2, 7, 8, 125, 4099})
    for (int R : {8, 16, 24, 64, 120, 128})
      for (int ranks : {16, 32, 64}) {
        const int parts = (R + ranks - 1) / ranks;
        std::vector<int> seen((size_t)tiles * parts, 0);
        for (int i = 0; i < tiles * parts; ++i) {
          const LoraPart at = lora_part((uint32_t)i, (uint32_t)(tiles * parts), R, ranks);
          expect(at.tile >= 0 && at.tile < tiles && at.rank >= 0 && at.rank < R && at.rank % ranks == 0, "part", i, at.tile, at.rank);
          if (at.tile >= 0 && at.tile < tiles && at.rank >= 0 && at.rank < R) ++seen[(size_t)at.tile * parts + at.rank / ranks];
        }
        for (size_t i = 0; i < seen.size(); ++i) expect(seen[i] == 1, "part once", (long long)i, R, ranks);
      }
  family("neighbours");

  for (int64_t T : {1, 2, 15, 16, 17, 48, 255, 256, 257, 1000, 1024, 1025, 4096, 4097, 65536, 1 << 20, 1 << 21})
    for (int64_t N : {1, 8, 255, 512, 513, 1001, 4096, 14336, 1 << 20})
      for (int64_t R = 8; R <= 128; R += 8) {
        const LoraForm f = lora_form(T, N, 64, R);
        const int64_t tiles = (T + 15) / 16, most = 65535;
        expect(f.deal >= 1 && f.deal <= 16 && f.up_deal >= 1 && f.up_deal <= 16, "deal", T, N, f.deal);
        expect(f.up_tiles >= 1 && f.up_tiles <= 16, "tiles", T, N, f.up_tiles);
        expect(f.down != LoraDown::kFused || (R <= 32 && tiles <= most), "fused", T, N, R);
        expect(f.down != LoraDown::kWide || f.deal == 1, "wide", T, N, R);
        expect((tiles + f.up_tiles - 1) / f.up_tiles <= most, "grid", T, N, f.up_tiles);
        expect(16 * lora_steps((int)R) >= R && 16 * (lora_steps((int)R) - 1) < R, "steps", R, 0, 0);
        // step k of a rank that is a multiple of 32 takes the fragments of step k - R / 32
        if (lora_halves((int)R)) expect(lora_steps((int)R) % 2 == 0 && 4 * (lora_steps((int)R) / 2) == R / 8, "halves", R, 0, 0);
      }
  family("forms");
  return 0;
}
