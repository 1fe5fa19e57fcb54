// Every access of the mixture-of-experts kernels to weights, activations and h (csrc/moe_offsets.hpp),
// evaluated on the host over widths of one block to many: none lies outside its operand, every
// block of every real row is taken once and from its own address, and what the first product
// writes of h is what the second reads. Prints "<family> accesses N violations V".
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "moe_offsets.hpp"

using namespace nvfp4;

static long long accesses, bad;
static void expect(bool ok, const char* what, long long a, long long b, long long c) {
  ++accesses;
  if (!ok && bad++ < 10) fprintf(stderr, "%s: %lld %lld %lld\n", what, a, b, c);
}
static int report(const char* family) {
  printf("%s accesses %lld violations %lld\n", family, accesses, bad);
  const int failed = bad != 0;
  accesses = bad = 0;
  return failed;
}
static int units(int nb) { return (nb + kUnit - 1) / kUnit; }
static void once(const std::vector<int>& seen, const char* what, int nb) {
  for (size_t i = 0; i < seen.size(); ++i) expect(seen[i] == 1, what, (long long)i, seen[i], nb);
}

// 16 rows of nb blocks, which may be all that their buffer holds.
static void weights(int nb) {
  const int64_t codes = 16ll * 16 * nb, scales = 16ll * nb;
  std::vector<int> code(16 * nb, 0), scale(16 * nb, 0);
  for (int u = 0; u < units(nb); ++u)
    for (int lane = 0; lane < 64; ++lane) {
      const int b0 = unit_start(u, nb), row = lane >> 2, part = lane & 3;
      for (int g = 0; g < 4; ++g) {
        const int block = b0 + 4 * g + part;
        const int64_t at = 16ll * b0 + (nb >= kUnit ? weight_code_at(lane, nb) + 64u * g : short_code_at(lane, g, nb));
        expect(at >= 0 && at + 16 <= codes, "code out of the rows", lane, u, nb);
        // blocks that the unit has not are cleared where unit_cut says so
        expect(unit_has(u, block, nb) || unit_cut(u, nb), "block neither used nor cleared", block, u, nb);
        if (!unit_has(u, block, nb)) continue;
        expect(at == 16ll * nb * row + 16ll * block, "code", at, block, nb);
        ++code[row * nb + block];
      }
      if (nb >= kUnit) {
        const int64_t at = b0 + (int64_t)weight_scale_at(lane, nb);
        expect(at >= 0 && at + 4 <= scales, "scale out of the rows", lane, u, nb);
      }
      for (int i = 0; i < 4; ++i) {
        const int block = b0 + 4 * part + i;
        const int64_t at = b0 + (nb >= kUnit ? (int64_t)weight_scale_at(lane, nb) + i : (int64_t)short_scale_at(lane, i, nb));
        expect(at >= 0 && at < scales, "scale byte out of the rows", lane, u, nb);
        if (!unit_has(u, block, nb)) continue;
        expect(at == (int64_t)nb * row + block, "scale", at, block, nb);
        ++scale[row * nb + block];
      }
    }
  once(code, "code taken", nb);
  once(scale, "scale taken", nb);
}

// Straight into registers: x (rows of 64 nb bytes) and a tile of h (16 columns in one window).
static void activations(int nb, int rows) {
  for (int form = 0; form < 2; ++form) {
    const int columns = form == 0 ? rows : 16, stride = form == 0 ? 16 : 256;
    const int64_t window = form == 0 ? 64ll * nb * rows : 1024ll * nb;
    std::vector<int> seen((size_t)columns * nb * 4, 0);
    for (int col = 0; col < columns; ++col)
      for (int u = 0; u < units(nb); ++u)
        for (int q = 0; q < 4; ++q)
          for (int i = 0; i < kUnit; ++i) {
            const int64_t start = form == 0 ? 64ll * nb * col : 16ll * col;
            const int64_t at = (uint32_t)((uint32_t)start + act_first(stride, u, nb, q) + act_step(stride, i));
            const int block = unit_start(u, nb) + 4 * (i >> 2) + q;
            expect(unit_has(u, block, nb) || unit_cut(u, nb), "activations neither used nor cleared", block, u, nb);
            if (!unit_has(u, block, nb)) continue;  // cleared; past the window nothing is read
            expect(at + 16 <= window, "activations past the window", at, block, nb);
            expect(at == start + (int64_t)stride * (4 * block + (i & 3)), "activations", at, block, nb);
            ++seen[((size_t)col * nb + block) * 4 + (i & 3)];
          }
    once(seen, "chunk of activations taken", nb);
  }
}

static void staged(int nb, int rows) {
  const int64_t window = 64ll * nb * rows;
  std::vector<int> seen((size_t)rows * nb * 4, 0);
  for (int slot = 0; slot < rows; ++slot)
    for (int u = 0; u < units(nb); ++u)
      for (int lane = 0; lane < 64; ++lane) {
        const int chunk = lane ^ (slot % 16);
        const uint32_t voff = stage_voff((uint32_t)(64 * nb * slot), chunk, u, nb);
        const int block = unit_start(u, nb) + (chunk >> 2);
        expect((voff < window) == unit_has(u, block, nb), "staged chunk of another unit", block, u, nb);
        if (voff >= window) continue;
        const int64_t at = (int64_t)voff + stage_soff(u, nb);
        expect(at == 64ll * nb * slot + 64ll * block + 16 * (chunk & 3) && at + 16 <= window, "staged", at, block, nb);
        ++seen[((size_t)slot * nb + block) * 4 + (chunk & 3)];
      }
  once(seen, "staged chunk taken", nb);
}

// h of one expert of so many slots: its writes, and the two forms of its reads.
static void h(int nb, int slots) {
  const int64_t I = 32ll * nb, tile = 32 * I, tiles = (slots + kTileSlots - 1) / kTileSlots;
  std::vector<int> written((size_t)(tiles * tile / 8), 0), read((size_t)slots * nb * 4 * 2, 0);
  for (int n = 0; n < slots; ++n)
    for (int64_t i = 0; i < I; i += 4)
      for (int part = 0; part < 2; ++part) {
        const int64_t at = h_at(n, i, I) + 16 * part;
        expect(at >= 0 && at + 8 <= tiles * tile && at % 8 == 0, "h written out of its tiles", n, i, nb);
        if (at >= 0 && at + 8 <= tiles * tile) expect(written[(size_t)(at / 8)]++ == 0, "h written twice", n, i, nb);
      }
  for (int c = 0; c < tiles; ++c)
    for (int u = 0; u < units(nb); ++u)
      for (int b = 0; b < kUnit; ++b)
        for (int lane = 0; lane < 64; ++lane) {
          const int slot = kTileSlots * c + ((lane & 15) >> 1), part = lane & 1, block = unit_start(u, nb) + b;
          const uint32_t voff = h_voff(lane, c, slots, u, b, nb);
          expect((voff < tile) == (slot < slots && unit_has(u, block, nb)), "h read that is not there", lane, block, nb);
          if (voff >= tile) continue;
          const int64_t at = c * tile + voff + h_soff(u, b, nb);
          expect(at + 16 <= (c + 1) * tile, "h read out of its tile", at, block, nb);
          expect(at == h_at(slot, 32ll * block + 8 * (lane >> 4), I) + 16 * part, "h read", at, block, nb);
          ++read[(((size_t)slot * nb + block) * 4 + (lane >> 4)) * 2 + part];
        }
  once(read, "h taken", nb);
  for (int n = 0; n < slots && n < kTileSlots; ++n)  // the second product of few tokens, from one tile
    for (int block = 0; block < nb; ++block)
      for (int i = 0; i < 4; ++i)
        for (int part = 0; part < 2; ++part)
          expect(16 * (2 * n + part) + 256 * (4 * block + i) == h_at(n, 32ll * block + 8 * i, I) + 16 * part, "h column", n, block, nb);
}

static void tiles(int E, int slots) {
  for (int turn = 0; turn < 200; ++turn) {
    std::vector<int> count(E, 0);
    const int reach = 1 + rand() % E;
    for (int s = 0; s < slots; ++s) ++count[rand() % (turn % 2 ? reach : E)];
    int64_t need = 0;
    for (int c : count) need += (c + kTileSlots - 1) / kTileSlots;
    expect(need <= moe_tiles(slots, E), "tiles", need, slots, E);
  }
  std::vector<int> worst(E, 0);  // every expert one slot past a tile, as far as slots go
  int64_t need = 0;
  for (int e = 0, left = slots; e < E && left > 0; ++e) {
    const int take = left < kTileSlots + 1 ? left : kTileSlots + 1;
    need += (take + kTileSlots - 1) / kTileSlots;
    left -= take;
  }
  expect(need <= moe_tiles(slots, E), "tiles", need, slots, E);
}

int main() {
  const int widths[] = {1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 18, 19, 20, 31, 32, 33, 44, 45, 48, 63, 64, 65, 127, 128, 129, 131};
  int failed = 0;
  for (int nb : widths) weights(nb);
  weights(1 << 15);
  failed += report("weights");
  for (int nb : widths)
    for (int rows : {1, 2, 5, 16, 64}) activations(nb, rows);
  failed += report("activations");
  for (int nb : widths)
    for (int rows : {1, 3, 16, 17, 64}) staged(nb, rows);
  staged(1 << 15, 64);
  failed += report("staged");
  for (int nb : widths)
    for (int slots : {1, 2, 7, 8, 9, 15, 16, 17, 33, 64}) h(nb, slots);
  failed += report("h");
  for (int E : {1, 2, 8, 60, 128, 512})
    for (int slots : {1, 8, 9, 64, 100, 512, 1024}) tiles(E, slots);
  failed += report("tiles");
  return failed;
}
