// Every operand read of the MXFP4 product's kernels (csrc/mx4_offsets.hpp), evaluated on the
// host over ragged shapes: no read that passes its window's range check lies outside the
// operand or its row, every 16-byte chunk of every real row is read from its own address, and
// all 16 bytes of every scale read lie in its row. Prints "<family> reads N violations V".
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "mx4_offsets.hpp"

using namespace nvfp4;

static long long reads, bad;
static void expect(bool ok, const char* what, long long a, long long b, long long c) {
  ++reads;
  if (!ok && bad++ < 10) fprintf(stderr, "%s: %lld %lld %lld\n", what, a, b, c);
}

// One operand of `total` rows, tiles of `tile` rows starting at row0, K parts.
static void tiled(int64_t total, int tile, int64_t K, int parts, int nbuf) {
  const int nbr = (int)(K / 32);
  const uint32_t pitch = (uint32_t)(K / 2);
  if (!mx4_parts_ok(nbr, parts)) return;
  const int64_t starts[2] = {0, (total - 1) / tile * tile};
  for (int64_t row0 : starts) {
    const int64_t rows = total - row0 < tile ? total - row0 : tile;
    const uint32_t window = window_bytes(row0, row0 + rows, pitch);
    std::vector<char> seen((size_t)rows * nbr, 0);
    for (int part = 0; part < parts; ++part) {
      const Mx4Part k = mx4_part(nbr, parts, part);
      for (int stage = 0; stage < k.nst + nbuf; ++stage)
        for (int wave = 0; wave < 4; ++wave)
          for (int lane = 0; lane < 64; ++lane)
            for (int j = 0; j < tile / 32; ++j) {
              const int lrow = 8 * wave + lane / 8, row = lrow + 32 * j;
              const int chunk = mx4_chunk(lane, lrow);
              const uint32_t voff = (mx4_code_voff(lrow, chunk, pitch) | mx4_code_mask(stage, chunk, k.nb)) +
                                    (uint32_t)(32 * j) * pitch;
              if (voff >= window) continue;
              const int64_t at = (int64_t)voff + (int64_t)(k.s0 + stage) * 128;
              const int block = 8 * (k.s0 + stage) + chunk;
              expect(row < rows && block < nbr && at == (int64_t)row * pitch + 16 * block, "code", row, block, at);
              if (row < rows && block < nbr) seen[(size_t)row * nbr + block] = 1;
            }
      for (int grp = 0; grp <= (k.nst - 1) / 8; ++grp)
        for (int quarter = 0; quarter < 4; ++quarter) {
          const int at = mx4_scale_at(k, grp, quarter);
          expect(at >= 0 && at + 16 <= nbr, "scale", part, grp, at);
        }
    }
    for (size_t i = 0; i < seen.size(); ++i) expect(seen[i], "chunk never read", (long long)i, K, parts);
  }
}

static void few_rows(int64_t total, int tile, int64_t K, int waves) {
  const int nbr = (int)(K / 32), ng = (nbr + 7) / 8;
  const uint32_t pitch = (uint32_t)(K / 2);
  const int64_t row0 = (total - 1) / tile * tile;
  const int rows = (int)(total - row0);
  const uint32_t window = window_bytes(row0, row0 + rows, pitch);
  std::vector<char> seen((size_t)rows * nbr, 0);
  for (int g = 0; g < ng + 4 * waves; ++g)
    for (int lane = 0; lane < 64; ++lane)
      for (int a = 0; a < tile / 16; ++a)
        for (int i = 0; i < 2; ++i) {
          const int q = lane / 16, r = 16 * a + lane % 16, row = r < rows ? r : rows - 1;
          const uint32_t voff = mx4_rows_voff(row, q, i, g, nbr, pitch);
          if (voff >= window) continue;
          const int block = 8 * g + 2 * q + i;
          const int64_t at = (int64_t)voff + 128ll * g;
          expect(block < nbr && at == (int64_t)row * pitch + 16 * block, "row", row, block, at);
          if (block < nbr) seen[(size_t)row * nbr + block] = 1;
        }
  for (size_t i = 0; i < seen.size(); ++i) expect(seen[i], "chunk never read", (long long)i, K, waves);
}

int main() {
  const int64_t rows[] = {1, 7, 31, 64, 65, 130, 255, 257, 300};
  const int64_t ks[] = {32, 64, 96, 256, 288, 480, 512, 544, 640, 768, 992, 1024, 1056, 1280, 1440, 2048, 2080, 2848, 4096, 4128};
  int failed = 0;
  for (int64_t n : rows)
    for (int64_t K : ks) {
      for (int tile : {64, 128, 256}) {
        tiled(n, tile, K, 1, 4);
        if (tile == 64) tiled(n, tile, K, 2, 3);
      }
    }
  printf("tiles reads %lld violations %lld\n", reads, bad);
  failed += bad != 0;
  reads = bad = 0;
  for (int64_t n : rows)
    for (int64_t K : ks)
      for (int tile : {16, 32, 64}) few_rows(n, tile, K, 16);
  printf("rows reads %lld violations %lld\n", reads, bad);
  failed += bad != 0;
  return failed;
}
