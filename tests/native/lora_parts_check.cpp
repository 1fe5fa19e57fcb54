// The order of v's parts in the low-rank adapters' second product (csrc/lora_offsets.hpp), evaluated on the host: every
// chunk of a row's [upper R, middle R, lower R] is taken once, within the row, by a step whose weights are those of
// its ranks. Prints "<family> checks N violations V".
#include <stdio.h>

#include <vector>

#include "lora_offsets.hpp"

using namespace nvfp4;

int main() {
  long long checks = 0, bad = 0;
  auto expect = [&](bool ok, const char* what, int a, int b, int c) {
    ++checks;
    if (!ok && bad++ < 10) fprintf(stderr, "%s: %d %d %d\n", what, a, b, c);
  };
  for (int R = 8; R <= 128; R += 8) {
    const int steps = lora_steps(R), last = (steps + 1) / 2, held = lora_halves(R) ? steps / 2 : steps, R8 = R / 8;
    std::vector<int> seen(3 * R8, 0);
    for (int k = 0; k < steps + last; ++k)
      for (int q = 0; q < 4; ++q) {
        const int c = lora_chunk(k, q, steps, R);
        expect(c >= -1 && c < 3 * R8, "range", R, k, c);
        if (c < 0 || c >= 3 * R8) continue;
        ++seen[c];
        // the fragment that the step multiplies, as it was loaded
        const int step = k < steps ? k % held : k - steps;
        expect(step < held && (4 * step + q) % R8 == c % R8 && 4 * step + q < 2 * R8, "weights", R, k, c);
      }
    expect(lora_tile_chunks(R) == 3 * R8 * 16, "tile", R, lora_tile_chunks(R), 0);
    for (int c = 0; c < 3 * R8; ++c) expect(seen[c] == 1, "once", R, c, seen[c]);
  }
  printf("parts checks %lld violations %lld\n", checks, bad);
  return 0;
}
