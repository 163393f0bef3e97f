// Host check of the streaming statistics' split: the list of a vocabulary row is the one of the CTA and
// segment that worked on it, and any 32-bit value, also none that a row has, names a list within
// bounds (after a wait that ran out the join reads ids that this call did not write).
#include <cstdio>

#include "stats.cuh"

using namespace dpo;

int main() {
  const int shapes[][2] = {{1, 1}, {9, 2}, {1000, 125}, {2000, 148}, {32000, 148}, {128256, 148},
                           {151936, 148}, {1 << 24, 148}, {151936, 16}};
  for (const auto& s : shapes) {
    const int V = s[0], ctas = s[1];
    const int tiles = (V + kSRows * ctas - 1) / (kSRows * ctas);
    const int rows = (V + ctas * tiles - 1) / (ctas * tiles);
    const StreamSplit split{V, ctas, rows};
    auto check = [&](int v, int got) {
      if (got >= 0 && got < ctas * kSSegs) return true;
      std::printf("V = %d, %d CTAs: row %d gives list %d\n", V, ctas, v, got);
      return false;
    };
    for (int cta = 0; cta < ctas; ++cta)
      for (int t = 0; t < split.tiles(cta); ++t)
        for (int r = 0; r < rows; ++r) {
          const int v = split.first(cta, t) + r;
          if (v < V && split.list_of(v) != cta * kSSegs + r / kSegRows) {
            std::printf("V = %d, %d CTAs: row %d is not in its list\n", V, ctas, v);
            return 1;
          }
        }
    unsigned x = 12345u;
    for (int i = 0; i < 200000; ++i) {
      x = x * 1664525u + 1013904223u;
      if (!check(static_cast<int>(x), split.list_of(static_cast<int>(x)))) return 1;
    }
    for (int v : {-1, -500000000, INT32_MIN, INT32_MAX, V, static_cast<int>(0xABABABABu)})
      if (!check(v, split.list_of(v))) return 1;
  }
  std::puts("ok");
  return 0;
}
