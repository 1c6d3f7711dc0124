// Host check of the cache's one-comparison code search (kv_buckets), built
// under sanitizers by tests/test_kv_abi.py: for every table, the bucket of the
// rounded 16 x + 16.5 and its one threshold give the count of the 15
// midpoints below x, on a fine sweep of [-1 - 2^-5, 1 + 2^-5] and at the
// neighbours of every threshold and bucket edge.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "nf4_table.h"

using namespace qlora;

static int failures = 0;

static void check(int ty, float x) {
  const Nf4Table& t = code_table(ty);
  const KvBuckets& b = kv_buckets(ty);
  unsigned want = 0;
  for (int j = 0; j < 15; ++j) want += (double)x > ((double)t.level[j] + (double)t.level[j + 1]) / 2;
  const int q = std::min(std::max((int)std::fma(x, 16.0f, 16.5f), 0), kKvBuckets - 1);
  const unsigned got = b.base[q] + (x >= b.thr[q] ? 1u : 0u);
  if (got != want && ++failures < 20) std::printf("table %d x %.9g: %u, not %u\n", ty, x, got, want);
}

int main() {
  const float top = 1.03125f;
  for (int ty = 0; ty < kCodeTables; ++ty) {
    for (int i = -1100000; i <= 1100000; ++i) {
      const float x = (float)i * 9.37e-7f;
      if (std::fabs(x) <= top) check(ty, x);
    }
    auto around = [&](float x) {
      float up = x, down = x;
      check(ty, x);
      for (int i = 0; i < 8; ++i) {
        up = std::nextafter(up, 2.f);
        down = std::nextafter(down, -2.f);
        if (std::fabs(up) <= top) check(ty, up);
        if (std::fabs(down) <= top) check(ty, down);
      }
    };
    for (float v : code_table(ty).thr) around(v);
    for (int q = 0; q <= kKvBuckets; ++q)
      if (std::fabs((q - 16.5f) / 16.f) <= top) around((q - 16.5f) / 16.f);
    around(0.f);
  }
  std::printf(failures ? "FAILED %d\n" : "OK\n", failures);
  return failures != 0;
}
