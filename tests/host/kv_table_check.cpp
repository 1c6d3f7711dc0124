// Host check of the cache's level tables, built under sanitizers by
// tests/test_kv_abi.py.  The one-comparison code search (kv_buckets): for every table, the bucket of the
// rounded 16 x + 16.5 and its one threshold give the count of the 15
// midpoints below x, on a fine sweep of [-1 - 2^-5, 1 + 2^-5] and at the
// neighbours of every threshold and bucket edge.
#include <algorithm>
#include <cmath>
#include <cstdint>
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

static double fp16_value(uint32_t b) {
  const int e = (int)(b >> 10) & 31, m = (int)b & 1023;
  const double v = e == 0 ? std::ldexp((double)m, -24) : std::ldexp(1024.0 + m, e - 25);
  return (b & 0x8000u) ? -v : v;
}

// The levels of the fp16 products: exact for the uniform and FP4 tables; for NF4
// each within fp16's half ulp, and their mean error small over the codes of normal
// data (frequencies of 64-element runs divided by their largest magnitude, from
// 2.56 million draws) and over all codes alike.
static void check_fp16() {
  const double normal[16] = {.019, .044, .058, .071, .081, .088, .092, .088, .081, .078, .073, .067, .058, .048, .036, .017};
  for (int ty = 0; ty < kCodeTables; ++ty) {
    double mean_all = 0, mean_normal = 0;
    for (int i = 0; i < 16; ++i) {
      const double l = code_table(ty).level[i];
      const double err = fp16_value(fp16_levels(ty).bits[i]) * (double)fp16_levels(ty).inv_kappa - l;
      const double most = std::fabs(l) * (ty == kTableNf4 ? std::ldexp(1.0, -11) : 2e-7);
      if (std::fabs(err) > most + 1e-12 && ++failures < 20) std::printf("table %d level %d off by %.3g\n", ty, i, err);
      mean_all += err / 16;
      mean_normal += err * normal[i];
    }
    if (ty == kTableNf4 && (std::fabs(mean_all) > 1e-6 || std::fabs(mean_normal) > 1e-6) && ++failures)
      std::printf("mean errors %.3g %.3g\n", mean_all, mean_normal);
  }
}

int main() {
  check_fp16();
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
