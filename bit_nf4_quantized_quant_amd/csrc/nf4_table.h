// The NF4 code table as passed to the kernels (plain data, host and device).
#pragma once

#include <cstdint>

namespace qlora {

// The 16 NF4 levels (fp32, ascending) and the 15 decision thresholds passed by
// value to every kernel that needs them.  thr[j] is the smallest fp32 number
// strictly above the midpoint of levels j and j+1, so for an fp32 quotient x
// the nearest level (the lower one on an exact tie) is #{ j : x >= thr[j] }.
struct Nf4Table {
  float level[16];
  float thr[15];
};

// The code tables the library knows (the C ABI's QLORA_TABLE_* values).
constexpr int kTableNf4 = 0, kTableUniform4 = 1, kTableFp4 = 2, kCodeTables = 3;

// Host: table `type` (0 <= type < kCodeTables), built once.  NF4 comes from
// the quantile construction.
const Nf4Table& code_table(int type);

// The thresholds by bucket, for a code search with one comparison: bucket q
// (0..32) is [q/16 - 1, (q+1)/16 - 1); it holds at most one threshold, thr[q]
// (+inf if none), and base[q] thresholds lie below it, so a quotient x in
// bucket q has code base[q] + (x >= thr[q]).  The bucket index may come from
// a rounded 16 x + 16: a quotient put one bucket off lies within 2^-23 of the
// shared edge, and since no threshold lies within 2^-20 of an edge, the code
// comes out the same.  ok = 0 if the table does not have these properties
// (the kernels then compare with all 15 thresholds).
struct Nf4Buckets {
  float thr[33];
  unsigned int base[33];
  int ok;
};

const Nf4Buckets& code_buckets(int type);

// The cache's code search: the code of a quotient x is the number of midpoints
// between neighbouring levels that lie below it (FP4's two zeros count as
// neighbours with a midpoint at 0, so a small positive x gets the upper one).
// Bucket q (0..33) is [(q - 16.5)/16, (q - 15.5)/16), its index the integer
// part of 16 x + 16.5; thr[q] is the smallest fp32 number above the bucket's
// one midpoint (+inf if none), base[q] the midpoints below the bucket.  Every
// table's midpoints, the one at zero included, lie at least 2^-10 away from
// these edges and no two share a bucket, so the search holds for every table
// and for quotients up to 1 + 2^-5 in magnitude.
constexpr int kKvBuckets = 34;
struct KvBuckets {
  float thr[kKvBuckets];
  unsigned int base[kKvBuckets];
};

const KvBuckets& kv_buckets(int type);

// The levels as the decode kernels feed them to bf16 dot products and matrix
// cores: bf16(kappa * L[i]), with the block sums scaled by 1/kappa at the end.
// kappa is the smallest integer in 1..64 for which every kappa * L[i] is a
// bf16 number (to 2^-20 relative) -- 15 for the uniform table, whose levels
// are odd multiples of 1/15, and 3 for FP4, whose levels are E2M1 values over
// 6 -- so those tables enter exactly; NF4's quantiles have no such multiple,
// kappa = 1, and the kernels take bf16(L).
struct DecodeLevels {
  uint16_t bf16[16];
  float kappa;
};

const DecodeLevels& decode_levels(int type);

// The levels as the cache's attention feeds them to fp16 matrix products:
// fp16(kappa * L[i]), the products scaled by 1 / kappa at the end.  For the
// uniform table kappa = 15 and for FP4 kappa = 3 make every level an fp16
// number.  No factor does that for NF4's quantiles, and a mean over many
// positions shrinks with their number while a mean rounding error of the levels
// does not: at 131072 positions fp16(L) itself (mean error -1.1e-5 over the codes
// that normal data take) puts the result 0.7 % off.  kappa = 1.7913437 leaves a
// mean error of 1.2e-7 over the codes of normal data, and below 9e-7 over those of
// Laplace, uniform and shifted normal data and over all codes alike; it is the
// best of 2^20 factors in [1, 2) by the largest of these five.
struct Fp16Levels {
  uint32_t bits[16];
  float inv_kappa;
};

const Fp16Levels& fp16_levels(int type);

}  // namespace qlora
