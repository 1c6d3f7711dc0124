// Storing tokens in the 4-bit key/value cache and reading them back (gfx950).
//
// A run of 64 elements x of one token and head, a = max |x|, is stored as
//   s = bf16(min(a, largest bf16)), 0 where a < 2^-126, NaN where a is not finite,
//   code = #{ j : fl(x fl(1/s)) >= thr[j] }          (the nearest level),
// one reciprocal a run and one product an element in place of the weights'
// division an element, which is what bounds their quantizer.  Both passes
// stream memory once and use no matrix core.
#include "common.h"
#include "kv.h"

namespace qlora {
namespace kv {
namespace {

constexpr int kThreads = 256;

// Eight consecutive elements as fp32: bf16 (16 bytes) or fp32 (32 bytes).
template <bool kF32>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
  if constexpr (kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(v[i]), x[2 * i + 1] = bf16_hi(v[i]);
  }
}

// ------------------------------------------------------------------ write
//
// Eight lanes hold one run, eight elements each.  A workgroup takes kIter times
// 32 runs, each time those of 32 / (D / 64) tokens of one head, so that a wave's
// code bytes go to consecutive rows of a page; all loads go out first.  The code
// search is one comparison against the single threshold of the quotient's bucket
// (KvBuckets): |q| <= 1 + 2^-7 whatever the run holds (the scale is the largest
// magnitude, rounded), or NaN, which converts to 0, so the index needs no clamp.
template <bool kF32, int kIter>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(WriteArgs a, int nb_shift, KvBuckets bk) {
  __shared__ float2 lut[kKvBuckets];
  const uint32_t head = blockIdx.x % a.c.heads, group = blockIdx.x / a.c.heads;
  const int which = blockIdx.y;
  const uint32_t run = threadIdx.x >> 3, piece = threadIdx.x & 7;
  const uint32_t blk = run & ((1u << nb_shift) - 1u);
  const int per = 32 >> nb_shift;                  // tokens per time
  const int64_t t0 = (int64_t)group * (per * kIter) + (run >> nb_shift);
  float x[kIter][8];
  uint32_t slot[kIter];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int64_t t = t0 + it * per;
    const int64_t tc = t < a.tokens ? t : a.tokens - 1;
    slot[it] = t < a.tokens ? (uint32_t)a.slots[tc] : 0xFFFFFFFFu;
    load8<kF32>(a.x[which], tc * a.token_stride[which] + head * a.head_stride[which] + blk * 64 + piece * 8, x[it]);
  }
  if (threadIdx.x < kKvBuckets)
    lut[threadIdx.x] = make_float2(bk.thr[threadIdx.x], __uint_as_float(bk.base[threadIdx.x]));
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if (slot[it] >= a.c.rows) continue;            // (whole runs leave: the reduction below stays inside a run)
    // the magnitudes' bit patterns order like the numbers, with infinities and NaN on top
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[it][i]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, false));    // quad_perm 1,0,3,2
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, false));    // quad_perm 2,3,0,1
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x141, 0xF, 0xF, false));   // row_half_mirror
    uint32_t sb = min(top + 0x7FFFu + ((top >> 16) & 1u), 0x7F7F0000u) >> 16;
    if (top < 0x00800000u) sb = 0;
    if (top >= 0x7F800000u) sb = 0x7FC0u;
    const float s = __uint_as_float(sb << 16);
    const float r = sb ? 1.0f / s : 0.0f;
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x[it][i] * r;
      const float2 e = lut[(int)__builtin_fmaf(q, 16.0f, 16.5f)];
      packed |= (__float_as_uint(e.y) + (q >= e.x ? 1u : 0u)) << (4 * i);
    }
    const uint32_t page = div_by(slot[it], a.c.page_div);
    const uint64_t row = (uint64_t)(page * a.c.heads + head) * a.c.page_size + (slot[it] - page * a.c.page_size);
    reinterpret_cast<uint32_t*>(a.c.codes[which])[(((row << nb_shift) + blk) << 3) + piece] = packed;
    if (piece == 0) a.c.scales[which][(row << nb_shift) + blk] = (uint16_t)sb;
  }
}

// ------------------------------------------------------------------ read
//
// The same shape the other way round: eight codes (one dword) a lane, eight
// values out.  The values leave by nontemporal stores: 32768 tokens of 8 heads
// of 128 to bf16 take 58 us through the caches, whose write-backs then come in
// no order, and 32 us (5.4 TB/s) past them.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(ReadArgs a, int nb_shift, Nf4Table tab) {
  __shared__ float lut[16];
  if (threadIdx.x < 16) lut[threadIdx.x] = tab.level[threadIdx.x];
  __syncthreads();
  const uint32_t head = blockIdx.x % a.c.heads, group = blockIdx.x / a.c.heads;
  const int which = blockIdx.y;
  const uint32_t run = threadIdx.x >> 3, piece = threadIdx.x & 7;
  const uint32_t blk = run & ((1u << nb_shift) - 1u);
  const int64_t t = (int64_t)group * (32 >> nb_shift) + (run >> nb_shift);
  if (t >= a.tokens) return;
  const uint32_t slot = (uint32_t)a.slots[t];
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (slot < a.c.rows) {
    const uint32_t page = div_by(slot, a.c.page_div);
    const uint64_t row = (uint64_t)(page * a.c.heads + head) * a.c.page_size + (slot - page * a.c.page_size);
    const uint32_t w = reinterpret_cast<const uint32_t*>(a.c.codes[which])[(((row << nb_shift) + blk) << 3) + piece];
    const float s = __uint_as_float((uint32_t)a.c.scales[which][(row << nb_shift) + blk] << 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = lut[(w >> (4 * i)) & 15u] * s;
  }
  const int64_t o = (((t * a.c.heads + head) << nb_shift) + blk) * 8 + piece;   // 8-element pieces
  if constexpr (kF32) {
    f32x4* p = reinterpret_cast<f32x4*>(a.out[which]) + 2 * o;
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, p);
    __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, p + 1);
  } else {
    const u32x4 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(a.out[which]) + o);
  }
}

int nb_shift_of(int D) { return D == 64 ? 0 : D == 128 ? 1 : 2; }

dim3 run_grid(const Cache& c, int64_t tokens, int iter) {
  const int64_t per = (32 >> nb_shift_of(c.D)) * iter;
  return dim3((unsigned)((tokens + per - 1) / per * c.heads), 2);
}

}  // namespace

hipError_t launch_kv_write(const WriteArgs& a, hipStream_t s) {
  // Past eight workgroups a CU each takes two groups of runs: 4096 tokens of 32
  // heads of 128 24 -> 19 us (four: 19.3, eight: 20); below that one group each
  // keeps every CU busy.
  const dim3 one = run_grid(a.c, a.tokens, 1);
  const bool many = one.x > 2048;
  const auto kernel = a.f32 ? (many ? kv_write_kernel<true, 2> : kv_write_kernel<true, 1>)
                            : (many ? kv_write_kernel<false, 2> : kv_write_kernel<false, 1>);
  hipLaunchKernelGGL(kernel, many ? run_grid(a.c, a.tokens, 2) : one, dim3(kThreads), 0, s, a, nb_shift_of(a.c.D),
                     kv_buckets(a.c.table));
  return hipGetLastError();
}

hipError_t launch_kv_read(const ReadArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((a.f32 ? kv_read_kernel<true> : kv_read_kernel<false>), run_grid(a.c, a.tokens, 1),
                     dim3(kThreads), 0, s, a, nb_shift_of(a.c.D), code_table(a.c.table));
  return hipGetLastError();
}

}  // namespace kv
}  // namespace qlora
