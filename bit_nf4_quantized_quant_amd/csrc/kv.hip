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
// Eight lanes hold one run, eight elements each.  A workgroup takes 32 runs:
// 32 / (D / 64) tokens of one head, so that a wave's code bytes go to
// consecutive rows of a page.  The code search is one comparison against the
// single threshold of the quotient's bucket (KvBuckets).
template <bool kF32>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(WriteArgs a, int nb_shift, KvBuckets bk) {
  __shared__ float2 lut[kKvBuckets];
  if (threadIdx.x < kKvBuckets)
    lut[threadIdx.x] = make_float2(bk.thr[threadIdx.x], __uint_as_float(bk.base[threadIdx.x]));
  __syncthreads();
  const uint32_t head = blockIdx.x % a.c.heads, group = blockIdx.x / a.c.heads;
  const int which = blockIdx.y;
  const uint32_t run = threadIdx.x >> 3, piece = threadIdx.x & 7;
  const uint32_t blk = run & ((1u << nb_shift) - 1u);
  const int64_t t = (int64_t)group * (32 >> nb_shift) + (run >> nb_shift);
  if (t >= a.tokens) return;                       // (whole runs leave: the reduction below stays inside a run)
  const int32_t slot = a.slots[t];
  float x[8];
  load8<kF32>(a.x[which], t * a.token_stride[which] + head * a.head_stride[which] + blk * 64 + piece * 8, x);
  if ((uint32_t)slot >= a.c.rows) return;
  // the magnitudes' bit patterns order like the numbers, with infinities and NaN on top
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
  uint32_t sb = min(top + 0x7FFFu + ((top >> 16) & 1u), 0x7F7F0000u) >> 16;
  if (top < 0x00800000u) sb = 0;
  if (top >= 0x7F800000u) sb = 0x7FC0u;
  const float s = __uint_as_float(sb << 16);
  const float r = sb ? 1.0f / s : 0.0f;
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * r;
    const int b = min(max((int)__builtin_fmaf(q, 16.0f, 16.5f), 0), kKvBuckets - 1);
    const float2 e = lut[b];
    packed |= (__float_as_uint(e.y) + (q >= e.x ? 1u : 0u)) << (4 * i);
  }
  const uint32_t page = div_by((uint32_t)slot, a.c.page_div);
  const uint64_t row = (uint64_t)(page * a.c.heads + head) * a.c.page_size + ((uint32_t)slot - page * a.c.page_size);
  reinterpret_cast<uint32_t*>(a.c.codes[which])[(((row << nb_shift) + blk) << 3) + piece] = packed;
  if (piece == 0) a.c.scales[which][(row << nb_shift) + blk] = (uint16_t)sb;
}

// ------------------------------------------------------------------ read
//
// The same shape the other way round: eight codes (one dword) a lane, eight
// values out.
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
    float4* p = reinterpret_cast<float4*>(a.out[which]) + 2 * o;
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    reinterpret_cast<uint4*>(a.out[which])[o] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                           pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

int nb_shift_of(int D) { return D == 64 ? 0 : D == 128 ? 1 : 2; }

dim3 run_grid(const Cache& c, int64_t tokens) {
  const int64_t per = 32 >> nb_shift_of(c.D);
  return dim3((unsigned)((tokens + per - 1) / per * c.heads), 2);
}

}  // namespace

hipError_t launch_kv_write(const WriteArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((a.f32 ? kv_write_kernel<true> : kv_write_kernel<false>), run_grid(a.c, a.tokens),
                     dim3(kThreads), 0, s, a, nb_shift_of(a.c.D), kv_buckets(a.c.table));
  return hipGetLastError();
}

hipError_t launch_kv_read(const ReadArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((a.f32 ? kv_read_kernel<true> : kv_read_kernel<false>), run_grid(a.c, a.tokens),
                     dim3(kThreads), 0, s, a, nb_shift_of(a.c.D), code_table(a.c.table));
  return hipGetLastError();
}

}  // namespace kv
}  // namespace qlora
