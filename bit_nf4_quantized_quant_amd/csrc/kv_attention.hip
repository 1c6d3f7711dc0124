// Attention over the 4-bit key/value cache (gfx950):
//   out_i = sum_j softmax_j(scale q_i k_j) v_j   over the positions j that query i sees.
//
// One workgroup a query row and head.  Each of its four waves takes every
// fourth tile of 64 positions: a lane forms one position's score, and then
// each lane sums its D / 64 elements over the tile.  The waves' running
// maxima and sums are joined at the end.
#include <cmath>
#include <cstring>
#include <mutex>

#include "kv_common.h"

namespace qlora {
namespace kv {
namespace {

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <int D>
__global__ void __launch_bounds__(256) kv_attention_kernel(AttnArgs a, Nf4Table tab) {
  constexpr int NB = D / 64;
  __shared__ float lut[16];
  __shared__ float qs[D];
  __shared__ float om[4][D], mm[4], ll[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.y, b = blockIdx.z, i = blockIdx.x;
  const int64_t q0 = a.q_starts ? max(a.q_starts[b], 0) : (int64_t)b * a.max_q;
  int64_t n = a.q_starts ? (int64_t)a.q_starts[b + 1] - q0 : a.max_q;
  n = min(min(n, a.max_q), a.tokens - q0);
  if (i >= n) return;
  const int64_t token = q0 + i;
  const int64_t len = min((int64_t)max(a.lengths[b], 0), a.table_width * a.c.page_size);
  const int64_t pos = (int64_t)a.lengths[b] - n + i;
  const int64_t hi = a.causal ? min(len, pos + 1) : len;
  const int64_t lo = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
  if (tid < 16) lut[tid] = tab.level[tid];
  if (tid < D) qs[tid] = __uint_as_float((uint32_t)a.q[token * a.token_stride + h * a.head_stride + tid] << 16) * a.scale;
  __syncthreads();
  const uint32_t head = h / (a.q_heads / a.c.heads);
  float m = -INFINITY, l = 0.f, o[NB];
#pragma unroll
  for (int e = 0; e < NB; ++e) o[e] = 0.f;
  for (int64_t t0 = lo + 64 * wave; t0 < hi; t0 += 256) {
    const int64_t t = t0 + lane;
    const uint32_t tt = (uint32_t)(t < hi ? t : hi - 1);
    const uint32_t pg = div_by(tt, a.c.page_div);
    const int32_t page = a.block_table[b * a.table_width + pg];
    const bool seen = t < hi && (uint32_t)page < a.c.pages;
    const uint64_t row = (uint64_t)((seen ? page : 0) * a.c.heads + head) * a.c.page_size + (tt - pg * a.c.page_size);
    float x = 0.f;
    for (int blk = 0; blk < NB; ++blk) {
      float part = 0.f;
      for (int w = 0; w < 8; ++w) {
        const uint32_t c = reinterpret_cast<const uint32_t*>(a.c.codes[0])[(row * NB + blk) * 8 + w];
#pragma unroll
        for (int e = 0; e < 8; ++e) part += lut[(c >> (4 * e)) & 15u] * qs[blk * 64 + w * 8 + e];
      }
      x += part * __uint_as_float((uint32_t)a.c.scales[0][row * NB + blk] << 16);
    }
    if (!seen) x = -INFINITY;
    const float mn = fmaxf(m, wave_max(x));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = __expf(m - ref), p = seen ? __expf(x - ref) : 0.f;
    m = mn;
    l = l * alpha + wave_add(p);
#pragma unroll
    for (int e = 0; e < NB; ++e) o[e] *= alpha;
    const int cnt = (int)min((int64_t)64, hi - t0);
    for (int j = 0; j < cnt; ++j) {
      const uint64_t rj = (uint64_t)(uint32_t)__shfl((int)(uint32_t)row, j) |
                          (uint64_t)(uint32_t)__shfl((int)(row >> 32), j) << 32;
      const float pj = __shfl(p, j);
      if (!__shfl((int)seen, j)) continue;
#pragma unroll
      for (int e = 0; e < NB; ++e) {
        const uint32_t c = a.c.codes[1][rj * (D / 2) + e * 32 + (lane >> 1)];
        const float v = lut[(lane & 1) ? c >> 4 : c & 15u] * __uint_as_float((uint32_t)a.c.scales[1][rj * NB + e] << 16);
        o[e] += pj * v;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < NB; ++e) om[wave][e * 64 + lane] = o[e];
  if (lane == 0) mm[wave] = m, ll[wave] = l;
  __syncthreads();
  const float M = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3]));
  const float ref = M == -INFINITY ? 0.f : M;
  float f[4], L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) f[w] = __expf(mm[w] - ref), L += f[w] * ll[w];
  if (tid < D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += f[w] * om[w][tid];
    a.out[(token * a.q_heads + h) * D + tid] = (uint16_t)pack_bf16x2(L > 0.f || L != L ? v / L : 0.f, 0.f);
  }
  if (a.lse && tid == 0) a.lse[token * a.q_heads + h] = L == 0.f ? -INFINITY : M + __logf(L);
}

// fp32 -> fp16 bits, round to nearest even, for magnitudes of fp16's normal range (or 0).
uint32_t f16_bits(float f) {
  uint32_t u;
  std::memcpy(&u, &f, 4);
  const uint32_t sign = (u >> 16) & 0x8000u;
  u &= 0x7FFFFFFFu;
  if (u == 0) return 0;
  u += 0xFFFu + ((u >> 13) & 1u);
  return sign | ((u >> 13) - (112u << 10));
}

}  // namespace

const Levels& levels_of(int table) {
  static Levels lv[kCodeTables];
  static std::once_flag once;
  std::call_once(once, [] {
    for (int ty = 0; ty < kCodeTables; ++ty) {
      // the uniform grid's levels are odd multiples of 1/15, FP4's are E2M1 numbers over 6
      const float kappa = ty == kTableUniform4 ? 15.f : ty == kTableFp4 ? 3.f : 1.f;
      lv[ty].inv_kappa = 1.0f / kappa;
      for (int i = 0; i < 16; ++i) lv[ty].h[i] = f16_bits(kappa * code_table(ty).level[i]);
    }
  });
  return lv[table];
}

size_t kv_attention_workspace_bytes(const AttnArgs& a) { return decode_fits(a) ? decode_workspace_bytes(a) : 0; }

hipError_t launch_kv_attention(const AttnArgs& a, hipStream_t s) {
  if (decode_fits(a)) return launch_decode(a, s);
  const dim3 grid((unsigned)a.max_q, (unsigned)a.q_heads, (unsigned)a.seqs);
  const Nf4Table& t = code_table(a.c.table);
  if (a.c.D == 64)
    hipLaunchKernelGGL(kv_attention_kernel<64>, grid, dim3(256), 0, s, a, t);
  else if (a.c.D == 128)
    hipLaunchKernelGGL(kv_attention_kernel<128>, grid, dim3(256), 0, s, a, t);
  else
    hipLaunchKernelGGL(kv_attention_kernel<256>, grid, dim3(256), 0, s, a, t);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace qlora
