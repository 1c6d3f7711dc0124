// Attention over the 4-bit key/value cache: the choice between the kernels for
// few and for many query rows, the split of the positions, and the kernel that
// joins the splits.
#include <algorithm>
#include <cmath>

#include "kv_common.h"
#include "launch.h"

namespace qlora {
namespace kv {
namespace {

// One row's result from `splits` partial ones, by a workgroup of 256: partial s,
// at row at(s) of o [rows][D] and stat [rows], holds exp2-weighted sums relative
// to its own reference.  D / 4 lanes hold four elements each and 1024 / D groups
// of them take the partials in turn, kChunk at a time.
template <int D, typename At>
__device__ __forceinline__ void join_row(int splits, At at, const float* o, const float2* stat, float inv_kappa,
                                         uint16_t* out, float* lse) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes, kChunk = 256;
  __shared__ float weight[kChunk];
  __shared__ float wave_top[4], wave_sum[4];
  __shared__ f32x4 acc[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // the common reference
  float top = -INFINITY;
  for (int s = tid; s < splits; s += kChunk) top = fmaxf(top, stat[at(s)].x);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  if (lane == 0) wave_top[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
  const float ref = top == -INFINITY ? 0.f : top;
  const int g = tid / kLanes, col = tid % kLanes;
  float sum = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += kChunk) {
    const int count = min(kChunk, splits - s0);
    __syncthreads();
    if (tid < count) {
      const float2 st = stat[at(s0 + tid)];
      weight[tid] = exp2_fast(st.x - ref);
      sum = __builtin_fmaf(weight[tid], st.y, sum);
    }
    __syncthreads();
#pragma unroll 4
    for (int s = g; s < count; s += kGroups) {
      const float f = weight[s];
      const f32x4 p = reinterpret_cast<const f32x4*>(o + at(s0 + s) * D)[col];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, p[e], v[e]);
    }
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
  if (lane == 0) wave_sum[wave] = sum;
  acc[tid] = v;
  __syncthreads();
  if (tid >= kLanes) return;
#pragma unroll
  for (int h = 1; h < kGroups; ++h) v += acc[h * kLanes + tid];
  sum = wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];
  const float inv = sum == 0.f ? 0.f : inv_kappa / sum;
  reinterpret_cast<u32x2*>(out)[tid] = u32x2{pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv)};
  if (lse && tid == 0) *lse = sum == 0.f ? -INFINITY : kLn2 * (top + __builtin_amdgcn_logf(sum));
}

template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(AttnArgs a, Split sp, float inv_kappa, Partial part) {
  const int group = (int)a.group_div.d;
  const int r = blockIdx.x % sp.rows, head = blockIdx.x / sp.rows, b = blockIdx.y;
  const Seq seq = sequence(a, b);
  const int rows = seq.n * group;
  if (r >= rows) return;
  const int r0 = r / sp.tile_rows * sp.tile_rows;
  const Span span = tile_span(a, seq, div_by(r0, a.group_div), div_by(min(r0 + sp.tile_rows, rows) - 1, a.group_div));
  const int i = div_by(r, a.group_div);
  const int64_t row = (int64_t)(seq.q0 + i) * a.q_heads + head * group + (r - i * group);
  join_row<D>(live_splits(span, sp.chunk, sp.splits), [&](int s) { return row * sp.splits + s; }, part.o, part.stat, inv_kappa,
              a.out + row * D, a.lse ? a.lse + row : nullptr);
}

}  // namespace

Split split_of(const AttnArgs& a, const Cost& cost, float* us) {
  constexpr int kMaxSplits = 128;
  constexpr float kJoin = 6.f;              // the joining launch, us: 4 on the device, and the host's 3.5
  constexpr float kJoinBytes = 4e6f;        // its bytes per us, written and read back
  const int64_t rows = a.max_q * (a.q_heads / a.c.heads), tiles = (rows + cost.tile_rows - 1) / cost.tile_rows;
  const int64_t pieces = a.seqs * a.c.heads * tiles;
  const int64_t span = std::max<int64_t>(1, a.window > 0 ? std::min(a.max_len, a.window + a.max_q + 15) : a.max_len);
  const int cus = cu_count();
  Split best{};
  *us = INFINITY;
  for (int64_t n = 1; n <= kMaxSplits; n *= 2) {
    const int64_t chunk = ((span + n - 1) / n + 255) / 256 * 256, splits = (span + chunk - 1) / chunk;
    const int64_t groups = pieces * splits, slots = (int64_t)cost.per_cu * cus;
    const float each = cost.base + (float)std::min(chunk, span) * (groups > cus ? cost.shared : cost.position);
    const float joined = (float)a.tokens * a.q_heads * splits * a.c.D * 8.f;
    const float t = (float)((groups + slots - 1) / slots) * each + (splits > 1 ? kJoin + joined / kJoinBytes : 0.f);
    if (t < *us) {
      *us = t;
      best = Split{(int)chunk, (int)splits, (int)rows, (int)tiles, cost.tile_rows};
    }
    if (chunk == 256) break;
  }
  return best;
}

// The kernel for few rows shares a tile's expanded codes between 32 query rows (16 at
// D = 256), that for many between 256, but its workgroup takes as long for one row as
// for 256.  So the choice is by the estimated times: 256 rows on each of 32 heads and
// 1000 positions, D = 128, take 19 us with the first and 40 us with the second (as 32
// workgroups do not fill the device); 128 rows on 128 heads and 300 positions 25 us and
// 16.5 us.
AttnPlan kv_attention_plan(const AttnArgs& a) {
  float few = 0.f, many = 0.f;
  const Split d = split_of(a, decode_cost(a), &few), p = split_of(a, prompt_cost(a), &many);
  AttnPlan plan{many < few, many < few ? p : d, 0};
  if (plan.split.splits > 1)
    plan.workspace = (size_t)(a.tokens * a.q_heads) * plan.split.splits * (a.c.D * sizeof(float) + sizeof(float2));
  return plan;
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
  const Split& sp = plan.split;
  Partial part;
  part.o = static_cast<float*>(a.workspace);
  part.stat = reinterpret_cast<float2*>(part.o + (size_t)(a.tokens * a.q_heads) * sp.splits * a.c.D);
  const hipError_t e = plan.prompt ? launch_prompt(a, sp, part, s) : launch_decode(a, sp, part, s);
  if (e != hipSuccess || sp.splits == 1) return e;
  const dim3 grid((unsigned)(sp.rows * a.c.heads), (unsigned)a.seqs);
  const auto kernel = a.c.D == 64 ? kv_join_kernel<64> : a.c.D == 128 ? kv_join_kernel<128> : kv_join_kernel<256>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, sp, fp16_levels(a.c.table).inv_kappa, part);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace qlora
