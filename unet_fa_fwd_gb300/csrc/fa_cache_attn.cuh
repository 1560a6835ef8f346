// fa_cache_attn.cuh — attention of bf16 queries to the paged e4m3 cache:
//   t_ij = scale * q_i . k_j,  O_i = sum_j softmax_j(t_ij) v_j,
//   LSE_i = ln sum_j e^(t_ij),
// over the keys j < len[b], with `causal` j <= q_start[b] + i too.  Query head
// hq reads key head hq / (Hq / Hk).  A row that sees no key gives O = 0 and
// LSE = -inf.
#pragma once

#include <cuda_bf16.h>
#include <climits>
#include <cstdint>

#include "fa_cache_geom.h"
#include "fa_cache_quant.cuh"
#include "sm100_ptx.cuh"

namespace fa {

struct CacheAttnParams {
  CacheView c;
  const __nv_bfloat16* q;  // [B][Hq][Nq][D]
  __nv_bfloat16* out;      // [B][Hq][Nq][D]
  float* lse;              // [B][Hq][Nq]
  const int* lens;         // [B]
  const int* q_start;      // [B] or nullptr: len - Nq
  int B, Hq, Nq, causal;
  float scale_log2;
  int* status;
};

// One block per query row: 128 keys at a time, one key per thread for the
// scores, one channel per thread for the values.
template <int D>
__global__ void __launch_bounds__(128) fa_cache_rows_kernel(const __grid_constant__ CacheAttnParams p) {
  __shared__ float q[D], prob[128], red[4];
  __shared__ int ids[128];
  const int tid = threadIdx.x;
  const long long row = blockIdx.x;
  const int i = (int)(row % p.Nq);
  const int hq = (int)(row / p.Nq % p.Hq), b = (int)(row / p.Nq / p.Hq);
  const int h = hq / (p.Hq / p.c.H);
  bool bad = false;
  const int most = (int)min((long long)p.c.width * p.c.page, (long long)INT32_MAX);
  const int len = cache_clamp(p.lens[b], most, bad);
  long long last = len;
  if (p.causal) last = min(last, (long long)(p.q_start ? p.q_start[b] : len - p.Nq) + i + 1);
  if (tid < D) q[tid] = __bfloat162float(p.q[row * D + tid]) * p.scale_log2;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  auto block_max = [&](float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if ((tid & 31) == 0) red[tid >> 5] = x;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  };
  for (long long k0 = 0; k0 < last; k0 += 128) {
    __syncthreads();
    const long long key = k0 + tid;
    float t = -INFINITY;
    if (key < last) {
      const int index = (int)(key / p.c.page);
      const int id = cache_page(p.c.table[(long long)b * p.c.width + index], p.c.num_pages, bad);
      ids[tid] = id;
      const long long base = (long long)id * p.c.H + h;
      const uint8_t* kr = p.c.code[0] + (base * p.c.page + key % p.c.page) * D;
      float dot = 0.f;
      for (int d = 0; d < D; d += 2) {
        const float2 f = e4m3x2_value(*reinterpret_cast<const uint16_t*>(kr + d));
        dot = fmaf(q[d], f.x, fmaf(q[d + 1], f.y, dot));
      }
      t = dot * p.c.scale[0][base];
    }
    const float m_new = fmaxf(m, block_max(t));
    const float e = t == -INFINITY ? 0.f : exp2f(t - m_new);
    prob[tid] = e;
    __syncthreads();
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - m_new);
    m = m_new;
    l *= alpha;
    acc *= alpha;
    const int n = (int)min(128LL, last - k0);
    for (int j = 0; j < n; ++j) {
      l += prob[j];
      if (tid < D) {
        const long long base = (long long)ids[j] * p.c.H + h;
        const float v = e4m3x2_value(p.c.code[1][(base * p.c.page + (k0 + j) % p.c.page) * D + tid]).x;
        acc = fmaf(prob[j] * p.c.scale[1][base], v, acc);
      }
    }
  }
  if (tid < D) p.out[row * D + tid] = __float2bfloat16_rn(l > 0.f ? acc / l : l);
  if (tid == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : (l == 0.f ? -INFINITY : l);
  if (bad) atomicCAS(p.status, 0, kStatusIndex);
}

}  // namespace fa
