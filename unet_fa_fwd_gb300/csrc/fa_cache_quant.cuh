// fa_cache_quant.cuh — the paged e4m3 key/value cache: tokens quantised as
// they are written, and read back as bf16.
//
// A page holds PAGE tokens of each head as e4m3 codes [PAGE][D] and one fp32
// scale: the least power of two s in [2^-117, 2^119] with max |x| <= 448 s
// over the page's tokens.  Tokens are appended; when a page's scale has to
// grow, the codes already there are multiplied by the ratio of the scales and
// rounded again.  Because the ratio is a power of two that is exact unless
// the code becomes an e4m3 subnormal, so what a page holds hardly depends on
// how its tokens were grouped into calls: an element is off by at most half a
// step of e4m3 (2^-4 relative, or 2^-10 s for subnormals), and by 2^-10 s more
// where it was rounded again into a subnormal.  code * s is always a bf16
// number, so reading back rounds nothing.
//
// e4m3 has no infinity: an element that is not finite is stored as NaN, and
// takes no part in the scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "fa_cache_geom.h"

namespace fa {

constexpr int kStatusIndex = 6;  // == FA_ERR_INDEX
constexpr int kWriteThreads = 128, kReadThreads = 256;

struct CacheView {
  uint8_t* code[2];   // k, v: [num_pages][H][page][D]
  float* scale[2];    // [num_pages][H]
  const int* table;   // [B][width]
  int width, num_pages, H, page;
};

__device__ __forceinline__ uint32_t e4m3x2_bits(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t bits) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)bits));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct CacheWriteParams {
  CacheView c;
  const __nv_bfloat16* x[2];
  long long xb[2], xh[2], xn[2];  // strides of k, v in elements
  const int* start;               // [B]: tokens already in the cache
  const int* count;               // [B] or nullptr: N each
  int B, N, slots;                // slots: pages a call can touch per sequence
  int* status;
};

// One block: one page of one head of one sequence, of k or v.  A thread holds
// its 8-element pieces of the new tokens in registers between the maximum and
// the rounding, so each input is read once.  Small blocks (the phases of a block
// do not overlap, those of different blocks do): 997 tokens of 7 x 8 heads of 64
// took 10.5 us with 256 threads.  Heads are adjacent blocks: in a slice of a
// token-major projection they are adjacent in memory.  10800 tokens of 24 heads
// of 128 take 33 to 35 us, 5.7 TB/s of 6.8: the loads, the maximum and the rounding
// of the five blocks that an SM holds do not hide one another entirely.
template <int D, int PAGE, bool VEC>
__global__ void __launch_bounds__(kWriteThreads) fa_cache_write_kernel(const __grid_constant__ CacheWriteParams p) {
  constexpr int CPR = D / 8;                                  // pieces per token
  constexpr int PIECES = PAGE * CPR;
  constexpr int PER = (PIECES + kWriteThreads - 1) / kWriteThreads;
  uint32_t blk = blockIdx.x;
  const int h = blk % p.c.H;
  blk /= p.c.H;
  const int slot = blk % p.slots;
  blk /= p.slots;
  const int kv = blk & 1, b = blk >> 1;
  const int tid = threadIdx.x;

  bool bad = false;
  const int most = (int)min((long long)p.c.width * PAGE, (long long)INT32_MAX);
  const int given = p.start[b], start = cache_clamp(given, most, bad);
  const int count = p.count ? cache_clamp(p.count[b], p.N, bad) : p.N;
  long long end = (long long)given + count;  // token i belongs at given + i, also before 0
  if (end > most) {
    bad = true;
    end = most;
  }
  const int index = start / PAGE + slot;  // page of the sequence
  const long long pos0 = (long long)index * PAGE;
  const bool any = pos0 < end && count > 0;
  int id = 0;
  if (any) {
    id = p.c.table[(long long)b * p.c.width + index];
    if (id < 0 || id >= p.c.num_pages) {  // nothing is written to a page outside the cache
      bad = true;
      id = -1;
    }
  }
  if (bad && tid == 0) atomicCAS(p.status, 0, kStatusIndex);
  if (!any || id < 0) return;
  const int old = start > pos0 ? (int)(start - pos0) : 0;     // tokens the page holds already
  const int last = (int)min((long long)PAGE, end - pos0);     // tokens it holds afterwards

  const __nv_bfloat16* x = p.x[kv] + b * p.xb[kv] + h * p.xh[kv];
  const long long first = pos0 - given;                       // token of the call in row 0 of the page
  uint4 raw[PER];
  uint32_t amax = 0;  // of the finite elements, as bf16 bits
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int piece = i * kWriteThreads + tid;
    const int row = piece / CPR;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (piece < PIECES && row >= old && row < last) {
      const __nv_bfloat16* src = x + (first + row) * p.xn[kv] + (piece % CPR) * 8;
      if constexpr (VEC) {
        raw[i] = *reinterpret_cast<const uint4*>(src);
      } else {
        alignas(16) __nv_bfloat16 t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = src[e];
        raw[i] = *reinterpret_cast<const uint4*>(t);
      }
    }
  }
  // The largest magnitude as bits, two elements at a time; infinities and NaN
  // come out as 0x7f80 or more.
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) amax = __vmaxu2(amax, w[e] & 0x7fff7fffu);
  }
  amax = max(amax & 0xffffu, amax >> 16);
  __shared__ uint32_t wmax[kWriteThreads / 32];
  auto block_max = [&](uint32_t x) {
    x = __reduce_max_sync(0xffffffffu, x);
    if ((tid & 31) == 0) wmax[tid >> 5] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWriteThreads / 32; ++w) x = max(x, wmax[w]);
    return x;
  };
  float* scale_at = p.c.scale[kv] + (long long)id * p.c.H + h;
  const float was = old ? *scale_at : 0.f;
  amax = block_max(amax);
  const bool finite = amax < 0x7f80u;  // block-uniform
  if (!finite) {  // once more without the elements that are not
    __syncthreads();
    amax = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
        amax = max(amax, max(lo >= 0x7f80u ? 0u : lo, hi >= 0x7f80u ? 0u : hi));
      }
    }
    amax = block_max(amax);
  }
  const float need = __int_as_float((cache_scale_exp(amax << 16) + 127) << 23);
  const float scale = fmaxf(was, need);
  uint8_t* page = p.c.code[kv] + ((long long)id * p.c.H + h) * (PAGE * D);
  if (old && scale > was) {  // block-uniform: the page's earlier tokens in the new scale
    const float ratio = was / scale;  // a power of two
    for (int piece = tid; piece < old * CPR; piece += kWriteThreads) {
      uint2 v = *reinterpret_cast<const uint2*>(page + piece * 8);
      uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 a = e4m3x2_value(w[k] & 0xffffu), c = e4m3x2_value(w[k] >> 16);
        w[k] = e4m3x2_bits(a.x * ratio, a.y * ratio) | (e4m3x2_bits(c.x * ratio, c.y * ratio) << 16);
      }
      *reinterpret_cast<uint2*>(page + piece * 8) = make_uint2(w[0], w[1]);
    }
  }
  if (tid == 0) *scale_at = scale;
  // scale is a power of two: 1 / scale is exact (2^119 has the subnormal-free
  // reciprocal 2^-119, 2^-117 the finite one 2^117).
  const float inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int piece = i * kWriteThreads + tid;
    const int row = piece / CPR;
    if (piece >= PIECES || row < old || row >= last) continue;
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo = __uint_as_float(w[e] << 16) * inv, hi = __uint_as_float(w[e] & 0xffff0000u) * inv;
      if (!finite) {  // x - x is 0, or NaN for an infinity
        lo += lo - lo;
        hi += hi - hi;
      }
      c[e] = e4m3x2_bits(lo, hi);
    }
    *reinterpret_cast<uint2*>(page + piece * 8) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
}

struct CacheReadParams {
  CacheView c;
  __nv_bfloat16* out[2];  // [B][H][N][D]
  const int* lens;        // [B]: tokens the sequence holds
  const int* first;       // [B] or nullptr: 0
  int B, N, blocks;       // blocks per (k or v, sequence, head)
  int* status;
};

// Tokens first .. first + N - 1 of each sequence as bf16; zero from the
// sequence's length on.  A thread turns 16 codes (one 16-byte load) into two
// 16-byte stores.  (More pieces a thread, or a block a page that reads the
// page's number and scale once, measured slower: 34 to 37 us for 10800 tokens of
// 24 heads of 128 where this takes 33, 6.0 TB/s; conversions and address
// arithmetic fill 71 % of the issue slots.)
template <int D>
__global__ void __launch_bounds__(kReadThreads) fa_cache_read_kernel(const __grid_constant__ CacheReadParams p) {
  constexpr int CPR = D / 16;
  uint32_t blk = blockIdx.x;
  const int part = blk % p.blocks;
  blk /= p.blocks;
  const int h = blk % p.c.H;
  blk /= p.c.H;
  const int kv = blk & 1, b = blk >> 1;
  const long long piece = (long long)part * kReadThreads + threadIdx.x;
  const long long row = piece / CPR;
  bool bad = false;
  const int most = p.c.width * p.c.page;
  const int len = cache_clamp(p.lens[b], most, bad);
  const int first = p.first ? cache_clamp(p.first[b], most, bad) : 0;
  if (row < p.N) {
    uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    const long long at = first + row;
    if (at < len) {
      const int shift = 31 - __clz(p.c.page);  // page is a power of two
      const int id = cache_page(p.c.table[(long long)b * p.c.width + (int)(at >> shift)], p.c.num_pages, bad);
      const long long base = (long long)id * p.c.H + h;
      const float scale = p.c.scale[kv][base];
      const uint4 v = *reinterpret_cast<const uint4*>(
          p.c.code[kv] + ((base << shift) + ((int)at & (p.c.page - 1))) * D + (int)(piece % CPR) * 16);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = e4m3x2_value((w[k / 2] >> (16 * (k & 1))) & 0xffffu);
        const __nv_bfloat162 t = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        o[k] = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(p.out[kv] + ((long long)b * p.c.H + h) * p.N * D) + piece * 2;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  if (bad) atomicCAS(p.status, 0, kStatusIndex);
}

}  // namespace fa
