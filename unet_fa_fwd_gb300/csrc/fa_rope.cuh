// fa_rope.cuh — rotary positions over several axes (time, height, width).
//
// The D / 2 pairs of a row are dealt to the axes in order (dims[a] / 2 pairs
// each); pair j of axis a turns by
//   angle = pos[b, n, a] * scale_a * theta_a^(-2 j / dims[a]),
//   (x0, x1) -> (x0 cos - x1 sin, x0 sin + x1 cos).
// The gradient is the rotation by -angle.
//
// F = frequency / (2 pi) is a 64-bit fixed-point fraction of a turn, and pos * F
// modulo 2^64 is the phase: the reduction to one turn loses nothing, at any int32
// position.  F itself comes from 64-bit floating point (an exponent, a power, two
// products): with f turns per unit of position it is off by e = |f| (5 +
// |ln theta|) 2^-53 at most and cut to 2^-64, so the phase is off by
// |pos| (e + 2^-64) turns.  Its top 32 bits are cut to an eighth of a turn either
// side of a quadrant before they become fp32.
//
// HBM bound: every element is read and written once.  A thread owns one
// 16-byte piece of a token's row (two, half a row apart, when the pairs are
// the row's halves), computes its pairs' sines and cosines once and walks the
// heads of q and k with them, so the trigonometry is shared by all of a
// block's heads.  119056 tokens of 24 + 24 heads of 128 in bf16 take 433 us, 6.7
// TB/s; the gradient of 16896 in fp32 125 us, 6.6 TB/s; one token 2.6 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace fa {

constexpr int kRopeMaxPairs = 64;
constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads whose loads are in flight together

struct RopeTensor {
  const void* in;
  void* out;
  long long in_b, in_h, in_n, out_b, out_h, out_n;  // strides in elements
  int H;
};

struct RopeParams {
  RopeTensor t[2];       // q, k (k.H = 0: none)
  const int* pos;        // [B][N][A], batch stride pos_b (0: shared)
  long long pos_b;
  int A, N, heads, heads_per_block;
  long long tokens;      // B * N
  int inverse;
  unsigned long long freq[kRopeMaxPairs];  // turns per unit of position, 0.64 fixed point
  unsigned char axis[kRopeMaxPairs];
};

// cos and sin of `phase` turns (0.64 fixed point).
__device__ __forceinline__ void rope_cos_sin(unsigned long long phase, float& c, float& s) {
  const uint32_t hi = (uint32_t)(phase >> 32);
  const uint32_t quad = (hi + 0x20000000u) >> 30;               // nearest quadrant
  const float x = (float)(int32_t)(hi - (quad << 30)) * 4.656612873077393e-10f;  // 2^-31: half turns
  float cs, sn;
  sincospif(x, &sn, &cs);
  c = (quad & 1u) ? ((quad & 2u) ? sn : -sn) : ((quad & 2u) ? -cs : cs);
  s = (quad & 1u) ? ((quad & 2u) ? -cs : cs) : ((quad & 2u) ? -sn : sn);
}

template <typename T>
__device__ __forceinline__ float rope_f(T x) {
  if constexpr (sizeof(T) == 4) return x;
  else return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T rope_t(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else return T(x);  // round to nearest even
}

// E consecutive elements, as one 16-byte access when they fill one (the host
// has checked the alignment), else one by one.
template <typename T, int E>
struct alignas(E * sizeof(T)) RopeVec {
  T v[E];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (E * sizeof(T) == 16) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (E * sizeof(T) == 16) {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = v[i];
    }
  }
};

// E: elements per access (16 bytes' worth, or 2 when the tensors are not
// 16-byte aligned).  HALVES: pairs (i, i + D/2), a thread owns E elements of
// each half; otherwise pairs (2i, 2i + 1), a thread owns E / 2 pairs.
template <typename T, int D, int E, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int CHUNKS = HALVES ? D / 2 / E : D / E;  // threads per token
  constexpr int PAIRS = HALVES ? E : E / 2;
  const long long i = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const long long token = i / CHUNKS;
  if (token >= p.tokens) return;
  const int chunk = (int)(i - token * CHUNKS);
  const long long b = token / p.N;
  const long long n = token - b * p.N;

  float c[PAIRS], s[PAIRS];
  const int* pos = p.pos + b * p.pos_b + n * p.A;
#pragma unroll
  for (int j = 0; j < PAIRS; ++j) {
    const int pair = chunk * PAIRS + j;
    const long long at = pos[p.axis[pair]];
    rope_cos_sin((unsigned long long)at * p.freq[pair], c[j], s[j]);
    if (p.inverse) s[j] = -s[j];
  }

  const int h0 = (int)blockIdx.y * p.heads_per_block;
  const int h1 = min(h0 + p.heads_per_block, p.heads);
  for (int h = h0; h < h1; h += kRopeBatch) {
    RopeVec<T, E> lo[kRopeBatch], hi[HALVES ? kRopeBatch : 1];
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) {
      if (h + u >= h1) break;
      const bool is_k = h + u >= p.t[0].H;
      const RopeTensor& t = p.t[is_k];
      const T* src = static_cast<const T*>(t.in) + b * t.in_b + (long long)(h + u - (is_k ? p.t[0].H : 0)) * t.in_h +
                     n * t.in_n + chunk * E;
      lo[u].load(src);
      if constexpr (HALVES) hi[u].load(src + D / 2);
    }
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) {
      if (h + u >= h1) break;
      const bool is_k = h + u >= p.t[0].H;
      const RopeTensor& t = p.t[is_k];
      T* dst = static_cast<T*>(t.out) + b * t.out_b + (long long)(h + u - (is_k ? p.t[0].H : 0)) * t.out_h +
               n * t.out_n + chunk * E;
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        T& a0 = HALVES ? lo[u].v[j] : lo[u].v[2 * j];
        T& a1 = HALVES ? hi[HALVES ? u : 0].v[j] : lo[u].v[2 * j + 1];
        const float x0 = rope_f(a0), x1 = rope_f(a1);
        a0 = rope_t<T>(x0 * c[j] - x1 * s[j]);
        a1 = rope_t<T>(x0 * s[j] + x1 * c[j]);
      }
      lo[u].store(dst);
      if constexpr (HALVES) hi[u].store(dst + D / 2);
    }
  }
}

}  // namespace fa
