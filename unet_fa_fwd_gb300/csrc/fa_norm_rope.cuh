// fa_norm_rope.cuh — norm of queries and keys for each head with the rotary
// positions in the same pass, and its gradient.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = R(pos) (w o n)
// (R: the rotation of fa_rope.cuh; w: a weight for each of the D elements, or
// none).  With g = R(-pos) dy, the gradient of the normalised row:
//   dw = sum over rows of g o n,   dx = r (g o w - n mean(g o w o n)).
//
// HBM bound: x (and dy) are read once and y (dx) written once; r is computed
// again in the gradient, so nothing is kept for it.  A thread owns one 16-byte
// piece of a token's row (when the pairs are the row's halves two, half a row
// apart, of 8 elements together in 16 bits: with 16, 219 registers left one block
// an SM) and walks heads with its pairs' sines and its weights in registers; the
// threads of a row are neighbours in a warp and sum by shuffles.  Four heads' loads
// are in flight together: the gradient's 16 warps an SM need that to cover HBM's
// latency (with two, 225 us for 200 below).
//
// dw: a thread adds up its elements over some 32 heads' rows at a time and keeps what
// adding these sums up rounds off (norm_add); a block's threads are joined by twos into
// one row of partial sums, and a second kernel adds the blocks' rows, in the same way as
// the thread.  So dw is about as exact as its terms however many rows there are, 1e-7 of
// its norm; in one chain a thread it was off by 2e-7 at 16896 tokens of 24 heads and 5e-7
// at 60000.  The order is fixed and there are no atomics: results repeat bit for bit.
//
// Measured: forward of 119056 tokens of 24 + 24 heads of 128 in bf16 472 us (6.2
// TB/s); gradient of 16896 tokens in fp32 200 us (6.2 TB/s), of 4608 in bf16 40 us
// (4.3 TB/s: twice the arithmetic a byte, 55 % of the issue slots, and the second
// kernel).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fa_rope.cuh"

namespace fa {

constexpr int kNormThreads = 256;
constexpr int kNormBackPerSm = 2;     // blocks of the gradient that are resident (128 registers: with the pairs as
                                      // halves in fp32, and off 16 bytes in 16 bits, they spill 36 to 52 bytes a thread)
constexpr int kNormMaxBlocks = 1024;  // blocks of the gradient (rows of partial sums)
constexpr int kNormReduceRows = 32;   // rows of threads of the second kernel

struct NormTensor {
  const void* x;
  const void* dy;  // gradient: of the output
  void* out;       // y, or dx
  long long x_b, x_h, x_n, dy_b, dy_h, dy_n, out_b, out_h, out_n;  // strides in elements
  const void* w;   // [D] or nullptr
  int H;
};

struct NormParams {
  NormTensor t[2];   // q, k (k.H = 0: none)
  const int* pos;    // [B][N][A], batch stride pos_b (0: shared)
  long long pos_b;
  int A, N, heads;
  int heads_per_item, groups;      // forward
  int batches[2];                  // gradient: batches of heads of q, of k
  int w_f32;         // weights are fp32, else of the tensors' type
  float eps;
  long long tokens;  // B * N
  long long blocks;  // blocks of tokens
  long long items;   // forward: token blocks x head groups; gradient: x batches of heads, q's before k's
  float* part;       // gradient with weights: [gridDim.x][2][D]
  unsigned long long freq[kRopeMaxPairs];
  unsigned char axis[kRopeMaxPairs];
};

// How a row is dealt to threads.
template <typename T, int D, bool HALVES, bool BACK>
struct NormShape {
  static constexpr int PIECES = HALVES ? 2 : 1;
  static constexpr int E = HALVES && sizeof(T) == 2 ? 4 : 16 / (int)sizeof(T);  // elements of a piece
  static constexpr int NE = E * PIECES, CHUNKS = D / NE;                        // of a thread; threads a row
  static constexpr int BATCH = 4;  // heads whose loads are in flight together
  static constexpr int TOKENS = kNormThreads / CHUNKS;
};

// E elements at p, 16 or 8 bytes' worth: one access where rows are 16-byte aligned
// (VEC), else one by one.
template <typename T, int E, bool VEC>
struct alignas(16) NormVec {
  T v[E];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC && E * sizeof(T) == 8) {
      *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
    } else if constexpr (VEC) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC && E * sizeof(T) == 8) {
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
    } else if constexpr (VEC) {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = v[i];
    }
  }
};

// Sum over the `CHUNKS` neighbouring lanes of a row, in every one of them.
template <int CHUNKS>
__device__ __forceinline__ float norm_row_sum(float v) {
#pragma unroll
  for (int m = 1; m < CHUNKS; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// (hi, lo) += (v, e): the sum of the high parts is rounded, what that takes off (exactly
// known) and the low parts add up in lo.
__device__ __forceinline__ void norm_add(float& hi, float& lo, float v, float e) {
  const float s = __fadd_rn(hi, v), was = __fadd_rn(s, -hi);
  lo = __fadd_rn(lo, __fadd_rn(e, __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -was)), __fadd_rn(v, -was))));
  hi = s;
}

template <typename T, int D, bool VEC, bool HALVES, bool BACK>
__global__ void __launch_bounds__(kNormThreads, VEC && !BACK ? 3 : 2)
    fa_norm_rope_kernel(const __grid_constant__ NormParams p) {
  using Shape = NormShape<T, D, HALVES, BACK>;
  constexpr int E = Shape::E, PIECES = Shape::PIECES, NE = Shape::NE, CHUNKS = Shape::CHUNKS, BATCH = Shape::BATCH;
  constexpr int PAIRS = NE / 2;
  static_assert(CHUNKS <= 32 && 32 % CHUNKS == 0, "a row's threads share a warp");
  using Vec = NormVec<T, E, VEC>;
  if constexpr (BACK) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the weights' kernel waits itself
  const int chunk = threadIdx.x % CHUNKS;
  // element i of this thread: column chunk * E + i, the second piece half a row on
  auto column = [&](int i) { return chunk * E + (i < E ? i : i - E + D / 2); };

  float acc[NE] = {};  // dw of one tensor, over the last rows
  // Heads h0 .. h1 - 1 of a block of tokens.
  auto rows = [&](long long tb, int h0, int h1) {
    long long token = tb * (kNormThreads / CHUNKS) + threadIdx.x / CHUNKS;
    const bool live = token < p.tokens;  // threads past the end read the last token and write nothing
    if (!live) token = p.tokens - 1;
    const long long b = token / p.N;
    const long long n = token - b * p.N;
    float c[PAIRS], s[PAIRS];
    const int* pos = p.pos + b * p.pos_b + n * p.A;
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const int pair = chunk * PAIRS + j;
      const long long at = pos[p.axis[pair]];
      rope_cos_sin((unsigned long long)at * p.freq[pair], c[j], s[j]);
    }
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
      const NormTensor& t = p.t[ti];
      const int base = ti ? p.t[0].H : 0;
      const int lo = max(h0, base) - base, hi = min(h1, base + t.H) - base;
      if (lo >= hi) continue;
      float w[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i)
        w[i] = !t.w ? 1.f : (p.w_f32 ? static_cast<const float*>(t.w)[column(i)]
                                     : rope_f(static_cast<const T*>(t.w)[column(i)]));
      const T* xp = static_cast<const T*>(t.x) + b * t.x_b + n * t.x_n + chunk * E;
      const T* dp = static_cast<const T*>(t.dy) + b * t.dy_b + n * t.dy_n + chunk * E;
      T* op = static_cast<T*>(t.out) + b * t.out_b + n * t.out_n + chunk * E;
      for (int h = lo; h < hi; h += BATCH) {
        Vec xv[BATCH][PIECES], dv[BACK ? BATCH : 1][PIECES];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          const long long hh = min(h + u, hi - 1);  // (past the end: the last head again, not written)
#pragma unroll
          for (int k = 0; k < PIECES; ++k) {
            xv[u][k].load(xp + hh * t.x_h + k * (D / 2));
            if constexpr (BACK) dv[u][k].load(dp + hh * t.dy_h + k * (D / 2));
          }
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          float x[NE], y[NE];
          float sq = 0.f, along = 0.f;
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            x[i] = rope_f(xv[u][i / E].v[i % E]);
            sq = fmaf(x[i], x[i], sq);
          }
          if constexpr (BACK) {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
              const int i0 = HALVES ? j : 2 * j, i1 = HALVES ? E + j : 2 * j + 1;
              const float d0 = rope_f(dv[u][i0 / E].v[i0 % E]), d1 = rope_f(dv[u][i1 / E].v[i1 % E]);
              y[i0] = d0 * c[j] + d1 * s[j];  // g
              y[i1] = d1 * c[j] - d0 * s[j];
              along = fmaf(y[i0] * w[i0], x[i0], along);
              along = fmaf(y[i1] * w[i1], x[i1], along);
            }
            along = norm_row_sum<CHUNKS>(along);
          }
          sq = norm_row_sum<CHUNKS>(sq);
          const float r = rsqrtf(fmaf(sq, 1.f / D, p.eps));
          if constexpr (BACK) {
            const float mean = r > 0.f ? along * r * (1.f / D) : 0.f;  // (r = 0: a row of zeros; `along` may be inf)
            const bool count = live && h + u < hi;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
              const float nrm = x[i] * r;
              if (count) acc[i] = fmaf(y[i], nrm, acc[i]);
              y[i] = r * (y[i] * w[i] - nrm * mean);
            }
          } else {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
              const int i0 = HALVES ? j : 2 * j, i1 = HALVES ? E + j : 2 * j + 1;
              const float a = x[i0] * r * w[i0], e = x[i1] * r * w[i1];
              y[i0] = a * c[j] - e * s[j];
              y[i1] = a * s[j] + e * c[j];
            }
          }
          if (live && h + u < hi) {
#pragma unroll
            for (int k = 0; k < PIECES; ++k) {
              Vec o;
#pragma unroll
              for (int i = 0; i < E; ++i) o.v[i] = rope_t<T>(y[k * E + i]);
              o.store(op + (long long)(h + u) * t.out_h + k * (D / 2));
            }
          }
        }
      }
    }
  };
  if constexpr (BACK) {  // an even share of all batches, in order
    __shared__ float sum[2][kNormThreads / 32][D];
    __shared__ float far[2][NE][kNormThreads];  // each thread's earlier sums, and what these round off
    constexpr int CHAIN = 32 / BATCH;           // batches of heads that acc takes up before it goes there
    const long long split = p.blocks * p.batches[0];
    long long i = p.items * blockIdx.x / gridDim.x;
    const long long end = p.items * (blockIdx.x + 1LL) / gridDim.x;
#pragma unroll 1
    for (int ti = 0; ti < 2; ++ti) {
      const long long base = ti ? split : 0, stop = ti ? end : min(end, split);
      const int batches = p.batches[ti], from = ti ? p.t[0].H : 0, to = ti ? p.heads : p.t[0].H;
      int held = 0, folds = 0;  // batches in acc, times that it went to far
      while (i < stop) {
        const long long tb = (i - base) / batches;
        const int first = (int)(i - base - tb * batches);
        const int n = (int)min((long long)min(batches - first, CHAIN), stop - i);
        if (p.part != nullptr && held + n > CHAIN) {
#pragma unroll
          for (int k = 0; k < NE; ++k) {
            float hi = folds ? far[0][k][threadIdx.x] : 0.f, lo = folds ? far[1][k][threadIdx.x] : 0.f;
            norm_add(hi, lo, acc[k], 0.f);
            far[0][k][threadIdx.x] = hi;
            far[1][k][threadIdx.x] = lo;
            acc[k] = 0.f;
          }
          held = 0;
          ++folds;
        }
        rows(tb, from + first * BATCH, min(from + (first + n) * BATCH, to));
        i += n;
        held += n;
      }
      if (p.part == nullptr) continue;
      // The warp's rows, then the block's warps, by twos.
      const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
      if (ti) __syncthreads();  // (the first tensor's sums have been read)
#pragma unroll
      for (int k = 0; k < NE; ++k) {
        float hi = acc[k], lo = 0.f;
        acc[k] = 0.f;
        if (folds) norm_add(hi, lo, far[0][k][threadIdx.x], far[1][k][threadIdx.x]);
#pragma unroll
        for (int m = CHUNKS; m < 32; m <<= 1) {
          hi += __shfl_xor_sync(0xffffffffu, hi, m);
          lo += __shfl_xor_sync(0xffffffffu, lo, m);
        }
        if (lane < CHUNKS) sum[0][warp][column(k)] = hi, sum[1][warp][column(k)] = lo;
      }
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kNormThreads) {
        float v[2][kNormThreads / 32];
#pragma unroll
        for (int k = 0; k < kNormThreads / 32; ++k) v[0][k] = sum[0][k][c], v[1][k] = sum[1][k][c];
#pragma unroll
        for (int m = 1; m < kNormThreads / 32; m <<= 1)
#pragma unroll
          for (int k = 0; k < kNormThreads / 32; k += 2 * m) v[0][k] += v[0][k + m], v[1][k] += v[1][k + m];
        p.part[((long long)blockIdx.x * 2 + ti) * D + c] = v[0][0] + v[1][0];
      }
    }
  } else {
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
      const long long tb = item / p.groups;
      const int h0 = (int)(item - tb * p.groups) * p.heads_per_item;
      rows(tb, h0, min(h0 + p.heads_per_item, p.heads));
    }
  }
}

// Weights' gradients from the blocks' partial sums [rows][2][D]: a block of 32
// columns x kNormReduceRows rows of threads.
static __global__ void __launch_bounds__(32 * kNormReduceRows)
    fa_norm_weight_kernel(const float* part, int rows, int D, float* dwq, float* dwk) {
  __shared__ float sum[2][kNormReduceRows][33];
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int i = blockIdx.x * 32 + lane;  // of 2 D
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
  float hi = 0.f, lo = 0.f;
  for (int k = row; k < rows; k += kNormReduceRows) norm_add(hi, lo, part[(long long)k * 2 * D + i], 0.f);
  sum[0][row][lane] = hi;
  sum[1][row][lane] = lo;
  __syncthreads();
  static_assert(kNormReduceRows == 32, "a warp joins a column");
  hi = sum[0][lane][row];
  lo = sum[1][lane][row];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1)
    norm_add(hi, lo, __shfl_xor_sync(0xffffffffu, hi, m), __shfl_xor_sync(0xffffffffu, lo, m));
  const int c = blockIdx.x * 32 + row;
  float* out = c < D ? dwq : dwk;
  if (lane == 0 && out) out[c < D ? c : c - D] = hi + lo;
}

}  // namespace fa
