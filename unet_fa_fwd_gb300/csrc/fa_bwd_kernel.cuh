// fa_bwd_kernel.cuh — the sm_103a attention gradient.
//
// With t_ij = log2(e) (scale q_i . k_j + mask_ij), L_i = log2(e) LSE_i from the
// forward and delta_i = dO_i . O_i - dLSE_i:
//   P_ij = 2^(t_ij - L_i),  dP_ij = dO_i . V_j,  dS_ij = P_ij (dP_ij - delta_i),
//   dV_j = sum_i P_ij dO_i,  dK_j = scale sum_i dS_ij Q_i,  dQ_i = scale sum_j dS_ij K_j.
// P is recomputed from L (no running maximum), so a tile's work is two products
// into tensor memory, one pass of the threads, and the products of its results.
// A row all of whose keys lie under a large finite mask has an LSE whose fp32 step
// hides the sum; there L is summed again, of scores less the row's largest mask
// value (bwd_resum), and t_ij is taken less that value too.
//
// Two kinds of unit, of 128 rows: keys (dK, dV; products S^T, dP^T, dV, dK) and
// queries (dQ; S, dP, dQ).  Seven products for the five that one kind would need:
// it would have to add dQ up in device memory across the key units, whose order
// changes the result from run to run, and move 64 KB of it a tile through shared
// memory or L2 atomics, where it would wait about as long as the two products
// take (an SM reads 128 bytes a clock of operands: the 64 KB of a 128 x 128 x 128
// product whose operands are in shared memory take as long as the product).
// Here every sum stays in tensor memory and results repeat bit for bit.
//
// One launch holds both kinds: the first CTAs (one per SM) walk key units, the
// rest query units, which start as SMs get free.  640 threads a CTA:
//   warps 0-15   four warpgroups, each with 32 of a tile's 128 columns; a warp
//                has 32 rows of the unit (lanes of tensor memory)
//   warp 16      TMA producer      warp 17  MMA issuer (owns tensor memory)
// Four warps a sub-partition: with two (64 columns a thread) heads of 64 take
// 8 % longer (measured on an earlier form of the loop), heads of 128 the same.
// L and delta are a query's: in query units a row's, so that a thread has one row
// and 32 columns; in key units a column's, where a thread has 4 rows and 8 columns
// (the 16 x 256 bit shape of tensor memory's accesses) and so a fourth of the reads
// of shared memory, whose 128 bytes a clock bound the kernel at D = 128: the
// operands and arriving tiles of a 128 x 128 tile take 2048 clocks (as long as its
// products), L and delta 512 more with a row a thread, 128 so.
// P and dS go back to tensor memory as bf16, the A operand of the products that
// take them; both sides' rows are operands K-major for S and dP and MN-major for
// the gradients, from one copy in shared memory.
//
// What bounds it.  D = 128: the tensor pipe, 83 % active with operands at the rate of
// shared memory, and for long runs the GPU's power: 4608 tokens of 24 heads 486 to
// 502 us, 16896 6.5 to 6.9 ms, 1.27 to 1.34 PFLOP/s of the five products that the
// gradient needs, 1.8 of the seven taken.  D = 64: a thread's chain of waits, loads of
// tensor memory, exponentials and roundings, whose phases all warps are in together
// (issue slots 57 % used, tensor pipe 59, exponential units 34): 4096 tokens of 8
// heads, batch 2, 174 us, 0.99 PFLOP/s.
//
// Waits are bounded: past the limit a CTA records FA_ERR_TIMEOUT in the device
// status word, drains its copies and MMAs, frees tensor memory and returns.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fa_bwd_geom.h"
#include "fa_fwd_kernel.cuh"
#include "sm100_ptx.cuh"

namespace fa {

// How masks are read (a kernel instantiation each).
enum : int { kBwdMaskNone = 0, kBwdMaskKey = 1, kBwdMaskAdd = 2, kBwdMaskBool = 3 };

// Strides of a [B][H][N][D] tensor, in elements.
struct BwdTensor {
  __nv_bfloat16* p;
  long long b, h, n;
};

// Of 128 queries (a tile), in the workspace: -L (-inf for rows that see nothing and rows
// past Nq) and -delta; under masks also flags, a byte for each warp that made them (16),
// and under fp32 masks negated references (0 where L is LSE's).
constexpr int kStatDelta = 128, kStatTile = 256, kFlagTile = 4;  // words
enum : uint32_t {  // (of the four bytes of a word)
  kFlagRefs = 0x01010101,  // some rows have references
  kFlagBare = 0x02020202   // some rows that see nothing hold numbers that are not finite, or past 2^60
};

// Under a finite mask LSE may be far from the scores.  Below this bound its half step is
// 2^-11, those of L and of the mask in the log2 domain 2^-10 each, so P is within 2^-9 of
// itself (bf16, which P is rounded to, has 2^-8); a step further each doubles.  From there
// on a row has a reference, the largest mask value that it sees: its mask is taken less
// that value, and L is the sum's own.
constexpr float kWeakLse = 16384.f;
__device__ __forceinline__ bool bwd_weak(float lse) { return fabsf(lse) >= kWeakLse && fabsf(lse) < INFINITY; }

struct BwdParams {
  BwdPlan plan[2];  // key units, query units
  int Hq, Hk, group, Nq, Nk, nqp;  // nqp: queries rounded up to whole tiles
  int causal;
  float scale, scale_log2;
  const float* stat;      // [B Hq][nqp / 128][kStatTile]
  const uint32_t* flags;  // [B Hq][nqp / 128][kFlagTile]
  const float* ref;       // [B Hq][nqp]; fp32 masks
  const void* mask;     // fp32 [B][Nk] or [B][mask_heads][Nq][Nk]
  int mask_heads;
  int mask_vec;         // its rows are 16-byte aligned
  // Boolean masks as bits (1: the pair is kept), by query rows and by key rows.
  const uint32_t* bits_q;  // [B][mask_heads][Nq][words_q]
  const uint32_t* bits_k;  // [B][mask_heads][Nk][words_k]
  int words_q, words_k;
  // Tiles with a pair that is kept, as bits.  Boolean masks: by query tiles
  // [B][mask_heads][tiles][tile_words_q] and by key tiles; key padding: [B][tile_words_q].
  const uint32_t *tiles_q, *tiles_k;
  int tile_words_q, tile_words_k;
  BwdTensor dq, dk, dv;
  float* part[2];       // partial sums of cut units
  unsigned long long timeout_ns;
  int* status;
  int* debug_record;
  int inject_stall;
  FastDiv div_hq, div_hk, div_group;
  CUtensorMap q, k, v, dout;
};

constexpr int kBwdGroups = 4;                    // warpgroups of rows
constexpr int kBwdWarps = 4 * kBwdGroups;
constexpr int kBwdCols = 128 / kBwdGroups;       // columns a thread has of a tile
constexpr int kBwdThreads = 32 * (kBwdWarps + 4);

template <int D, int MK>
struct BwdCfg {
  using F = Cfg<D>;
  static constexpr int TILE = 128 * D * 2;  // bytes of a 128-row tile
  // A fp32 mask's values are staged by each warp for itself, MASK_COLS columns at a time.
  static constexpr int MASK_COLS = MK != kBwdMaskAdd ? 0 : (D == 128 ? 16 : 32);
  static constexpr int MASK_BYTES = kBwdWarps * 32 * MASK_COLS * 4;
  // Rings of the walked tiles (key units: Q, read again by dK an iteration
  // later, and dO; query units: K and V).  At D = 128 the slots that fit.
  static constexpr int RING0 = D == 128 ? (MK == kBwdMaskAdd ? 2 : 3) : 4;
  static constexpr int RING1 = D == 128 ? 2 : 4;
  static constexpr int STAT_BYTES = 2 * (kStatTile + kFlagTile) * 4;  // key units: two slots of -L, -delta; of flags
  static constexpr int SMEM_BAR = 512;
  static constexpr int SMEM_USED = (2 + RING0 + RING1) * TILE + STAT_BYTES + MASK_BYTES + SMEM_BAR;
  // (more than half of the SM's, so that one CTA has its tensor memory alone)
  static constexpr int SMEM_BYTES = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
  // The launch reserves 96 registers a thread; the rows' warpgroups take from the other.
  static constexpr int REGS_ROWS = 104, REGS_OTHER = 64;
  static_assert(128 * kBwdGroups * REGS_ROWS + 128 * REGS_OTHER <= kBwdThreads * 96, "register split");
};

// Tensor memory of a kind of unit: accumulators, S (two where they fit), dP.
template <int D, bool KV>
struct BwdCols {
  static constexpr int ACC = KV ? 2 * D : D;
  static constexpr int NS = ACC + 3 * 128 <= 512 ? 2 : 1;
  static constexpr int S = ACC, DP = ACC + NS * 128;
  static_assert(DP + 128 <= 512, "tensor-memory columns");
};

constexpr int kBwdMaxRing = 4;

struct BwdBars {
  uint64_t a_full, a_empty, b_full, b_empty;  // the unit's rows
  uint64_t r0_full[kBwdMaxRing], r0_empty[kBwdMaxRing], r1_full[kBwdMaxRing], r1_empty[kBwdMaxRing];
  uint64_t st_full[2], st_empty[2];
  uint64_t s_full[2], p_ready[2], dp_full, dp_free, ds_ready[2], acc_full, drain;
  uint32_t tmem_base;
  volatile int abort_flag;
};
static_assert(sizeof(BwdBars) <= 512, "barriers");

static __device__ __forceinline__ bool bwd_wait_slow(uint32_t bar, uint32_t parity, BwdBars* bars,
                                                  unsigned long long timeout_ns, int* status) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (true) {
    if (ptx::mbar_try_wait_sleep(bar, parity, kSuspendNs)) return true;
    if (bars->abort_flag) return false;
    if (ptx::global_timer_ns() - t0 > timeout_ns) {
      bars->abort_flag = 1;
      atomicCAS(status, 0, kStatusTimeout);
      return false;
    }
  }
}

// Bounded wait for an mbarrier phase, by one thread or by a whole warp.
__device__ __forceinline__ bool bwd_wait(uint64_t& bar, uint32_t parity, BwdBars* bars, const BwdParams& p) {
  const uint32_t b = ptx::smem_u32(&bar);
  return ptx::mbar_try_wait(b, parity) || bwd_wait_slow(b, parity, bars, p.timeout_ns, p.status);
}
__device__ __forceinline__ bool bwd_wait_warp(uint64_t& bar, uint32_t parity, BwdBars* bars, const BwdParams& p) {
  const uint32_t b = ptx::smem_u32(&bar);
  if (__all_sync(0xffffffffu, ptx::mbar_try_wait(b, parity))) return true;
  return __all_sync(0xffffffffu, bwd_wait_slow(b, parity, bars, p.timeout_ns, p.status));
}

// Two phases (the first nullptr: one) by a whole warp, asked for at once.
__device__ __forceinline__ bool bwd_wait_warp(uint64_t* b0, uint32_t p0, uint64_t& b1, uint32_t p1, BwdBars* bars,
                                              const BwdParams& p) {
  bool there = ptx::mbar_try_wait(ptx::smem_u32(&b1), p1);
  if (b0) there = ptx::mbar_try_wait(ptx::smem_u32(b0), p0) && there;
  if (__all_sync(0xffffffffu, there)) return true;
  return (!b0 || bwd_wait_warp(*b0, p0, bars, p)) && bwd_wait_warp(b1, p1, bars, p);
}

// Debug builds: see fa_check.
enum : int { kCheckGradUnit = 8, kCheckGradStore = 9, kCheckGradSlot = 10 };
__device__ __forceinline__ bool bwd_check(const BwdParams& p, BwdBars* bars, bool cond, int id, long long a,
                                          long long b) {
#ifdef FA_DEBUG
  if (!cond) {
    atomicCAS(p.status, 0, kStatusDebugCheck);
    if (atomicCAS(&p.debug_record[0], 0, id) == 0) {
      p.debug_record[1] = (int)blockIdx.x;
      p.debug_record[2] = (int)threadIdx.x;
      p.debug_record[3] = (int)a;
      p.debug_record[4] = (int)b;
    }
    atomicAdd(&p.debug_record[7], 1);
    bars->abort_flag = 1;
  }
  return cond;
#else
  (void)p; (void)bars; (void)id; (void)a; (void)b;
  return cond || true;
#endif
}

// Untiled copy global -> shared (both 16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// S = A B^T of two K-major 128-row tiles into 128 columns at d.
template <int D>
__device__ __forceinline__ void bwd_mma_scores(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi) {
  using C = Cfg<D>;
  constexpr uint32_t IDESC = make_idesc(128, 128, false);
  if constexpr (D == 128)
    ptx::mma_ss_x8_el<C::s_off(1), C::s_off(2), C::s_off(3), C::s_off(4), C::s_off(5), C::s_off(6), C::s_off(7)>(
        d, a_lo, hi, b_lo, hi, IDESC, 0);
  else if constexpr (D == 64)
    ptx::mma_ss_x4_el<C::s_off(1), C::s_off(2), C::s_off(3)>(d, a_lo, hi, b_lo, hi, IDESC, 0);
  else
    ptx::mma_ss_x2_el<C::s_off(1)>(d, a_lo, hi, b_lo, hi, IDESC, 0);
}

// acc += X T: X bf16 in tensor memory, each warpgroup's 32 columns at the start
// of the 32 that they were computed from; T a 128-row tile, MN-major.
template <int D>
__device__ __forceinline__ void bwd_mma_grad(uint32_t acc, uint32_t x, uint32_t t_lo, uint32_t t_hi, bool first) {
  constexpr uint32_t IDESC = make_idesc(128, D, true);
  constexpr uint32_t STEP = (16 * Cfg<D>::SW) >> 4;
  ptx::mma_ts_x8_by2_el<STEP>(acc, x, t_lo, t_hi, IDESC, first ? 0u : 1u);
}

template <int D>
__device__ __forceinline__ void bwd_load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row, int h,
                                              int b) {
  using C = Cfg<D>;
#pragma unroll
  for (int c = 0; c < C::NCHUNK; ++c)
    ptx::tma_load_4d(dst + c * C::CHUNK_BYTES, map, bar, c * C::CHUNK_ELEMS, row, h, b);
}

// Staging of a fp32 mask [rows][Nk]: a warp copies the values of its 32 rows and
// SC columns of a tile into `buf` (its own), for itself.  Key units (KV): a
// warp's rows are keys and columns are queries, kept as [SC][32], each pair of
// queries turned by 8 keys more; query units: a row's SC values together, 16-byte
// pieces swizzled.  So the lanes' reads do not meet.  Values outside the mask read 0.
template <bool KV, int SC>
struct BwdStage {
  static constexpr int PIECES = SC / 4;
  static __device__ __forceinline__ int swizzle(int r) { return SC == 32 ? (r & 7) : ((r >> 1) & 3); }
  static __device__ __forceinline__ int turned(int key, int c) { return (key + 8 * (c / 2)) & 31; }
  // (Addresses go up by a constant from copy to copy: the mask's cost is
  // instructions.  What lies outside copies no byte and is zero.)
  static __device__ __forceinline__ void copy(uint32_t buf, const float* base, int row0, int col0, int Nq, int Nk,
                                              int vec, int lane) {
    const int q0 = KV ? col0 : row0, k0 = KV ? row0 : col0;
    if (vec) {  // 16 bytes a lane (Nk is a multiple of 4)
      constexpr int LANES = KV ? 8 : PIECES, STEP = 32 / LANES;  // of a mask row; mask rows a copy
      const int r = lane / LANES, g = lane % LANES, k = k0 + 4 * g;
      const float* src = base + (size_t)(q0 + r) * Nk + k;
      const size_t step = (size_t)STEP * Nk;
      const int rows = k < Nk ? Nq - q0 - r : 0;
      // 16-byte piece of the row; other in every second copy by `flip`
      const int piece = KV ? (g + 2 * (r / 2)) & 7 : g ^ swizzle(r);
      constexpr int flip = KV || SC == 32 ? 4 : 0, ROW = KV ? 128 : SC * 4;
      const uint32_t dst = buf + r * ROW;
#pragma unroll
      for (int i = 0; i < PIECES; ++i, src += step)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * STEP * ROW +
                                                                          ((piece ^ (i % 2 * flip)) << 4)),
                     "l"(src), "r"(i * STEP < rows ? 16 : 0)
                     : "memory");
    } else {  // 4 bytes a lane
      constexpr int LANES = KV ? 32 : SC, STEP = 32 / LANES;
      const int r = lane / LANES, c = lane % LANES, k = k0 + c;
      const float* src = base + (size_t)(q0 + r) * Nk + k;
      const size_t step = (size_t)STEP * Nk;
      const int rows = k < Nk ? Nq - q0 - r : 0;
#pragma unroll 8
      for (int i = 0; i < SC; ++i, src += step) {
        const int at = KV ? i * 32 + turned(c, i)
                          : (i * STEP + r) * SC + (((c / 4) ^ swizzle(i * STEP + r)) << 2) + c % 4;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(buf + at * 4), "l"(src),
                     "r"(i * STEP < rows ? 4 : 0)
                     : "memory");
      }
    }
  }
  // Adds the negated references (key units: of the SC queries from ref[0] on; query units:
  // of the lane's row) to what has been staged.
  static __device__ __forceinline__ void refer(float* buf, const float* ref, int lane) {
    const float own = KV ? (lane < SC ? __ldcg(ref + lane) : 0.f) : *ref;
#pragma unroll 1
    for (int c = 0; c < SC; ++c)
      buf[KV ? c * 32 + lane : lane * SC + c] += KV ? __shfl_sync(0xffffffffu, own, c) : own;
    __syncwarp();
  }
  // The lane's 16 values of the columns c0 .. c0 + 15 (key units: of 4 rows and 4
  // columns, in the order of bwd_elements).
  static __device__ __forceinline__ void read(const float* buf, int c0, int lane, float (&m)[16]) {
    if constexpr (KV) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int c = c0 + 8 * (e / 8) + 2 * (lane % 4) + e % 2, key = lane / 4 + 8 * (e / 2 % 4);
        m[e] = buf[c * 32 + turned(key, c)];
      }
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 v = *reinterpret_cast<const float4*>(buf + lane * SC + (((c0 / 4 + g) ^ swizzle(lane)) << 2));
        m[4 * g] = v.x;
        m[4 * g + 1] = v.y;
        m[4 * g + 2] = v.z;
        m[4 * g + 3] = v.w;
      }
    }
  }
};

// The 32 elements that a thread has of a tile, from the 32 columns at `t`.  Query
// units: its row's 32 columns.  Key units (bwd_elements): element 8 i + 2 r + c is
// row lane / 4 + 8 r, column 8 i + 2 (lane % 4) + c.
template <bool KV>
__device__ __forceinline__ void bwd_load_elements(uint32_t t, uint32_t (&r)[32]) {
  if constexpr (KV)
    ptx::tmem_ld2x16x256b_x4(t, r);
  else
    ptx::tmem_ld32x32b_x32(t, r);
}
// Of a key unit the elements of the 8 columns at `t` (i = 0).
__device__ __forceinline__ void bwd_load_elements(uint32_t t, uint32_t (&r)[8]) { ptx::tmem_ld2x16x256b_x1(t, r); }
// Pairs of a key unit's elements in that order, as the 16 columns at `t`.
__device__ __forceinline__ void bwd_store_pairs(uint32_t t, const uint32_t (&w)[16]) { ptx::tmem_st2x16x128b_x4(t, w); }

// NC columns of a thread's accumulator row at `t`, times `mul`, rounded to `dst`
// (16-byte aligned; neighbouring lanes' rows are `row_step` elements apart; `rows`:
// how many from the lane's on are in the tensor).  Neighbouring lanes first exchange
// 16-byte pieces so that up to four store 64 bytes of one row together: a store of
// every lane to a row of its own takes a clock a row (units of one tile each at
// D = 64: 1100 clocks of 4050).
// `keep` false: the lane's own row is zeros (`zero`: every row of the warp).
template <int NC>
__device__ __forceinline__ void bwd_store_row(uint32_t t, float mul, bool zero, bool keep, bool ok, int rows, int lane,
                                              __nv_bfloat16* dst, long long row_step) {
  constexpr int CH = NC >= 32 ? 4 : NC / 8;  // lanes that share rows, and their pieces
  const int l = lane % CH;
#pragma unroll
  for (int cb = 0; cb < NC; cb += 8 * CH) {
    uint32_t v[CH][4];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      uint32_t r[8];
      if (zero) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = 0u;
      } else {
        ptx::tmem_ld32x32b_x8(t + cb + 8 * c, r);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[c][i] = keep ? ptx::pack_bf16x2(__uint_as_float(r[2 * i]) * mul, __uint_as_float(r[2 * i + 1]) * mul) : 0u;
    }
    // v[c] of lane l becomes piece l of lane c's row.
#pragma unroll
    for (int m = 1; m < CH; m <<= 1)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (c & m) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool upper = (l & m) != 0;
          const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? v[c][i] : v[c | m][i], m);
          if (upper)
            v[c][i] = got;
          else
            v[c | m][i] = got;
        }
      }
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (ok && c - l < rows)
        *reinterpret_cast<uint4*>(dst + (c - l) * row_step + cb + 8 * l) = make_uint4(v[c][0], v[c][1], v[c][2], v[c][3]);
  }
}
template <int NC>
__device__ __forceinline__ void bwd_store_part(uint32_t t, bool zero, bool keep, bool ok, float* dst, int row) {
#pragma unroll
  for (int cb = 0; cb < NC; cb += 8) {
    uint32_t r[8];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = 0u;
    } else {
      ptx::tmem_ld32x32b_x8(t + cb, r);
      if (!keep) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = 0u;
      }
    }
    if (ok) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<uint4*>(dst + ((size_t)(cb / 4 + q) * 128 + row) * 4) =
            make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
    }
  }
}

// Where a piece's iterations lie: query head (of a group that shares the key
// head) and tile of the other side.  Tiles of which a boolean or key-padding mask
// keeps nothing are left out (their P and dS are 0); `count` is how many are left.
template <int MK, bool KV>
struct BwdIter {
  static constexpr bool SKIP = MK == kBwdMaskBool || (MK == kBwdMaskKey && !KV);
  int g, tile;    // head in the group, tile
  int first, n;
  int it, end;    // as if none were left out
  int count;
  const uint32_t* words;  // tiles' bits, of the group's first head
  int words_head;         // from one head of the group to the next

  __device__ __forceinline__ void start(const BwdParams& p, const BwdUnits& u, const BwdPiece& pc, int b, int h) {
    u.range(pc.tile, first, n);
    it = pc.it0;
    end = pc.it1;
    g = n > 0 && u.group > 1 ? it / n : 0;
    tile = first + it - g * n;
    count = end - it;
    if constexpr (MK == kBwdMaskKey) {
      words = p.tiles_q + (size_t)b * p.tile_words_q;
      words_head = 0;
      if (KV && !((words[pc.tile / 32] >> (pc.tile % 32)) & 1u)) count = 0;
    } else if constexpr (MK == kBwdMaskBool) {
      const int head = p.mask_heads == 1 ? 0 : (KV ? h * p.group : h), per = KV ? p.tile_words_k : p.tile_words_q;
      words = (KV ? p.tiles_k : p.tiles_q) + ((size_t)(b * p.mask_heads + head) * u.tiles + pc.tile) * per;
      words_head = p.mask_heads == 1 ? 0 : u.tiles * per;
    }
    if constexpr (SKIP) {
      count = 0;
      BwdIter i = *this;
      while (i.it < end) {
        int span;
        count += __popc(i.ahead(span));
        i.move(span);
      }
      seek();
    }
  }
  // Bits of the next tiles that share a word, and how many these are.
  __device__ __forceinline__ uint32_t ahead(int& span) const {
    span = min(min(32 - tile % 32, first + n - tile), end - it);
    return words[(size_t)g * words_head + tile / 32] >> (tile % 32) & (~0u >> (32 - span));
  }
  __device__ __forceinline__ void move(int by) {
    it += by;
    tile += by;
    if (tile == first + n) {
      tile = first;
      ++g;
    }
  }
  __device__ __forceinline__ void seek() {
    while (it < end) {
      int span;
      const uint32_t w = ahead(span);
      if (w) {
        move(__ffs(w) - 1);
        return;
      }
      move(span);
    }
  }
  __device__ __forceinline__ void next() {
    move(1);
    if constexpr (SKIP) seek();
  }
};

// Key units: what a tile's queries that see nothing hold goes nowhere.  Their P and dS
// are 0, but 0 times what is not finite is not: their rows of Q and dO become zeros before
// the products that sum over queries, and their columns of S and dP too (S may be inf
// where q is merely large).  By all rows' warps, ahead of their P, each for 8 rows and its
// own part of tensor memory; false: a wait ran out.
template <int D>
__device__ __noinline__ bool bwd_scrub(const BwdParams& p, BwdBars* bars, const float* nlse, uint32_t tS, uint32_t tDP,
                                       uint8_t* q, uint8_t* dout, uint32_t dp_parity) {
  using F = Cfg<D>;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, col0 = warp / 4 * kBwdCols;
  if (!bwd_wait_warp(bars->dp_full, dp_parity, bars, p)) return false;  // (dP reads dO until then)
  ptx::tc_fence_after_sync();
  for (int i = 0; i < kBwdCols; i += 8) {
    uint32_t s[8], d[8];
    ptx::tmem_ld32x32b_x8(tS + i, s);
    ptx::tmem_ld32x32b_x8(tDP + i, d);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (nlse[col0 + i + c] == -INFINITY) s[c] = d[c] = 0u;
    ptx::tmem_st32x32b_x8(tS + i, s);
    ptx::tmem_st32x32b_x8(tDP + i, d);
  }
  ptx::tmem_wait_st();
  // A row is D / (64 or 32) spans of the swizzle, which moves 16-byte pieces within one.
  constexpr int BYTES = D / 2;  // of a lane, a quarter of a row
  const int row = warp * 8 + lane / 4, at = lane % 4 * BYTES;
  if (nlse[row] == -INFINITY) {
    const int off = at / F::SW * F::CHUNK_BYTES + row * F::SW + at % F::SW;
#pragma unroll
    for (int i = 0; i < BYTES; i += 16)
      *reinterpret_cast<uint4*>(q + off + i) = *reinterpret_cast<uint4*>(dout + off + i) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the products that follow see the zeros
  __syncwarp();
  return true;
}

// A CTA's units of one kind: dK and dV of 128 keys (KV), or dQ of 128 queries.
template <int D, int MK, bool KV>
__device__ __forceinline__ void bwd_units(const BwdParams& p, int cta, uint8_t* smem, BwdBars* bars, uint32_t tmem) {
  using C = BwdCfg<D, MK>;
  using T = BwdCols<D, KV>;
  using F = Cfg<D>;
  const BwdPlan& plan = p.plan[KV ? 0 : 1];
  uint8_t* sA = smem;  // the unit's rows: K and V, or Q and dO
  uint8_t* sB = sA + C::TILE;
  uint8_t* sR0 = sB + C::TILE;  // the tiles it walks
  uint8_t* sR1 = sR0 + C::RING0 * C::TILE;
  float* sStat = reinterpret_cast<float*>(sR1 + C::RING1 * C::TILE);
  // (from lane 0, so that the compiler knows that a warp's lanes agree)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0);
  const uint32_t lane = threadIdx.x % 32;
  auto finish = [&]() {
    ptx::named_barrier_sync(1, kBwdThreads);
    if (warp == kBwdWarps + 1) {
      ptx::tc_fence_after_sync();
      ptx::tmem_dealloc(tmem, 512);
    }
  };
  auto piece_ok = [&](const BwdPiece& pc) {
    return bwd_check(p, bars, pc.head >= 0 && pc.head < plan.units.heads && pc.tile >= 0 &&
                                  pc.tile < plan.units.tiles && pc.it0 >= 0 &&
                                  pc.it1 <= plan.units.iterations(pc.tile) && pc.it0 <= pc.it1,
                     kCheckGradUnit, pc.head, pc.tile);
  };
  const int heads = KV ? p.Hk : p.Hq;
  const FastDiv& div_h = KV ? p.div_hk : p.div_hq;
  auto query_tile = [&](int b, int hq, int tile) { return ((size_t)b * p.Hq + hq) * (p.nqp / 128) + tile; };

  if (warp >= kBwdWarps) {
    ptx::setmaxnreg_dec<C::REGS_OTHER>();
    if (warp == kBwdWarps) {
      // ---------------------------------------------------------- producer --
      if (lane == 0) {
        const CUtensorMap *mA = KV ? &p.k : &p.q, *mB = KV ? &p.v : &p.dout;
        const CUtensorMap *m0 = KV ? &p.q : &p.k, *m1 = KV ? &p.dout : &p.v;
        ptx::tma_prefetch_desc(mA);
        ptx::tma_prefetch_desc(m0);
        ptx::tma_prefetch_desc(mB);
        ptx::tma_prefetch_desc(m1);
        uint32_t na = 0, nb = 0, j = 0;  // tiles of the unit's rows, iterations begun
        uint32_t n0 = 0, n1 = 0, nst = 0;  // copies issued to each ring
        bool ok = true;
        BwdWalk walk;
        BwdPiece pc;
        while (ok && walk.next(plan, cta, pc)) {
          if (!piece_ok(pc)) break;
          if (pc.it0 == pc.it1) continue;
          const int b = (int)div_h.div((uint32_t)pc.head), h = pc.head - b * heads;
          // heads of the tiles walked: a group of query heads, or the key head
          const int h_other = KV ? h * p.group : (int)p.div_group.div((uint32_t)h);
          auto load_unit = [&](const CUtensorMap* map, uint8_t* dst, uint64_t& full, uint64_t& empty, uint32_t& n) {
            if (!bwd_wait(empty, (n & 1) ^ 1, bars, p)) return false;
            ptx::mbar_arrive_expect_tx(ptx::smem_u32(&full), C::TILE);
            bwd_load_tile<D>(ptx::smem_u32(dst), map, ptx::smem_u32(&full), pc.tile * 128, h, b);
            ++n;
            return true;
          };
          BwdIter<MK, KV> at;
          at.start(p, plan.units, pc, b, h);
          for (int i = 0; ok && i < at.count; ++i, ++j, at.next()) {
            const int ho = h_other + (KV ? at.g : 0);
            if (i == 0) ok = load_unit(mA, sA, bars->a_full, bars->a_empty, na);
            if (!ok) break;
            const uint32_t s0 = j % C::RING0, s1 = j % C::RING1;
            ok = bwd_wait(bars->r0_empty[s0], ((j / C::RING0) & 1) ^ 1, bars, p);
            if (!ok) break;
            if (p.inject_stall && blockIdx.x == 0 && j == 3) {  // nothing arrives: the others time out
              ok = false;
              break;
            }
            uint32_t full = ptx::smem_u32(&bars->r0_full[s0]);
            ptx::mbar_arrive_expect_tx(full, C::TILE);
            bwd_load_tile<D>(ptx::smem_u32(sR0 + s0 * C::TILE), m0, full, at.tile * 128, ho, b);
            ++n0;
            if (i == 0) ok = load_unit(mB, sB, bars->b_full, bars->b_empty, nb);
            if (!ok) break;
            if constexpr (KV) {
              const uint32_t ss = j & 1;
              ok = bwd_wait(bars->st_empty[ss], ((j / 2) & 1) ^ 1, bars, p);
              if (!ok) break;
              full = ptx::smem_u32(&bars->st_full[ss]);
              constexpr bool FLAGS = MK != kBwdMaskNone;
              const size_t qt = query_tile(b, ho, at.tile);
              ptx::mbar_arrive_expect_tx(full, (kStatTile + (FLAGS ? kFlagTile : 0)) * 4);
              bulk_load(ptx::smem_u32(sStat + ss * kStatTile), p.stat + qt * kStatTile, kStatTile * 4, full);
              if constexpr (FLAGS)
                bulk_load(ptx::smem_u32(sStat + 2 * kStatTile + ss * kFlagTile), p.flags + qt * kFlagTile,
                          kFlagTile * 4, full);
              ++nst;
            }
            ok = bwd_wait(bars->r1_empty[s1], ((j / C::RING1) & 1) ^ 1, bars, p);
            if (!ok) break;
            full = ptx::smem_u32(&bars->r1_full[s1]);
            ptx::mbar_arrive_expect_tx(full, C::TILE);
            bwd_load_tile<D>(ptx::smem_u32(sR1 + s1 * C::TILE), m1, full, at.tile * 128, ho, b);
            ++n1;
          }
        }
        // Wait (bounded) until every copy has landed: after an abort nobody
        // else waits for them, and the CTA must not exit with copies in flight.
        auto landed = [&](uint64_t& bar, uint32_t n) {
          if (n == 0) return;
          const uint64_t t0 = ptx::global_timer_ns();
          while (!ptx::mbar_try_wait(ptx::smem_u32(&bar), (n - 1) & 1) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
          }
        };
        landed(bars->a_full, na);
        landed(bars->b_full, nb);
        for (uint32_t s = 0; s < C::RING0; ++s) landed(bars->r0_full[s], (n0 + C::RING0 - 1 - s) / C::RING0);
        for (uint32_t s = 0; s < C::RING1; ++s) landed(bars->r1_full[s], (n1 + C::RING1 - 1 - s) / C::RING1);
        for (uint32_t s = 0; s < 2; ++s) landed(bars->st_full[s], (nst + 1 - s) / 2);
      }
      __syncwarp();
    } else if (warp == kBwdWarps + 1) {
      // --------------------------------------------------------------- MMA --
      // Descriptors: K-major (scores) and MN-major (gradients) views of the tiles.
      const uint64_t k_major = smem_desc(0, 16, F::SBO, F::LAYOUT);
      const uint64_t mn_major = smem_desc(0, F::CHUNK_BYTES, F::SBO, F::LAYOUT);
      const uint32_t k_hi = (uint32_t)(k_major >> 32), k_lo = (uint32_t)k_major;
      const uint32_t mn_hi = (uint32_t)(mn_major >> 32), mn_lo = (uint32_t)mn_major;
      auto at16 = [](const uint8_t* s) { return ptx::smem_u32(s) >> 4; };
      const uint32_t a16 = at16(sA), b16 = at16(sB), r0 = at16(sR0), r1 = at16(sR1);
      constexpr uint32_t TILE16 = C::TILE >> 4;
      uint32_t nu = 0;  // pieces
      uint32_t j = 0;   // iterations
      bool ok = true;
      auto commit = [&](uint64_t& b) { ptx::mma_commit_el(ptx::smem_u32(&b)); };
      // S (dP) of iteration i: the unit's rows by the ring's tile.
      auto scores = [&](uint32_t i) -> bool {
        const uint32_t s = i % C::RING0;
        if (!bwd_wait_warp(bars->r0_full[s], (i / C::RING0) & 1, bars, p)) return false;
        ptx::tc_fence_after_sync();
        bwd_mma_scores<D>(tmem + T::S + (i % T::NS) * 128, k_lo + a16, k_lo + r0 + s * TILE16, k_hi);
        commit(bars->s_full[i % T::NS]);
        return true;
      };
      auto dprob = [&](uint32_t i) -> bool {
        const uint32_t s = i % C::RING1;
        if (!bwd_wait_warp(bars->r1_full[s], (i / C::RING1) & 1, bars, p)) return false;
        ptx::tc_fence_after_sync();
        bwd_mma_scores<D>(tmem + T::DP, k_lo + b16, k_lo + r1 + s * TILE16, k_hi);
        commit(bars->dp_full);
        if constexpr (!KV) commit(bars->r1_empty[s]);  // V is not needed again
        return true;
      };
      BwdWalk walk;
      BwdPiece pc;
      while (ok && walk.next(plan, cta, pc)) {
        if (!__all_sync(0xffffffffu, piece_ok(pc))) break;
        const int b = (int)div_h.div((uint32_t)pc.head);
        BwdIter<MK, KV> at;
        at.start(p, plan.units, pc, b, pc.head - b * heads);
        const uint32_t n = (uint32_t)at.count;
        if (n == 0) continue;
        ok = bwd_wait_warp(bars->a_full, nu & 1, bars, p) && scores(j);
        if (ok && n == 1) commit(bars->a_empty);
        ok = ok && bwd_wait_warp(bars->b_full, nu & 1, bars, p) && dprob(j);
        if (ok && n == 1) commit(bars->b_empty);
        if (ok && T::NS == 2 && n > 1) {
          ok = scores(j + 1);
          if (ok && n == 2) commit(bars->a_empty);
        }
        if (!ok) break;
        for (uint32_t i = 0; ok && i < n; ++i, ++j) {
          const uint32_t s0 = j % C::RING0, s1 = j % C::RING1, sb = j % T::NS;
          const uint32_t tS = tmem + T::S + sb * 128;
          if constexpr (KV) {
            // dV += P^T dO
            ok = bwd_wait_warp(bars->p_ready[sb], (j / T::NS) & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_mma_grad<D>(tmem, tS, mn_lo + r1 + s1 * TILE16, mn_hi, i == 0);
            commit(bars->r1_empty[s1]);
            if constexpr (T::NS == 1) {  // dS takes dP's place
              if (i + 1 < n) {
                ok = scores(j + 1);
                if (!ok) break;
                if (i + 2 == n) commit(bars->a_empty);
              }
            } else {  // dS lies beside P: dP is free once it has been read
              if (i + 1 < n) {
                ok = bwd_wait_warp(bars->dp_free, j & 1, bars, p) && dprob(j + 1);
                if (!ok) break;
                if (i + 2 == n) commit(bars->b_empty);
              }
            }
            // dK += dS^T Q
            ok = bwd_wait_warp(bars->ds_ready[sb], (j / T::NS) & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_mma_grad<D>(tmem + D, T::NS == 1 ? tmem + T::DP : tS + 16, mn_lo + r0 + s0 * TILE16, mn_hi, i == 0);
            commit(bars->r0_empty[s0]);
            if constexpr (T::NS == 1) {
              if (i + 1 < n) {
                ok = dprob(j + 1);
                if (!ok) break;
                if (i + 2 == n) commit(bars->b_empty);
              }
            } else {
              if (i + 2 < n) {
                ok = scores(j + 2);
                if (!ok) break;
                if (i + 3 == n) commit(bars->a_empty);
              }
            }
          } else {
            if (i + 1 < n) {
              ok = bwd_wait_warp(bars->dp_free, j & 1, bars, p);
              if (!ok) break;
              ok = dprob(j + 1);
              if (!ok) break;
              if (i + 2 == n) commit(bars->b_empty);
            }
            // dQ += dS K
            ok = bwd_wait_warp(bars->ds_ready[sb], (j / T::NS) & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_mma_grad<D>(tmem, tS, mn_lo + r0 + s0 * TILE16, mn_hi, i == 0);
            commit(bars->r0_empty[s0]);
            if (i + T::NS < n) {
              ok = scores(j + T::NS);
              if (!ok) break;
              if (i + T::NS + 1 == n) commit(bars->a_empty);
            }
          }
        }
        if (!ok) break;
        commit(bars->acc_full);
        ++nu;
      }
      // Drain this warp's MMAs before tensor memory can be freed.
      commit(bars->drain);
      const uint64_t t0 = ptx::global_timer_ns();
      while (!ptx::mbar_try_wait(ptx::smem_u32(&bars->drain), 0) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
      }
      __syncwarp();
    }
    finish();
    return;
  }

  ptx::setmaxnreg_inc<C::REGS_ROWS>();
  {
    // --------------------------------------------------------- the threads --
    const int wg = warp / 4;
    const int row = (warp % 4) * 32 + (int)lane;  // of the accumulators
    // Key units: the first of the four rows, 8 apart, and the first column of the
    // pairs, 8 apart, of this thread in a tile.
    constexpr int ROWS = KV ? 4 : 1;
    const int row4 = KV ? (warp % 4) * 32 + (int)lane / 4 : row, col2 = 2 * ((int)lane % 4);
    const uint32_t t0 = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    const float sl2 = p.scale_log2;
    constexpr float kLog2e = 1.4426950408889634f;
    auto arrive = [&](uint64_t& b) {  // one arrival per warp
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&b));
    };
    using Stage = BwdStage<KV, MK == kBwdMaskAdd ? C::MASK_COLS : 32>;
    float* sMask = sStat + C::STAT_BYTES / 4 + warp * 32 * C::MASK_COLS;
    constexpr bool REFS = MK == kBwdMaskKey || MK == kBwdMaskAdd;  // rows may have references
    uint32_t j = 0, nu = 0;
    bool ok = true;
    // A piece, and what follows from it.  The next one is made out while the last
    // products of a piece are waited for: its chain of divisions and loads takes as
    // long as a tile (units of one tile each: 2.9 us a unit for 1.9).
    struct Work {
      BwdPiece pc;
      int b, h;
      BwdIter<MK, KV> at;
      float nlse, ndelta, nref;  // of a query unit's row
    };
    BwdWalk walk;
    auto next_work = [&](Work& w) {
      if (!walk.next(plan, cta, w.pc)) return false;
      if (!__all_sync(0xffffffffu, piece_ok(w.pc))) {
        ok = false;
        return false;
      }
      w.b = (int)div_h.div((uint32_t)w.pc.head);
      w.h = w.pc.head - w.b * heads;
      w.nlse = w.ndelta = w.nref = 0.f;
      if constexpr (!KV) {
        const size_t qt = query_tile(w.b, w.h, w.pc.tile);
        w.nlse = __ldcg(p.stat + qt * kStatTile + row);
        w.ndelta = __ldcg(p.stat + qt * kStatTile + kStatDelta + row);
        if constexpr (REFS) w.nref = __ldcg(p.ref + qt * 128 + row);
      }
      w.at.start(p, plan.units, w.pc, w.b, w.h);
      return true;
    };
    Work work;
    for (bool have = next_work(work); ok && have;) {
      const BwdPiece pc = work.pc;
      const int b = work.b, h = work.h;
      const int my = pc.tile * 128 + row, my4 = pc.tile * 128 + row4;  // this thread's key or query
      const float nlse = work.nlse, ndelta = work.ndelta, nref = work.nref;
      const bool refs = MK == kBwdMaskAdd && !KV && __any_sync(0xffffffffu, nref != 0.f);
      float key_add[4] = {};
      if constexpr (KV && MK == kBwdMaskKey) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          key_add[r] = __ldg(static_cast<const float*>(p.mask) + (size_t)b * p.Nk + min(my4 + 8 * r, p.Nk - 1)) * kLog2e;
      }
      BwdIter<MK, KV> at = work.at;
      const int n = at.count;
      // The first mask values of the iteration at `i`, which are fetched an iteration ahead.
      uint32_t bits[ROWS] = {};
      auto mask_head = [&](const BwdIter<MK, KV>& i) {
        return (size_t)b * p.mask_heads + (p.mask_heads == 1 ? 0 : (KV ? h * p.group + i.g : h));
      };
      auto stage = [&](const BwdIter<MK, KV>& i, int c0) {
        Stage::copy(ptx::smem_u32(sMask), static_cast<const float*>(p.mask) + mask_head(i) * p.Nq * p.Nk,
                    pc.tile * 128 + (warp % 4) * 32, i.tile * 128 + wg * kBwdCols + c0, p.Nq, p.Nk, p.mask_vec,
                    (int)lane);
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      auto fetch = [&](const BwdIter<MK, KV>& i) {
        if constexpr (MK == kBwdMaskBool) {
          const int rows = KV ? p.Nk : p.Nq, words = KV ? p.words_k : p.words_q;
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
            bits[r] = __ldcg((KV ? p.bits_k : p.bits_q) + (mask_head(i) * rows + min(my4 + 8 * r, rows - 1)) * words +
                            i.tile * 4 + wg);
        } else if constexpr (MK == kBwdMaskAdd) {
          stage(i, 0);
        }
      };
      if (n > 0) fetch(at);
      for (int it = 0; it < n; ++it, ++j) {
        const uint32_t sb = j % T::NS;
        const uint32_t tS = t0 + T::S + sb * 128 + wg * kBwdCols, tDP = t0 + T::DP + wg * kBwdCols;
        const int col0 = at.tile * 128 + wg * kBwdCols;  // this thread's first query or key of the tile
        const BwdIter<MK, KV> now = at;
        at.next();
        const float *lcol = nullptr, *dcol = nullptr;  // -L and -delta of this thread's columns
        if constexpr (KV) {
          lcol = sStat + (j & 1) * kStatTile + wg * kBwdCols + col2;
          dcol = lcol + kStatDelta;
        }
        // Pairs that the row does not see: above the diagonal, and keys past Nk
        // (as columns; as rows their gradients are not stored).
        uint32_t seen[ROWS];
        bool edge = false;
        // (a tile that is seen whole needs no look)
        const bool below = !p.causal || (KV ? now.tile > pc.tile : now.tile < pc.tile);
        const bool whole = MK != kBwdMaskBool && below && (KV || (now.tile + 1) * 128 <= p.Nk);
        if (!whole) {
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            seen[r] = ~0u;
            if constexpr (KV) {
              if (p.causal) {
                const int lo = my4 + 8 * r - col0;  // columns from lo on
                seen[r] = lo <= 0 ? ~0u : (lo >= 32 ? 0u : ~0u << lo);
              }
            } else {
              int n = min(32, p.Nk - col0);  // columns below n
              if (p.causal) n = min(n, my - col0 + 1);
              seen[r] = n >= 32 ? ~0u : (n <= 0 ? 0u : ~0u >> (32 - n));
            }
            if constexpr (MK == kBwdMaskBool) seen[r] &= bits[r];
            edge = edge || seen[r] != ~0u;
          }
          if constexpr (MK == kBwdMaskBool) {
            if (it + 1 < n) fetch(at);
          }
          edge = __any_sync(0xffffffffu, edge);
        }
        ok = bwd_wait_warp(KV ? &bars->st_full[j & 1] : nullptr, (j / 2) & 1, bars->s_full[sb], (j / T::NS) & 1, bars, p);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        uint32_t flags = 0;  // (read ahead of the scores, whose wait hides it)
        if constexpr (KV && MK != kBwdMaskNone) {
          const uint4 f = *reinterpret_cast<const uint4*>(sStat + 2 * kStatTile + (j & 1) * kFlagTile);
          flags = f.x | f.y | f.z | f.w;
        }
        float pr[kBwdCols];  // in the order of bwd_elements
        {
          uint32_t r[kBwdCols];
          bwd_load_elements<KV>(tS, r);
          if constexpr (KV && MK != kBwdMaskNone) {
            if (flags & kFlagBare) {
              ok = bwd_scrub<D>(p, bars, sStat + (j & 1) * kStatTile, tS, tDP, sR0 + j % C::RING0 * C::TILE,
                                sR1 + j % C::RING1 * C::TILE, j & 1);
              if (!ok) break;
              bwd_load_elements<KV>(tS, r);
            }
          }
#pragma unroll
          for (int c = 0; c < kBwdCols; ++c) pr[c] = __uint_as_float(r[c]);
        }
#pragma unroll
        for (int cb = 0; cb < kBwdCols; cb += 16) {
          float m[16];
          if constexpr (MK == kBwdMaskAdd) {
            if (cb % C::MASK_COLS == 0) {
              asm volatile("cp.async.wait_all;" ::: "memory");
              __syncwarp();
              if (KV ? flags & kFlagRefs : refs)
                Stage::refer(sMask,
                             KV ? p.ref + query_tile(b, h * p.group + now.g, now.tile) * 128 + wg * kBwdCols + cb : &nref,
                             (int)lane);
            }
            Stage::read(sMask, cb % C::MASK_COLS, (int)lane, m);
            if ((cb + 16) % C::MASK_COLS == 0) {  // the buffer has been read
              __syncwarp();
              if (cb + 16 < kBwdCols)
                stage(now, cb + 16);
              else if (it + 1 < n)
                fetch(at);
            }
          } else if constexpr (MK == kBwdMaskKey && !KV) {
            const float* mrow = static_cast<const float*>(p.mask) + (size_t)b * p.Nk;
#pragma unroll
            for (int c = 0; c < 16; ++c) m[c] = (__ldg(mrow + min(col0 + cb + c, p.Nk - 1)) + nref) * kLog2e;
          }
#pragma unroll
          for (int c = cb; c < cb + 16; c += 2) {
            float2 a = make_float2(nlse, nlse);
            if constexpr (KV) {
              a = *reinterpret_cast<const float2*>(lcol + c / 8 * 8);
              if constexpr (MK == kBwdMaskKey) a = __fadd2_rn(a, make_float2(key_add[c / 2 % 4], key_add[c / 2 % 4]));
            }
            if constexpr (MK == kBwdMaskAdd)
              a = __ffma2_rn(make_float2(m[c - cb], m[c - cb + 1]), make_float2(kLog2e, kLog2e), a);
            else if constexpr (MK == kBwdMaskKey && !KV)
              a = __fadd2_rn(a, make_float2(m[c - cb], m[c - cb + 1]));
            const float2 x = __ffma2_rn(make_float2(pr[c], pr[c + 1]), make_float2(sl2, sl2), a);
            const float2 e = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
            pr[c] = e.x;
            pr[c + 1] = e.y;
          }
        }
        if constexpr (MK == kBwdMaskKey && KV) {
          // Queries with a reference: their columns again, S is still there.
          if (flags & kFlagRefs) {
            const float* ref = p.ref + query_tile(b, h * p.group + now.g, now.tile) * 128 + wg * kBwdCols + col2;
            const float* mrow = static_cast<const float*>(p.mask) + (size_t)b * p.Nk;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t t[8];
              bwd_load_elements(tS + 8 * i, t);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int c = 8 * i + e % 2;
                const float nr = __ldcg(ref + c);
                if (nr == 0.f) continue;
                const float m = (__ldg(mrow + min(my4 + 8 * (e / 2), p.Nk - 1)) + nr) * kLog2e;
                pr[8 * i + e] = ptx::ex2(fmaf(__uint_as_float(t[e]), sl2, m + lcol[c]));
              }
            }
          }
        }
        if (edge) {
          if constexpr (KV) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
              const uint32_t w = seen[r] >> col2;
#pragma unroll
              for (int c = 0; c < 8; ++c)
                if (!((w >> (c / 2 * 8 + c % 2)) & 1u)) pr[c / 2 * 8 + 2 * r + c % 2] = 0.f;
            }
          } else {
#pragma unroll
            for (int c = 0; c < kBwdCols; ++c)
              if (!((seen[0] >> c) & 1u)) pr[c] = 0.f;
          }
        }
        if constexpr (KV) {  // over the columns just read
          uint32_t packed[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) packed[c] = ptx::pack_bf16x2(pr[2 * c], pr[2 * c + 1]);
          bwd_store_pairs(tS, packed);
          ptx::tmem_wait_st();
          ptx::tc_fence_before_sync();
          arrive(bars->p_ready[sb]);
        }
        ok = bwd_wait_warp(bars->dp_full, j & 1, bars, p);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        constexpr bool DP_FREE = !KV || T::NS == 2;  // dS goes over S's columns, not dP's
        auto dp_read = [&]() {
          if constexpr (DP_FREE) {
            ptx::tc_fence_before_sync();
            arrive(bars->dp_free);
          }
        };
        if constexpr (KV) {
          uint32_t r[32], packed[16];
          bwd_load_elements<true>(tDP, r);
          dp_read();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 d = *reinterpret_cast<const float2*>(dcol + 8 * i);
#pragma unroll
            for (int k = 8 * i; k < 8 * i + 8; k += 2) {
              const float2 x = __fadd2_rn(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])),
                                          d);
              const float2 s = __fmul2_rn(x, make_float2(pr[k], pr[k + 1]));
              packed[k / 2] = ptx::pack_bf16x2(s.x, s.y);
            }
          }
          bwd_store_pairs(DP_FREE ? tS + 16 : tDP, packed);
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t r[16], packed[8];
            ptx::tmem_ld32x32b_x16(tDP + half * 16, r);
            if (half == 1) dp_read();
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const int k = half * 16 + c;
              const float2 x = __fadd2_rn(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])),
                                          make_float2(ndelta, ndelta));
              const float2 s = __fmul2_rn(x, make_float2(pr[k], pr[k + 1]));
              packed[c / 2] = ptx::pack_bf16x2(s.x, s.y);
            }
            ptx::tmem_st32x32b_x8(tS + half * 8, packed);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        arrive(bars->ds_ready[sb]);
        if constexpr (KV) arrive(bars->st_empty[j & 1]);
      }
      if (!ok) break;

      // The unit's gradients, a quarter of the accumulators' columns each.
      constexpr int NC = T::ACC / kBwdGroups;
      const uint32_t tA = t0 + wg * NC;
      const bool is_dv = KV && wg < kBwdGroups / 2, zero = n == 0;
      // (the products of a query that sees nothing may be no numbers)
      const bool keep = KV || MK == kBwdMaskNone || nlse != -INFINITY;
      const BwdTensor& o = KV ? (is_dv ? p.dv : p.dk) : p.dq;
      const int col = KV ? (wg % (kBwdGroups / 2)) * NC : wg * NC;
      __nv_bfloat16* dst = o.p + b * o.b + h * o.h + (long long)my * o.n + col;
      have = next_work(work);
      if (!zero) {
        ok = bwd_wait_warp(bars->acc_full, nu & 1, bars, p) && ok;
        if (!ok) break;
        ++nu;
        ptx::tc_fence_after_sync();
      }
      if (pc.slot < 0) {
        const bool in = bwd_check(p, bars, pc.head < plan.units.heads && col + NC <= D, kCheckGradStore, pc.head, my);
        bwd_store_row<NC>(tA, is_dv ? 1.f : p.scale, zero, keep, in, (KV ? p.Nk : p.Nq) - my, (int)lane, dst, o.n);
      } else {
        const bool in = bwd_check(p, bars, pc.slot < 2 * plan.ctas, kCheckGradSlot, pc.slot, pc.head);
        float* part = p.part[KV ? 0 : 1] + (size_t)pc.slot * (128 * T::ACC) + wg * NC * 128;
        bwd_store_part<NC>(tA, zero, keep, in, part, row);
      }
      ptx::tc_fence_before_sync();
    }
    // (after an abort a mask's copies may be on their way to this CTA's shared memory)
    if constexpr (MK == kBwdMaskAdd) asm volatile("cp.async.wait_all;" ::: "memory");
    ptx::tc_fence_before_sync();
  }
  finish();
}

template <int D, int MK>
__global__ void __launch_bounds__(kBwdThreads, 1) fa_bwd_kernel(const __grid_constant__ BwdParams p) {
  using C = BwdCfg<D, MK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  BwdBars* bars = reinterpret_cast<BwdBars*>(smem + (2 + C::RING0 + C::RING1) * C::TILE + C::STAT_BYTES + C::MASK_BYTES);
  if (ptx::smem_u32(smem) & 1023u) {  // (the swizzled layouts need it; dynamic shared memory starts there)
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    auto init = [](uint64_t& b, uint32_t n) { ptx::mbar_init(ptx::smem_u32(&b), n); };
    init(bars->a_full, 1);
    init(bars->a_empty, 1);
    init(bars->b_full, 1);
    init(bars->b_empty, 1);
    for (int i = 0; i < C::RING0; ++i) init(bars->r0_full[i], 1), init(bars->r0_empty[i], 1);
    for (int i = 0; i < C::RING1; ++i) init(bars->r1_full[i], 1), init(bars->r1_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      init(bars->st_full[i], 1);
      init(bars->st_empty[i], kBwdWarps);
      init(bars->s_full[i], 1);
      init(bars->p_ready[i], kBwdWarps);
      init(bars->ds_ready[i], kBwdWarps);
    }
    init(bars->dp_full, 1);
    init(bars->dp_free, kBwdWarps);
    init(bars->acc_full, 1);
    init(bars->drain, 1);
    bars->abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (threadIdx.x / 32 == kBwdWarps + 1) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // -L, -delta and a mask's bits are there
  const int cta = blockIdx.x, keys = p.plan[0].ctas;
  if (cta < keys)
    bwd_units<D, MK, true>(p, cta, smem, bars, tmem);
  else
    bwd_units<D, MK, false>(p, cta - keys, smem, bars, tmem);
}

// The statistics of every query row, and of the rows that fill up the last tile:
// L_i = log2(e) LSE_i (+inf for a row that sees nothing, so that its P is 0),
// delta_i = dO_i . O_i - dLSE_i.  HBM bound (O and dO are read once: 4608 tokens of
// 24 heads of 128 11 us, 5.1 TB/s cold; 14 with one row a thread); D / 8 neighbouring lanes share a row.
struct BwdPrepParams {
  BwdTensor out, dout, q, k, v;
  const float *lse, *dlse;  // [B][Hq][Nq]; dlse may be nullptr
  float *stat, *ref;        // as BwdParams
  uint8_t* flags;
  int Hq, Nq, nqp;
  const float* mask;        // of references: key padding ([B][Nk], mask_rows 0) or additive
  int mask_heads, mask_rows, causal, group;
  float scale_log2;
  FastDiv div_h;
  int head_blocks;     // blocks of a head's rows
  FastDiv div_blocks;
  // Tiles with a kept pair, as bits (BwdParams), by the blocks behind the rows':
  // of a boolean mask from `some`, or of a key-padding mask.
  long long row_blocks;
  const uint32_t* some;    // [heads][query tiles][key tiles]
  const float* key_mask;   // [heads][Nk]
  uint32_t *tiles_q, *tiles_k;
  int heads, tiles_of_q, tiles_of_k, Nk, tile_words_q, tile_words_k;
};

// A warp makes one word.
static __device__ __forceinline__ void bwd_tile_bits(const BwdPrepParams& p, long long i) {
  const int lane = threadIdx.x % 32;
  if (p.key_mask) {
    if (i >= (long long)p.heads * p.tile_words_q) return;
    const int b = (int)(i / p.tile_words_q), w = (int)(i - (long long)b * p.tile_words_q);
    uint32_t word = 0;
    for (int t = 0; t < 32 && w * 32 + t < p.tiles_of_k; ++t) {
      bool some = false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int k = (w * 32 + t) * 128 + c * 32 + lane;
        some = some || (k < p.Nk && p.key_mask[(size_t)b * p.Nk + k] != -INFINITY);
      }
      if (__any_sync(0xffffffffu, some)) word |= 1u << t;
    }
    if (lane == 0) p.tiles_q[i] = word;
    return;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // `some` is there
  const long long by_q = (long long)p.heads * p.tiles_of_q * p.tile_words_q;
  const long long by_k = (long long)p.heads * p.tiles_of_k * p.tile_words_k;
  if (i >= by_q + by_k) return;
  const bool q = i < by_q;
  const long long at = q ? i : i - by_q;
  const int words = q ? p.tile_words_q : p.tile_words_k, tiles = q ? p.tiles_of_q : p.tiles_of_k;
  const long long row = at / words;
  const int head = (int)(row / tiles), tile = (int)(row - (long long)head * tiles);
  const int other = (int)(at - row * words) * 32 + lane, tq = q ? tile : other, tk = q ? other : tile;
  const bool some = tq < p.tiles_of_q && tk < p.tiles_of_k &&
                    p.some[((size_t)head * p.tiles_of_q + tq) * p.tiles_of_k + tk] != 0;
  const uint32_t word = __ballot_sync(0xffffffffu, some);
  if (lane == 0) (q ? p.tiles_q : p.tiles_k)[at] = word;
}

// Rows of a block (they divide a tile's 128).
template <int D>
constexpr int kBwdPrepRows = D == 128 ? 64 : 128;

// A row's sums so far: of 2^(x + (mask - ref) log2(e) - most) over its keys, and of that
// times dP; `ref` the largest mask and `most` the largest exponent that it has met.
struct BwdRowSum {
  float ref = -INFINITY, most = -INFINITY, sum = 0.f, along = 0.f;
  // Takes the sum to another, larger reference.
  __device__ __forceinline__ void refer(float to) {
    if (to > ref) {
      most += (ref - to) * 1.4426950408889634f;
      ref = to;
    }
  }
  __device__ __forceinline__ void raise(float to) {
    if (to > most) {
      const float by = ptx::ex2(most - to);
      sum *= by;
      along *= by;
      most = to;
    }
  }
  __device__ __forceinline__ void join(BwdRowSum o) {
    refer(o.ref);
    o.refer(ref);
    raise(o.most);
    if (o.most == -INFINITY) return;
    const float by = ptx::ex2(o.most - most);
    sum += o.sum * by;
    along += o.along * by;
  }
};

// The references of a warp's 16 rows whose LSE is too large to give P, and L and delta
// anew: log2 of the sum of 2^(scale s + mask - ref), and the sum of P dP less dLSE (such a
// row's O is of scores that the forward has rounded with the mask).  Rows whose scores
// make LSE large, not their mask, stay as they are: LSE and O come from those scores.
// Row i of the 16 is n0 + i / RUN * STEP + i % RUN (`weak`: bit i).  Such rows are padding
// and few, so the products are a warp's (mma.sync, 16 x 8 x 16) and their operands come
// from global memory, 16 bytes a lane: of every 32 elements lane l has those from
// 8 (l % 4) on, in rows and keys alike, which is an order of the sum over the head
// dimension.  Out of line: warps without such rows take no registers.
template <int D, int RUN, int STEP>
__device__ __noinline__ void bwd_resum(const BwdPrepParams& p, int bh, int n0, uint32_t weak) {
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr int KEYS = 2;  // eights of keys whose products are under way together
  const int lane = threadIdx.x % 32;
  const int b = (int)p.div_h.div((uint32_t)bh), h = bh - b * p.Hq;
  const __nv_bfloat16* q = p.q.p + b * p.q.b + h * p.q.h + 8 * (lane % 4);
  const __nv_bfloat16* k = p.k.p + b * p.k.b + (long long)(h / p.group) * p.k.h + 8 * (lane % 4);
  const __nv_bfloat16* v = p.v.p + b * p.v.b + (long long)(h / p.group) * p.v.h + 8 * (lane % 4);
  const float* mask = p.mask + (p.mask_rows ? ((size_t)b * p.mask_heads + (p.mask_heads == 1 ? 0 : h)) * p.Nq * p.Nk
                                            : (size_t)b * p.Nk);
  const int Nk = p.Nk;
  const float scale = p.scale_log2;
  // This lane's rows of a product, lane / 4 and lane / 4 + 8, and how many keys they see (by the triangle).
  int n[2], end[2];
  const float* m[2];
  const __nv_bfloat16 *row[2], *grad[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = lane / 4 + 8 * e;
    n[e] = n0 + i / RUN * STEP + i % RUN;
    end[e] = !(weak >> i & 1) ? 0 : p.causal ? min(Nk, n[e] + 1) : Nk;
    const int at = min(n[e], p.Nq - 1);
    m[e] = mask + (p.mask_rows ? (size_t)at * Nk : 0) + 2 * (lane % 4);
    row[e] = q + at * p.q.n;
    grad[e] = p.dout.p + b * p.dout.b + h * p.dout.h + 8 * (lane % 4) + at * p.dout.n;
  }
  // Products of the lane's rows of `a` and of keys j0 .. j0 + 8 KEYS - 1 of `x`.
  auto product = [&](float (&c)[KEYS][4], const __nv_bfloat16* const (&a)[2], const __nv_bfloat16* x, long long x_n,
                     int j0) {
#pragma unroll 1
    for (int d = 0; d < D; d += 32) {
      uint4 ra[2], rx[KEYS];
#pragma unroll
      for (int e = 0; e < 2; ++e) ra[e] = *reinterpret_cast<const uint4*>(a[e] + d);
#pragma unroll
      for (int i = 0; i < KEYS; ++i)
        rx[i] = *reinterpret_cast<const uint4*>(x + min(j0 + 8 * i + lane / 4, Nk - 1) * x_n + d);
      auto mma = [](float (&y)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(y[0]), "+f"(y[1]), "+f"(y[2]), "+f"(y[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
      };
#pragma unroll
      for (int i = 0; i < KEYS; ++i) {
        mma(c[i], ra[0].x, ra[1].x, ra[0].y, ra[1].y, rx[i].x, rx[i].y);
        mma(c[i], ra[0].z, ra[1].z, ra[0].w, ra[1].w, rx[i].z, rx[i].w);
      }
    }
  };
  const int most = __reduce_max_sync(0xffffffffu, max(end[0], end[1]));
  BwdRowSum of[2];
  for (int j0 = 0; j0 < most; j0 += 8 * KEYS) {
    float c[KEYS][4] = {}, dp[KEYS][4] = {};
    product(c, row, k, p.k.n, j0);
    product(dp, grad, v, p.v.n, j0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // the lane's rows; columns 2 (lane % 4), + 1 of each eight
      float add[2 * KEYS], ref = of[e].ref;
#pragma unroll
      for (int i = 0; i < 2 * KEYS; ++i) {  // (all loads at once, the last key's again behind it)
        const int j = j0 + 8 * (i / 2) + i % 2, at = min(j, Nk - 1 - 2 * (lane % 4));
        add[i] = m[e][at];
        if (j + 2 * (lane % 4) >= end[e]) add[i] = -INFINITY;
        ref = fmaxf(ref, add[i]);
      }
      if (ref == -INFINITY) continue;
      of[e].refer(ref);
      float top = of[e].most;
#pragma unroll
      for (int i = 0; i < 2 * KEYS; ++i) {
        float& x = c[i / 2][2 * e + i % 2];
        x = fmaf(x, scale, (add[i] - ref) * kLog2e);
        top = fmaxf(top, x);
      }
      of[e].raise(top);
#pragma unroll
      for (int i = 0; i < 2 * KEYS; ++i) {
        const float w = ptx::ex2(c[i / 2][2 * e + i % 2] - of[e].most);
        of[e].sum += w;
        if (w > 0.f) of[e].along = fmaf(w, dp[i / 2][2 * e + i % 2], of[e].along);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      BwdRowSum o;
      o.ref = __shfl_xor_sync(0xffffffffu, of[e].ref, x);
      o.most = __shfl_xor_sync(0xffffffffu, of[e].most, x);
      o.sum = __shfl_xor_sync(0xffffffffu, of[e].sum, x);
      o.along = __shfl_xor_sync(0xffffffffu, of[e].along, x);
      of[e].join(o);
    }
    if (lane % 4 == 0 && (weak >> (lane / 4 + 8 * e) & 1) && fabsf(of[e].ref) >= kWeakLse / 4) {
      float* stat = p.stat + ((size_t)bh * (p.nqp / 128) + n[e] / 128) * kStatTile + n[e] % 128;
      const bool sees = of[e].sum > 0.f;
      stat[0] = sees ? -(of[e].most + log2f(of[e].sum)) : -INFINITY;
      stat[kStatDelta] = sees ? (p.dlse ? p.dlse[(size_t)bh * p.Nq + n[e]] : 0.f) - of[e].along / of[e].sum : 0.f;
      p.ref[(size_t)bh * p.nqp + n[e]] = sees ? -of[e].ref : 0.f;
    }
  }
}

// Whether a number is not finite or past 2^60, under which products of 128 such numbers
// are finite (their own and with keys like them).
__device__ __forceinline__ bool bwd_large(const uint4& v) {
  bool large = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    large = large || (w & 0x7fffu) >= 0x5d80u || (w >> 16 & 0x7fffu) >= 0x5d80u;
  }
  return large;
}

// MASKED: rows may see nothing; REFS (an additive or key-padding mask): they may need
// references.
template <int D, bool MASKED, bool REFS>
__global__ void __launch_bounds__(256, 4) fa_bwd_prep_kernel(const __grid_constant__ BwdPrepParams p) {
  constexpr int L = D / 8;  // lanes a row
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x >= p.row_blocks) {
    bwd_tile_bits(p, (blockIdx.x - p.row_blocks) * 8 + threadIdx.x / 32);
    return;
  }
  // A block's rows are of one head.  All of a thread's loads go out together.
  constexpr int STEP = 256 / L, U = kBwdPrepRows<D> / STEP;
  const int bh = (int)p.div_blocks.div(blockIdx.x);
  const int b = (int)p.div_h.div((uint32_t)bh), h = bh - b * p.Hq, piece = threadIdx.x % L;
  const __nv_bfloat16 *out = p.out.p + b * p.out.b + h * p.out.h + piece * 8,
                      *dout = p.dout.p + b * p.dout.b + h * p.dout.h + piece * 8;
  uint4 o[U] = {}, g[U] = {};
  float lse[U], sum[U];
  const int block_row = (int)(blockIdx.x - (unsigned)bh * p.head_blocks) * kBwdPrepRows<D>;
  const size_t tile = (size_t)bh * (p.nqp / 128) + block_row / 128;
  float* stat = p.stat + tile * kStatTile + block_row % 128 + threadIdx.x / L;
  const int n0 = block_row + threadIdx.x / L;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = n0 + u * STEP;
    sum[u] = 0.f;
    lse[u] = -INFINITY;
    if (n < p.Nq) {
      o[u] = *reinterpret_cast<const uint4*>(out + n * p.out.n);
      g[u] = *reinterpret_cast<const uint4*>(dout + n * p.dout.n);
      if (MASKED || piece == 0) lse[u] = p.lse[(size_t)bh * p.Nq + n];
      if (piece == 0 && p.dlse) sum[u] = -p.dlse[(size_t)bh * p.Nq + n];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t ow[4] = {o[u].x, o[u].y, o[u].z, o[u].w}, gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // a bf16 is the upper half of its fp32
      dot = fmaf(__uint_as_float(ow[k] << 16), __uint_as_float(gw[k] << 16), dot);
      dot = fmaf(__uint_as_float(ow[k] & 0xffff0000u), __uint_as_float(gw[k] & 0xffff0000u), dot);
    }
#pragma unroll
    for (int m = 1; m < L; m <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
    if (piece == 0) {
      float* at = stat + u * STEP;
      const bool sees = lse[u] != -INFINITY;  // (dLSE of a row that sees nothing may be anything)
      at[0] = sees ? -lse[u] * 1.4426950408889634f : -INFINITY;
      at[kStatDelta] = sees ? -(dot + sum[u]) : 0.f;
      if constexpr (REFS) p.ref[tile * 128 + block_row % 128 + threadIdx.x / L + u * STEP] = 0.f;
    }
  }
  if constexpr (MASKED) {  // the flags of the warp's rows
    bool bare = false;
    uint32_t weak = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + u * STEP;
      if (n < p.Nq && lse[u] == -INFINITY)
        bare = bare || bwd_large(g[u]) ||
               bwd_large(*reinterpret_cast<const uint4*>(p.q.p + b * p.q.b + h * p.q.h + n * p.q.n + piece * 8));
      if constexpr (REFS) weak |= bwd_weak(lse[u]) ? 1u << u : 0u;
    }
    uint32_t flags = __any_sync(0xffffffffu, bare) ? kFlagBare & 0xff : 0;
    if constexpr (REFS) {
      if (__any_sync(0xffffffffu, weak)) {
        flags |= kFlagRefs & 0xff;
        constexpr int RUN = 32 / L;  // rows of a warp at a time
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < U * RUN; ++i)
          bits |= (__shfl_sync(0xffffffffu, weak, i % RUN * L) >> (i / RUN) & 1u) << i;
        __syncwarp();  // (-L and -delta of these rows are written again)
        bwd_resum<D, RUN, STEP>(p, bh, n0 - threadIdx.x % 32 / L, bits);
      }
    }
    if (threadIdx.x % 32 == 0) {  // (tiles of one block: 2 bytes a warp)
      const int warp = block_row % 128 / 8 + threadIdx.x / 32;
      if (kBwdPrepRows<D> == 128)
        reinterpret_cast<uint16_t*>(p.flags + tile * kFlagTile * 4)[warp] = flags;
      else
        p.flags[tile * kFlagTile * 4 + warp] = flags;
    }
  }
}

// A boolean mask as bits, by query rows and by key rows: a block turns a tile, a warp
// 16 rows of 128 bytes, a lane 4 of each.  Rows start at any byte: a lane reads the
// aligned words that its bytes lie in (words with no byte of the row are not read) and
// shifts them together.  What bounds it is stores, each to a row of its own, so a row's
// four words are put together first (2 x 1777 x 1777 pairs cold: 7 us; 11 with single
// words, 13 with single bytes by key rows).
struct BwdBitsParams {
  const uint8_t* mask;  // [B mask_heads][Nq][Nk]
  uint32_t *bits_q, *bits_k;
  uint32_t* some;                // [B mask_heads][query tiles][key tiles]: the tile keeps a pair
  int Nq, Nk, tiles_q, tiles_k;
};

static __global__ void __launch_bounds__(256) fa_bwd_bits_kernel(const __grid_constant__ BwdBitsParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ __align__(16) uint32_t by_row[128][4];
  __shared__ __align__(16) uint16_t by_key[8][128];  // by warp
  const int per = p.tiles_q * p.tiles_k;
  const long long bh = blockIdx.x / per;
  const int tile = (int)(blockIdx.x - bh * per), tq = tile / p.tiles_k, tk = tile - tq * p.tiles_k;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int k = tk * 128 + lane * 4;  // this lane's first key
  const int q0 = tq * 128 + warp * 16, rows = p.Nq - q0, valid = min(max(p.Nk - k, 0), 4);
  const uint32_t keep = valid == 4 ? ~0u : (1u << (8 * valid)) - 1;
  const uint8_t* at = p.mask + (bh * p.Nq + q0) * p.Nk + k;
  uint32_t lo[16], hi[16];
#pragma unroll
  for (int y = 0; y < 16; ++y) {
    const uint8_t* q = at + (long long)y * p.Nk;
    const int off = (int)(reinterpret_cast<uintptr_t>(q) & 3);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(q - off);
    const bool live = y < rows && valid > 0;
    lo[y] = live ? __ldg(w) : 0;
    hi[y] = live && off + valid > 4 ? __ldg(w + 1) : 0;
  }
  uint32_t col[4] = {}, word[2] = {}, any = 0;
#pragma unroll
  for (int y = 0; y < 16; ++y) {
    const int off = (int)(reinterpret_cast<uintptr_t>(at + (long long)y * p.Nk) & 3);
    uint32_t t = __funnelshift_r(lo[y], hi[y], 8 * off) & keep;
    t |= t >> 4;  // bit 0 of each byte: any of its bits (what shifts in from the next byte stays above bit 0)
    t |= t >> 2;
    t |= t >> 1;
    t &= 0x01010101u;
    any |= t;
#pragma unroll
    for (int c = 0; c < 4; ++c) col[c] |= ((t >> (8 * c)) & 1u) << y;
    uint32_t r = (t * 0x01020408u) >> 24 << (4 * (lane % 8));  // the four bits together
    r |= __shfl_xor_sync(0xffffffffu, r, 1);
    r |= __shfl_xor_sync(0xffffffffu, r, 2);
    r |= __shfl_xor_sync(0xffffffffu, r, 4);
    if (lane % 8 == y % 8) word[y / 8] = r;
  }
  by_row[warp * 16 + lane % 8][lane / 8] = word[0];
  by_row[warp * 16 + 8 + lane % 8][lane / 8] = word[1];
  *reinterpret_cast<uint2*>(&by_key[warp][lane * 4]) = make_uint2(col[0] | col[1] << 16, col[2] | col[3] << 16);
  any = __syncthreads_or(any != 0);
  if (threadIdx.x == 0) p.some[blockIdx.x] = any;
  const int i = threadIdx.x % 128;
  if (threadIdx.x < 128) {
    const int q = tq * 128 + i;
    if (q < p.Nq)
      reinterpret_cast<uint4*>(p.bits_q)[((size_t)bh * p.Nq + q) * p.tiles_k + tk] =
          *reinterpret_cast<const uint4*>(by_row[i]);
  } else if (tk * 128 + i < p.Nk) {
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = by_key[2 * c][i] | (uint32_t)by_key[2 * c + 1][i] << 16;
    reinterpret_cast<uint4*>(p.bits_k)[((size_t)bh * p.Nk + tk * 128 + i) * p.tiles_q + tq] =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Joins the partial sums of cut units, in the order of their pieces.  Block
// (c, y): the unit that starts in CTA c's range (key units' CTAs, then query
// units'), 8 columns of its accumulators.  Latency bound (7 to 11 us cold); its
// blocks start beside the last of the kernel before it.
template <int D>
__global__ void __launch_bounds__(128) fa_bwd_join_kernel(const __grid_constant__ BwdParams p) {
  const bool kv = blockIdx.x < (unsigned)p.plan[0].ctas;
  const int cta = kv ? (int)blockIdx.x : (int)blockIdx.x - p.plan[0].ctas;
  const int col = blockIdx.y * 8, row = threadIdx.x, acc_cols = kv ? 2 * D : D;
  if (col >= acc_cols) return;
  const BwdPlan& plan = p.plan[kv ? 0 : 1];
  int unit, last, slot;
  if (!bwd_join(plan, cta, unit, last, slot)) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
  const float* part = p.part[kv ? 0 : 1];
  float acc[8] = {};
  for (int c = cta; c <= last; ++c) {
    if (c > cta) {
      slot = 2 * c;
      if (plan.cut[c].unit == plan.cut[c + 1].unit && plan.cut[c].it == plan.cut[c + 1].it) continue;
    }
    const float4* src = reinterpret_cast<const float4*>(part + (size_t)slot * (128 * acc_cols)) +
                        (size_t)(col / 4) * 128 + row;
    const float4 a = src[0], e = src[128];
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += e.x; acc[5] += e.y; acc[6] += e.z; acc[7] += e.w;
  }
  int head, tile;
  plan.units.locate(unit, head, tile);
  const int heads = kv ? p.Hk : p.Hq;
  const int b = (int)(kv ? p.div_hk : p.div_hq).div((uint32_t)head), h = head - b * heads;
  const int my = tile * 128 + row;
  if (my >= (kv ? p.Nk : p.Nq)) return;
  const bool is_dv = kv && col < D;
  const BwdTensor& o = kv ? (is_dv ? p.dv : p.dk) : p.dq;
  const float mul = is_dv ? 1.f : p.scale;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = ptx::pack_bf16x2(acc[2 * i] * mul, acc[2 * i + 1] * mul);
  *reinterpret_cast<uint4*>(o.p + b * o.b + h * o.h + (long long)my * o.n + (col < D ? col : col - D)) =
      make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace fa
