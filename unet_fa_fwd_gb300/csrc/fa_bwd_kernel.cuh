// fa_bwd_kernel.cuh — the sm_103a attention gradient.
//
// With t_ij = log2(e) (scale q_i . k_j + mask_ij), L_i = log2(e) LSE_i from the
// forward and delta_i = dO_i . O_i - dLSE_i:
//   P_ij = 2^(t_ij - L_i),  dP_ij = dO_i . V_j,  dS_ij = P_ij (dP_ij - delta_i),
//   dV_j = sum_i P_ij dO_i,  dK_j = scale sum_i dS_ij Q_i,  dQ_i = scale sum_j dS_ij K_j.
// P is recomputed from L (no running maximum), so a tile's work is two products
// into tensor memory, one pass of the threads, and the products of its results.
//
// Two kernels, each over units of 128 rows: keys (dK, dV; products S^T, dP^T, dV, dK)
// and queries (dQ; S, dP, dQ).  Seven products for the five that one kernel
// would need: such a kernel has to add dQ up in device memory across the key
// units, whose order changes the result from run to run, and moves 64 KB of it a
// tile through shared memory or L2 atomics, where it would wait about as long as
// the two products take (an SM reads 128 bytes a clock of operands: 64 KB for a
// 128 x 128 x 128 product of shared memory's operands takes as long as the
// product).  Here every sum stays in tensor memory and results repeat bit for bit.
//
// A CTA (one per SM) of 384 threads:
//   warps 0-3, 4-7  two warpgroups; a thread has a row of the unit (one lane of
//                   tensor memory) and half of a tile's 128 columns
//   warp 8          TMA producer      warp 9  MMA issuer (owns tensor memory)
// P and dS go back to tensor memory as bf16, the A operand of the products that
// take them; both sides' rows are operands K-major for S and dP and MN-major for
// the gradients, from one copy in shared memory.
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

struct BwdParams {
  BwdPlan plan;
  int Hq, Hk, group, Nq, Nk, nqp;  // nqp: queries rounded up to whole tiles
  int causal;
  float scale, scale_log2;
  const float* nlse;    // [B Hq][nqp]: -L, -inf for rows that see nothing and rows past Nq
  const float* delta;   // [B Hq][nqp]
  const void* mask;     // fp32 [B][Nk], or fp32 / uint8 [B][mask_heads][Nq][Nk]
  int mask_heads, mask_vec;
  BwdTensor out0, out1;  // dV and dK, or dQ
  float* part;           // partial sums of cut units
  unsigned long long timeout_ns;
  int* status;
  int* debug_record;
  int inject_stall;
  FastDiv div_h, div_group;  // by the unit side's heads, by group
  // the unit's rows (0, 1) and the tiles it walks (2, 3): K, V, Q, dO or Q, dO, K, V
  CUtensorMap map[4];
};

template <int D, bool KV>
struct BwdCfg {
  using F = Cfg<D>;
  static constexpr int TILE = 128 * D * 2;  // bytes of a 128-row tile
  // Rings of the walked tiles.  dK dV: Q (read again by dK, two iterations
  // long) and dO; dQ: K and V.  At D = 128 the five slots that fit.
  static constexpr int RING0 = D == 128 ? 3 : 4;
  static constexpr int RING1 = D == 128 ? 2 : 4;
  static constexpr int STATS = 2;               // dK dV: slots of -L and delta of 128 queries
  static constexpr int STAT_BYTES = KV ? 1024 : 0;
  static constexpr int SMEM_BAR = 512;
  static constexpr int SMEM_USED = (2 + RING0 + RING1) * TILE + STATS * STAT_BYTES + SMEM_BAR;
  // (more than half of the SM's, so that one CTA has its tensor memory alone)
  static constexpr int SMEM_BYTES = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
  // Tensor memory: accumulators, S (two where they fit), dP.
  static constexpr int ACC = KV ? 2 * D : D;
  static constexpr int NS = ACC + 3 * 128 <= 512 ? 2 : 1;
  static constexpr int COL_S = ACC, COL_DP = ACC + NS * 128;
  static_assert(COL_DP + 128 <= 512, "tensor-memory columns");
  static constexpr int THREADS = 384;
  static constexpr int REGS_ROWS = 208, REGS_OTHER = 88;
  static_assert(2 * 128 * REGS_ROWS + 128 * REGS_OTHER <= THREADS * 168, "register split");
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

// acc += X T: X bf16 in tensor memory (64 columns' worth at x, the other half
// at x + 64), T a 128-row tile, MN-major.
template <int D>
__device__ __forceinline__ void bwd_mma_grad(uint32_t acc, uint32_t x, uint32_t t_lo, uint32_t t_hi, bool first) {
  constexpr uint32_t IDESC = make_idesc(128, D, true);
  constexpr uint32_t STEP = (16 * Cfg<D>::SW) >> 4;
  ptx::mma_ts_x4_el<STEP>(acc, x, t_lo, t_hi, IDESC, first ? 0u : 1u);
  ptx::mma_ts_x4_el<STEP>(acc, x + 64, t_lo + 4 * STEP, t_hi, IDESC, 1u);
}

template <int D>
__device__ __forceinline__ void bwd_load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row, int h,
                                              int b) {
  using C = Cfg<D>;
#pragma unroll
  for (int c = 0; c < C::NCHUNK; ++c)
    ptx::tma_load_4d(dst + c * C::CHUNK_BYTES, map, bar, c * C::CHUNK_ELEMS, row, h, b);
}

// Mask values of 32 columns of a thread's row, as what is added to t (log2
// domain; -inf: excluded).  at(c): the address of column c's value.
template <int MK, typename At>
__device__ __forceinline__ void bwd_mask32(float (&m)[32], At at) {
  constexpr float kLog2e = 1.4426950408889634f;
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    if constexpr (MK == kBwdMaskBool)
      m[c] = __ldg(static_cast<const uint8_t*>(static_cast<const void*>(at(c)))) ? 0.f : -INFINITY;
    else
      m[c] = __ldg(static_cast<const float*>(static_cast<const void*>(at(c)))) * kLog2e;
  }
}

// 2^(s sl2 + add) of a pair.
__device__ __forceinline__ float2 bwd_exp(float s0, float s1, float sl2, float2 add) {
  const float2 x = __ffma2_rn(make_float2(s0, s1), make_float2(sl2, sl2), add);
  return make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
}

// The columns [0, D) of a thread's accumulator row at `t`, NC of them, times
// `mul`, rounded to the row at `dst` (16-byte aligned), or as they are to a slot
// of partial sums (laid out [columns / 4][128 rows][4]).
template <int NC>
__device__ __forceinline__ void bwd_store_row(uint32_t t, float mul, bool zero, bool ok, __nv_bfloat16* dst) {
#pragma unroll
  for (int cb = 0; cb < NC; cb += 16) {
    uint32_t r[16];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = 0u;
    } else {
      ptx::tmem_ld32x32b_x16(t + cb, r);
    }
    if (ok) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = ptx::pack_bf16x2(__uint_as_float(r[8 * q + 2 * i]) * mul, __uint_as_float(r[8 * q + 2 * i + 1]) * mul);
        *reinterpret_cast<uint4*>(dst + cb + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}
template <int NC>
__device__ __forceinline__ void bwd_store_part(uint32_t t, bool ok, float* dst, int row) {
#pragma unroll
  for (int cb = 0; cb < NC; cb += 16) {
    uint32_t r[16];
    ptx::tmem_ld32x32b_x16(t + cb, r);
    if (ok) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(dst + ((size_t)(cb / 4 + q) * 128 + row) * 4) =
            make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
    }
  }
}

// Where a piece's iterations lie: query head (of a group that shares the key
// head) and tile of the other side.
struct BwdIter {
  int g, tile;  // head in the group, tile
  int first, n;
  __device__ __forceinline__ void start(const BwdUnits& u, int unit_tile, int it) {
    u.range(unit_tile, first, n);
    g = n > 0 && u.group > 1 ? it / n : 0;
    tile = first + it - g * n;
  }
  __device__ __forceinline__ void next() {
    if (++tile == first + n) {
      tile = first;
      ++g;
    }
  }
};

// KV: dK and dV of 128 keys; else dQ of 128 queries.
template <int D, int MK, bool KV>
__global__ void __launch_bounds__(BwdCfg<D, KV>::THREADS, 1) fa_bwd_kernel(const __grid_constant__ BwdParams p) {
  using C = BwdCfg<D, KV>;
  using F = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::TILE;
  uint8_t* sR0 = sB + C::TILE;
  uint8_t* sR1 = sR0 + C::RING0 * C::TILE;
  float* sStat = reinterpret_cast<float*>(sR1 + C::RING1 * C::TILE);
  BwdBars* bars = reinterpret_cast<BwdBars*>(sR1 + C::RING1 * C::TILE + C::STATS * C::STAT_BYTES);
  const int warp = threadIdx.x / 32;
  const uint32_t lane = threadIdx.x % 32;

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
      init(bars->st_empty[i], 8);
      init(bars->s_full[i], 1);
      init(bars->p_ready[i], 8);
      init(bars->ds_ready[i], 8);
    }
    init(bars->dp_full, 1);
    init(bars->dp_free, 8);
    init(bars->acc_full, 1);
    init(bars->drain, 1);
    bars->abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  auto finish = [&]() {
    ptx::named_barrier_sync(1, C::THREADS);
    if (warp == 9) {
      ptx::tc_fence_after_sync();
      ptx::tmem_dealloc(tmem, 512);
    }
  };
  auto piece_ok = [&](const BwdPiece& pc) {
    return bwd_check(p, bars, pc.head >= 0 && pc.head < p.plan.units.heads && pc.tile >= 0 &&
                                  pc.tile < p.plan.units.tiles && pc.it0 >= 0 &&
                                  pc.it1 <= p.plan.units.iterations(pc.tile) && pc.it0 <= pc.it1,
                     kCheckGradUnit, pc.head, pc.tile);
  };

  if (warp >= 8) {
    ptx::setmaxnreg_dec<C::REGS_OTHER>();
    if (warp == 8) {
      // ---------------------------------------------------------- producer --
      if (lane == 0) {
        for (int i = 0; i < 4; ++i) ptx::tma_prefetch_desc(&p.map[i]);
        uint32_t na = 0, nb = 0, j = 0;  // tiles of the unit's rows, iterations begun
        uint32_t n0 = 0, n1 = 0, nst = 0;  // copies issued to each ring
        bool ok = true;
        BwdWalk walk;
        BwdPiece pc;
        while (ok && walk.next(p.plan, blockIdx.x, pc)) {
          if (!piece_ok(pc)) break;
          if (pc.it0 == pc.it1) continue;
          const int b = (int)p.div_h.div((uint32_t)pc.head), h = pc.head - b * (KV ? p.Hk : p.Hq);
          // heads of the tiles walked: a group of query heads, or the key head
          const int h_other = KV ? h * p.group : (int)p.div_group.div((uint32_t)h);
          auto load_unit = [&](int i, uint8_t* dst, uint64_t& full, uint64_t& empty, uint32_t& n) {
            if (!bwd_wait(empty, (n & 1) ^ 1, bars, p)) return false;
            ptx::mbar_arrive_expect_tx(ptx::smem_u32(&full), C::TILE);
            bwd_load_tile<D>(ptx::smem_u32(dst), &p.map[i], ptx::smem_u32(&full), pc.tile * 128, h, b);
            ++n;
            return true;
          };
          BwdIter at;
          at.start(p.plan.units, pc.tile, pc.it0);
          for (int it = pc.it0; ok && it < pc.it1; ++it, ++j, at.next()) {
            const int ho = h_other + (KV ? at.g : 0);
            if (it == pc.it0) ok = load_unit(0, sA, bars->a_full, bars->a_empty, na);
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
            bwd_load_tile<D>(ptx::smem_u32(sR0 + s0 * C::TILE), &p.map[2], full, at.tile * 128, ho, b);
            ++n0;
            if (it == pc.it0) ok = load_unit(1, sB, bars->b_full, bars->b_empty, nb);
            if (!ok) break;
            if constexpr (KV) {
              const uint32_t ss = j & 1;
              ok = bwd_wait(bars->st_empty[ss], ((j / 2) & 1) ^ 1, bars, p);
              if (!ok) break;
              full = ptx::smem_u32(&bars->st_full[ss]);
              ptx::mbar_arrive_expect_tx(full, 1024);
              const size_t row = ((size_t)b * p.Hq + ho) * p.nqp + (size_t)at.tile * 128;
              bulk_load(ptx::smem_u32(sStat + ss * 256), p.nlse + row, 512, full);
              bulk_load(ptx::smem_u32(sStat + ss * 256 + 128), p.delta + row, 512, full);
              ++nst;
            }
            ok = bwd_wait(bars->r1_empty[s1], ((j / C::RING1) & 1) ^ 1, bars, p);
            if (!ok) break;
            full = ptx::smem_u32(&bars->r1_full[s1]);
            ptx::mbar_arrive_expect_tx(full, C::TILE);
            bwd_load_tile<D>(ptx::smem_u32(sR1 + s1 * C::TILE), &p.map[3], full, at.tile * 128, ho, b);
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
    } else if (warp == 9) {
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
        bwd_mma_scores<D>(tmem + C::COL_S + (i % C::NS) * 128, k_lo + a16, k_lo + r0 + s * TILE16, k_hi);
        commit(bars->s_full[i % C::NS]);
        return true;
      };
      auto dprob = [&](uint32_t i) -> bool {
        const uint32_t s = i % C::RING1;
        if (!bwd_wait_warp(bars->r1_full[s], (i / C::RING1) & 1, bars, p)) return false;
        ptx::tc_fence_after_sync();
        bwd_mma_scores<D>(tmem + C::COL_DP, k_lo + b16, k_lo + r1 + s * TILE16, k_hi);
        commit(bars->dp_full);
        if constexpr (!KV) commit(bars->r1_empty[s]);  // V is not needed again
        return true;
      };
      BwdWalk walk;
      BwdPiece pc;
      while (ok && walk.next(p.plan, blockIdx.x, pc)) {
        const uint32_t n = (uint32_t)(pc.it1 - pc.it0);
        if (n == 0) continue;
        ok = bwd_wait_warp(bars->a_full, nu & 1, bars, p) && scores(j);
        if (ok && n == 1) commit(bars->a_empty);
        ok = ok && bwd_wait_warp(bars->b_full, nu & 1, bars, p) && dprob(j);
        if (ok && n == 1) commit(bars->b_empty);
        if (ok && C::NS == 2 && n > 1) {
          ok = scores(j + 1);
          if (ok && n == 2) commit(bars->a_empty);
        }
        if (!ok) break;
        for (uint32_t i = 0; ok && i < n; ++i, ++j) {
          const uint32_t s0 = j % C::RING0, s1 = j % C::RING1, sb = j % C::NS;
          const uint32_t tS = tmem + C::COL_S + sb * 128;
          if constexpr (KV) {
            // dV += P^T dO
            ok = bwd_wait_warp(bars->p_ready[sb], (j / C::NS) & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_mma_grad<D>(tmem, tS, mn_lo + r1 + s1 * TILE16, mn_hi, i == 0);
            commit(bars->r1_empty[s1]);
            if (i + C::NS < n) {
              ok = scores(j + C::NS);
              if (!ok) break;
              if (i + C::NS + 1 == n) commit(bars->a_empty);
            }
            // dK += dS^T Q
            ok = bwd_wait_warp(bars->ds_ready[0], j & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_mma_grad<D>(tmem + D, tmem + C::COL_DP, mn_lo + r0 + s0 * TILE16, mn_hi, i == 0);
            commit(bars->r0_empty[s0]);
            if (i + 1 < n) {
              ok = dprob(j + 1);
              if (!ok) break;
              if (i + 2 == n) commit(bars->b_empty);
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
            ok = bwd_wait_warp(bars->ds_ready[sb], (j / C::NS) & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_mma_grad<D>(tmem, tS, mn_lo + r0 + s0 * TILE16, mn_hi, i == 0);
            commit(bars->r0_empty[s0]);
            if (i + C::NS < n) {
              ok = scores(j + C::NS);
              if (!ok) break;
              if (i + C::NS + 1 == n) commit(bars->a_empty);
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
    const int row = (warp % 4) * 32 + (int)lane;
    const uint32_t t0 = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    const float sl2 = p.scale_log2;
    constexpr float kLog2e = 1.4426950408889634f;
    auto arrive = [&](uint64_t& b) {  // one arrival per warp
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&b));
    };
    uint32_t j = 0, nu = 0;
    bool ok = true;
    BwdWalk walk;
    BwdPiece pc;
    while (ok && walk.next(p.plan, blockIdx.x, pc)) {
      ok = __all_sync(0xffffffffu, piece_ok(pc));
      if (!ok) break;
      const int b = (int)p.div_h.div((uint32_t)pc.head), h = pc.head - b * (KV ? p.Hk : p.Hq);
      const int my = pc.tile * 128 + row;  // this thread's key or query
      const int mine = min(my, (KV ? p.Nk : p.Nq) - 1);
      float nlse = 0.f, delta = 0.f, key_add = 0.f;
      if constexpr (!KV) {
        const size_t at = (size_t)pc.head * p.nqp + my;
        nlse = __ldg(p.nlse + at);
        delta = __ldg(p.delta + at);
      } else if constexpr (MK == kBwdMaskKey) {
        key_add = __ldg(static_cast<const float*>(p.mask) + (size_t)b * p.Nk + mine) * kLog2e;
      }
      BwdIter at;
      at.start(p.plan.units, pc.tile, pc.it0);
      for (int it = pc.it0; it < pc.it1; ++it, ++j, at.next()) {
        const uint32_t sb = j % C::NS;
        const uint32_t tS = t0 + C::COL_S + sb * 128 + wg * 64, tDP = t0 + C::COL_DP + wg * 64;
        const int col0 = at.tile * 128 + wg * 64;  // this thread's first query or key of the tile
        // The first mask values, loaded before S is ready.
        float m[MK == kBwdMaskNone || (KV && MK == kBwdMaskKey) ? 1 : 32];
        auto load_mask = [&](int half) {
          if constexpr (MK == kBwdMaskAdd || MK == kBwdMaskBool) {
            constexpr int SZ = MK == kBwdMaskBool ? 1 : 4;
            const int hq = KV ? h * p.group + at.g : h;
            const char* base = static_cast<const char*>(p.mask) +
                               ((size_t)b * p.mask_heads + (p.mask_heads == 1 ? 0 : hq)) * p.Nq * p.Nk * SZ;
            if constexpr (KV) {  // neighbouring lanes read neighbouring keys
              bwd_mask32<MK>(m, [&](int c) {
                return base + ((size_t)min(col0 + half * 32 + c, p.Nq - 1) * p.Nk + mine) * SZ;
              });
            } else {
              const char* mrow = base + (size_t)mine * p.Nk * SZ;
              bwd_mask32<MK>(m, [&](int c) { return mrow + (size_t)min(col0 + half * 32 + c, p.Nk - 1) * SZ; });
            }
          } else if constexpr (!KV && MK == kBwdMaskKey) {
            const float* mrow = static_cast<const float*>(p.mask) + (size_t)b * p.Nk;
            bwd_mask32<MK>(m, [&](int c) { return mrow + min(col0 + half * 32 + c, p.Nk - 1); });
          }
        };
        load_mask(0);
        const float4 *l4 = nullptr, *d4 = nullptr;
        if constexpr (KV) {
          ok = bwd_wait_warp(bars->st_full[j & 1], (j / 2) & 1, bars, p);
          if (!ok) break;
          l4 = reinterpret_cast<const float4*>(sStat + (j & 1) * 256 + wg * 64);
          d4 = l4 + 32;
        }
        // Pairs that the row does not see: above the diagonal, and keys past Nk
        // (as columns; as rows their gradients are not stored).
        int lo = 0, hi = 64;  // columns seen
        if constexpr (KV) {
          if (p.causal) lo = my - col0;
        } else {
          hi = min(hi, p.Nk - col0);
          if (p.causal) hi = min(hi, my - col0 + 1);
        }
        const bool edge = __any_sync(0xffffffffu, lo > 0 || hi < 64);
        ok = bwd_wait_warp(bars->s_full[sb], (j / C::NS) & 1, bars, p);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        float pr[64];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32];
          ptx::tmem_ld32x32b_x32(tS + half * 32, r);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float2 a0, a1;
            if constexpr (KV) {
              const float4 l = l4[half * 8 + c / 4];
              a0 = make_float2(l.x, l.y);
              a1 = make_float2(l.z, l.w);
              if constexpr (MK == kBwdMaskKey) {
                a0 = __fadd2_rn(a0, make_float2(key_add, key_add));
                a1 = __fadd2_rn(a1, make_float2(key_add, key_add));
              }
            } else {
              a0 = a1 = make_float2(nlse, nlse);
            }
            if constexpr (sizeof(m) > sizeof(float)) {
              a0 = __fadd2_rn(a0, make_float2(m[c], m[c + 1]));
              a1 = __fadd2_rn(a1, make_float2(m[c + 2], m[c + 3]));
            }
            const float2 e0 = bwd_exp(__uint_as_float(r[c]), __uint_as_float(r[c + 1]), sl2, a0);
            const float2 e1 = bwd_exp(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]), sl2, a1);
            const int k = half * 32 + c;
            pr[k] = e0.x;
            pr[k + 1] = e0.y;
            pr[k + 2] = e1.x;
            pr[k + 3] = e1.y;
          }
          if (half == 0) load_mask(1);
          if (edge) {
#pragma unroll
            for (int c = half * 32; c < half * 32 + 32; ++c)
              if (c < lo || c >= hi) pr[c] = 0.f;
          }
          if constexpr (KV) {  // over the columns just read
            uint32_t packed[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) packed[c] = ptx::pack_bf16x2(pr[half * 32 + 2 * c], pr[half * 32 + 2 * c + 1]);
            ptx::tmem_st32x32b_x16(tS + half * 16, packed);
          }
        }
        if constexpr (KV) {
          ptx::tmem_wait_st();
          ptx::tc_fence_before_sync();
          arrive(bars->p_ready[sb]);
        }
        ok = bwd_wait_warp(bars->dp_full, j & 1, bars, p);
        if (!ok) break;
        ptx::tc_fence_after_sync();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32], packed[16];
          ptx::tmem_ld32x32b_x32(tDP + half * 32, r);
          if constexpr (!KV) {
            if (half == 1) {  // dP has been read
              ptx::tc_fence_before_sync();
              arrive(bars->dp_free);
            }
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float4 d = make_float4(delta, delta, delta, delta);
            if constexpr (KV) d = d4[half * 8 + c / 4];
            const int k = half * 32 + c;
            const float2 x0 = __fadd2_rn(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])),
                                         make_float2(-d.x, -d.y));
            const float2 x1 = __fadd2_rn(make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])),
                                         make_float2(-d.z, -d.w));
            const float2 s0 = __fmul2_rn(x0, make_float2(pr[k], pr[k + 1]));
            const float2 s1 = __fmul2_rn(x1, make_float2(pr[k + 2], pr[k + 3]));
            packed[c / 2] = ptx::pack_bf16x2(s0.x, s0.y);
            packed[c / 2 + 1] = ptx::pack_bf16x2(s1.x, s1.y);
          }
          // over columns that have been read: dP's (dK dV), or S's
          ptx::tmem_st32x32b_x16((KV ? tDP : tS) + half * 16, packed);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        if constexpr (KV) {
          arrive(bars->ds_ready[0]);
          arrive(bars->st_empty[j & 1]);
        } else {
          arrive(bars->ds_ready[sb]);
        }
      }
      if (!ok) break;

      // The unit's gradients: dV by the first warpgroup and dK by the second, or
      // half of dQ's columns by each.
      const bool zero = pc.it0 == pc.it1;
      if (!zero) {
        ok = bwd_wait_warp(bars->acc_full, nu & 1, bars, p);
        if (!ok) break;
        ++nu;
        ptx::tc_fence_after_sync();
      }
      constexpr int NC = KV ? D : D / 2;
      const uint32_t tA = t0 + wg * NC;
      const int rows = KV ? p.Nk : p.Nq;
      if (pc.slot < 0) {
        const BwdTensor& o = KV && wg == 1 ? p.out1 : p.out0;
        const bool in = my < rows && bwd_check(p, bars, b * (KV ? p.Hk : p.Hq) + h < p.plan.units.heads,
                                               kCheckGradStore, pc.head, my);
        __nv_bfloat16* dst = o.p + b * o.b + h * o.h + (long long)my * o.n + (KV ? 0 : wg * NC);
        bwd_store_row<NC>(tA, KV && wg == 0 ? 1.f : p.scale, zero, in, dst);
      } else {
        const bool in = bwd_check(p, bars, pc.slot < 2 * p.plan.ctas, kCheckGradSlot, pc.slot, pc.head);
        bwd_store_part<NC>(tA, in, p.part + ((size_t)pc.slot * 2 + wg) * (128 * NC), row);
      }
      ptx::tc_fence_before_sync();
    }
    ptx::tc_fence_before_sync();
  }
  finish();
}

// -L and delta of every query row, and of the rows that fill up the last tile:
// L_i = log2(e) LSE_i (+inf for a row that sees nothing, so that its P is 0),
// delta_i = dO_i . O_i - dLSE_i.  HBM bound (O and dO are read once); D / 8
// neighbouring lanes share a row.
struct BwdPrepParams {
  BwdTensor out, dout;
  const float *lse, *dlse;  // [B][Hq][Nq]; dlse may be nullptr
  float *nlse, *delta;      // [B Hq][nqp]
  int Hq, Nq, nqp;
  long long rows;  // B Hq nqp
  FastDiv div_h;
};

template <int D>
__global__ void __launch_bounds__(256) fa_bwd_prep_kernel(const __grid_constant__ BwdPrepParams p) {
  constexpr int L = D / 8;  // lanes a row
  const long long i = (long long)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int piece = threadIdx.x % L;
  const bool live = i < p.rows;
  const long long bh = (live ? i : 0) / p.nqp;
  const int n = live ? (int)(i - bh * p.nqp) : 0;
  const int b = (int)p.div_h.div((uint32_t)bh), h = (int)bh - b * p.Hq;
  const bool in = live && n < p.Nq;
  float sum = 0.f;
  if (in) {
    const uint4 o = *reinterpret_cast<const uint4*>(p.out.p + b * p.out.b + h * p.out.h + n * p.out.n + piece * 8);
    const uint4 g = *reinterpret_cast<const uint4*>(p.dout.p + b * p.dout.b + h * p.dout.h + n * p.dout.n + piece * 8);
    const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // a bf16 is the upper half of its fp32
      sum = fmaf(__uint_as_float(ow[k] << 16), __uint_as_float(gw[k] << 16), sum);
      sum = fmaf(__uint_as_float(ow[k] & 0xffff0000u), __uint_as_float(gw[k] & 0xffff0000u), sum);
    }
  }
#pragma unroll
  for (int m = 1; m < L; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  if (live && piece == 0) {
    float nlse = -INFINITY;
    if (in) {
      const size_t at = (size_t)bh * p.Nq + n;
      const float lse = p.lse[at];
      if (lse != -INFINITY) nlse = -lse * 1.4426950408889634f;
      if (p.dlse) sum -= p.dlse[at];
    }
    p.nlse[i] = nlse;
    p.delta[i] = in ? sum : 0.f;
  }
}

// Joins the partial sums of cut units, in the order of their pieces.  Block
// (c, y, z): the unit that starts in CTA c's range, 8 columns, dV / dK (or dQ's halves).
template <int D, bool KV>
__global__ void __launch_bounds__(128) fa_bwd_join_kernel(const __grid_constant__ BwdParams p) {
  constexpr int NC = KV ? D : D / 2;
  int unit, last, slot;
  if (!bwd_join(p.plan, blockIdx.x, unit, last, slot)) return;
  const int row = threadIdx.x, col = blockIdx.y * 8, half = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
  float acc[8] = {};
  for (int c = blockIdx.x; c <= last; ++c) {
    if (c > (int)blockIdx.x) {
      slot = 2 * c;
      if (p.plan.cut[c].unit == p.plan.cut[c + 1].unit && p.plan.cut[c].it == p.plan.cut[c + 1].it) continue;
    }
    const float4* src = reinterpret_cast<const float4*>(p.part + ((size_t)slot * 2 + half) * (128 * NC)) +
                        (size_t)(col / 4) * 128 + row;
    const float4 a = src[0], e = src[128];
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += e.x; acc[5] += e.y; acc[6] += e.z; acc[7] += e.w;
  }
  int head, tile;
  p.plan.units.locate(unit, head, tile);
  const int heads = KV ? p.Hk : p.Hq;
  const int b = (int)p.div_h.div((uint32_t)head), h = head - b * heads;
  const int my = tile * 128 + row;
  if (my >= (KV ? p.Nk : p.Nq)) return;
  const BwdTensor& o = KV && half == 1 ? p.out1 : p.out0;
  const float mul = KV && half == 0 ? 1.f : p.scale;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = ptx::pack_bf16x2(acc[2 * i] * mul, acc[2 * i + 1] * mul);
  *reinterpret_cast<uint4*>(o.p + b * o.b + h * o.h + (long long)my * o.n + (KV ? 0 : half * NC) + col) =
      make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace fa
