// fa_cache_chunk.cuh — the cached attention (see fa_cache_attn.cuh) for many
// rows: prompts, chunks of video, and drafts of grouped heads.
//
// Here the tensor cores are the bound, so the products have the rows on the M
// side, as in the forward kernel: 256 rows (two tiles of 128) a CTA, one thread
// a row in the softmax, P over S in tensor memory, two softmax warpgroups that
// ping-pong.
//
// S = Q K^T runs as e4m3 x e4m3 with K's codes as they are: a row of Q is
// s (hi + lo), two e4m3 numbers (s a power of two that puts the row's largest
// element in (224, 448]), and S accumulates both products.  Two e4m3 MMAs cost
// what one bf16 MMA does, and K needs no conversion.  An element of q is exact
// above 2^-10 of its row's largest, and off by 2^-18 of that below.  The scales
// of q's row and of K's page go into the softmax's multiplier.
//
// P V runs in f16, which holds every e4m3 number: two warps turn V's codes into
// f16 in the layout that the MMA reads, one tile ahead.  (One instruction for
// two codes.  Code times scale in bf16 instead cost two to four times as many,
// and those two warps became the bound: 394 us for 2048 rows of 24 heads on
// 16896 keys of 128, 510 us by moving bits, where f16 alone brought it to 292.)
// P is rounded to f16: 11 bits, or 2^-25 of the row's largest p.  It carries its
// page's scale of V relative to the largest that the row has seen so far, v_ref, so
// that 2^-25 stands for at most v_ref / scale times as much of p; O is in units of
// v_ref and rescaled when that grows.
//
// In the tiles of which some row of the unit does not see every key (the
// diagonal's with causal, and a sequence's last) codes of V that are NaN become
// zeros, so that 0 times NaN does not reach the rows that do not see their keys.
// A row that does see one finds out at its end (chunk_sees_nan) and gives NaN.
//
// Units' tiles are cut into equal ranges, one per CTA (1 CTA per SM), as in
// fa_cache_attn.cuh: 192 units of 256 rows on 152 SMs would leave a third of
// the second round idle.
//
// Those 2048 rows, causal, take 255 to 260 us with the join of the cut units:
// 1.53 to 1.56 PFLOP/s, tensor pipe 70 % active.  What is left is the softmax
// between a tile's two products and what a stretch costs once (Q's two parts,
// the epilogue); without cut units (19 heads, not causal) the rate is 1.68
// PFLOP/s.  10800 rows on themselves, the last row tile of 48, take 563 us, 1.27
// PFLOP/s: 43 row tiles with 1 to 85 key tiles each.
//
// PAIR.  With 128 rows or fewer there is one row tile, and its S, softmax and
// P V would wait for one another; the two warpgroups then take the even and the
// odd key tiles of the same rows, with a maximum, a sum and an O each, and the
// second's results are joined to the first's at the end of the stretch.
// (Deeper rings of codes in the other row tile's shared memory measured slower.)
//
// Warps: 0-3 and 4-7 softmax of the two row tiles, 8 producer, 9 MMA issuer,
// 10-11 V conversion.
#pragma once

#include "fa_cache_attn.cuh"
#include "fa_cache_launch.h"

namespace fa {

constexpr int kChunkThreads = 384;
constexpr int kChunkConvert = 64;  // threads that convert V
constexpr int kChunkStagesMax = 8;

template <int D, bool PAIR>
struct ChunkCfg {
  static constexpr int T8 = kCacheTile * D;              // 128 rows in e4m3
  static constexpr int T16 = 2 * T8;                     // in f16
  static constexpr int SW = D >= 64 ? 128 : 64;          // swizzle span of the f16 tile
  static constexpr int CHUNK = kCacheTile * SW;          // its 128-row blocks of SW bytes
  static constexpr uint32_t LAYOUT8 = D == 128 ? 2u : (D == 64 ? 4u : 6u);
  static constexpr uint32_t LAYOUT16 = D >= 64 ? 2u : 4u;
  static constexpr int Q_TILES = PAIR ? 1 : 2;
  static constexpr int V_STAGES = kChunkVStages;         // V in f16
  static constexpr int K_STAGES = chunk_k_stages(D, PAIR);  // K and V codes
  static constexpr int SMEM_BYTES = 2 * Q_TILES * T8 + 2 * K_STAGES * T8 + V_STAGES * T16 + 2048;
  static_assert(K_STAGES <= kChunkStagesMax && K_STAGES + V_STAGES < kChunkMeta, "rings");
  static constexpr int COL_S = 0, COL_O = 256;           // S and O of tile t: + 128 t, + D t
};

struct ChunkBars {
  uint64_t k_full[kChunkStagesMax], k_empty[kChunkStagesMax], v8_full[kChunkStagesMax], v8_empty[kChunkStagesMax];
  uint64_t v_full[2], v_empty[2];
  uint64_t meta_full[kChunkMeta];
  uint64_t q_ready[2], s_full[2], p_half[2], p_ready[2], o_full[2], joined, drain;
  CacheRange plan;
  uint32_t tmem_base;
  volatile int abort_flag;
  volatile int v_nan;  // a NaN was taken out of some tile's V
  alignas(16) float ks[kChunkMeta][4];
  alignas(16) float vs[kChunkMeta][4];  // scales of a tile's 32-token groups
};
static_assert(sizeof(ChunkBars) <= 2048, "barrier space");

// 16 codes as f16 (exact; NaN stays NaN).
__device__ __forceinline__ void chunk_f16(const uint4& v, uint4 (&out)[2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[k]) : "h"((uint16_t)(w[k / 2] >> (16 * (k & 1)))));
  out[0] = make_uint4(o[0], o[1], o[2], o[3]);
  out[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// The last key that every row of a stretch's unit sees (limits grow with the row).
__device__ __forceinline__ int chunk_least(const CacheRows& rows, const CacheSegment& sg) {
  return rows.limit(sg.len, sg.first, (int)rows.by_g.div((uint32_t)sg.rt * kChunkRows));
}

// Whether one of the keys first .. last of a sequence has a NaN in V (one
// thread; out of line and slow, for rows of a CTA that has met one).
template <int D>
__device__ __noinline__ bool chunk_sees_nan(const CacheView& c, int b, int h, int first, int last) {
  const int shift = 31 - __clz(c.page);  // page is a power of two
  bool bad = false;
  uint32_t nan = 0;
  for (int key = first; key <= last && !nan; ++key) {
    const long long at = (long long)cache_page(c.table[(long long)b * c.width + (key >> shift)], c.num_pages, bad) * c.H + h;
    const uint4* row = reinterpret_cast<const uint4*>(c.code[1] + ((at << shift) + (key & (c.page - 1))) * D);
    for (int i = 0; i < D / 16; ++i) nan |= e4m3_nan(row[i]);
  }
  return nan != 0;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ONE: a page is a whole tile (128 tokens), so a tile has one scale.
// PAIR: one row tile, two key tiles at a time (R <= 128).
template <int D, bool ONE, bool PAIR>
__global__ void __launch_bounds__(kChunkThreads, 1) fa_cache_chunk_kernel(const __grid_constant__ CacheAttnParams p) {
  using C = ChunkCfg<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                              // tile t: hi at 2 t, lo at 2 t + 1
  uint8_t* sK = sQ + 2 * C::Q_TILES * C::T8;
  uint8_t* sV8 = sK + C::K_STAGES * C::T8;
  uint8_t* sV = sV8 + C::K_STAGES * C::T8;
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(sV + C::V_STAGES * C::T16);
  const int warp = threadIdx.x / 32;
  const uint32_t lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    if (p.cut) p.cut[blockIdx.x].x = -1;
    for (int s = 0; s < C::K_STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->k_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->k_empty[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->v8_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->v8_empty[s]), kChunkConvert);
    }
    for (int s = 0; s < C::V_STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->v_full[s]), kChunkConvert);
      ptx::mbar_init(ptx::smem_u32(&bars->v_empty[s]), 1);
    }
    for (int s = 0; s < kChunkMeta; ++s) ptx::mbar_init(ptx::smem_u32(&bars->meta_full[s]), 1);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bars->q_ready[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bars->s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->p_half[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bars->p_ready[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bars->o_full[t]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->joined), 128);
    ptx::mbar_init(ptx::smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    bars->v_nan = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 8) cache_plan(p.rows, p.ctas, p.status, lane, &bars->plan);
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  CacheWalk walk;
  walk.start(p.rows, bars->plan.t0, bars->plan.t1, bars->plan.b0, bars->plan.base0);
  CacheSegment sg;
  auto finish = [&]() {
    ptx::named_barrier_sync(1, kChunkThreads);
    if (warp == 9) {
      ptx::tc_fence_after_sync();
      ptx::tmem_dealloc(tmem, 512);
    }
  };

  if (warp >= 10) {
    // -------------------------------------------------------- V conversion --
    // A warp's 32 lanes take 16-byte pieces so that eight lanes in a row read
    // and write all banks: four pieces of a row and of the row 5 away in the
    // swizzle pattern (D = 32: two pieces of four rows).
    constexpr int CPR = D / 16, HALVES = D == 128 ? 2 : 1, RPI = D == 32 ? 16 : 8;
    constexpr int STEPS = kCacheTile / RPI / 2 * HALVES;  // 32 pieces a warp each
    static_assert(CPR * kCacheTile == kChunkConvert * STEPS, "pieces of a tile");
    const int w = warp - 10;
    const int q = (int)lane >> 2;
    const int in_row = D == 32 ? (int)lane >> 1 : (q >> 1) ^ ((q & 1) * 5);
    const int in_col = D == 32 ? (int)lane & 1 : (int)lane & 3;
    uint32_t it = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int least = chunk_least(p.rows, sg);
      for (int j = 0; j < sg.ntiles; ++j, ++it) {
        const uint32_t s8 = it % C::K_STAGES, s16 = it % C::V_STAGES;
        ok = cache_wait(&bars->v8_full[s8], (it / C::K_STAGES) & 1, bars, p);
        if (!ok) break;
        uint8_t* src = sV8 + s8 * C::T8;
        uint8_t* dst = sV + s16 * C::T16;
        // Rows past the length may hold anything, NaN among it: zeros.
        const int held = sg.len - (sg.tile0 + j) * kCacheTile;
        // Piece k of this lane: its row and 16-channel column, its 32 bytes of f16.
        auto row_of = [&](int k) { return ((k / HALVES) * 2 + w) * RPI + in_row; };
        auto col_of = [&](int k) { return (HALVES == 2 ? (k & 1) * 4 : 0) + in_col; };
        // NaN in this lane's own pieces: before the wait for room in the ring, which
        // hides it, and rolled up (cold code costs its instruction misses).
        if ((sg.tile0 + j) * kCacheTile + (kCacheTile - 1) > least) {
#pragma unroll 1
          for (int k = 0; k < STEPS; ++k) {
            uint4* piece = reinterpret_cast<uint4*>(src + cache_swizzle<D>(row_of(k), 16 * col_of(k)));
            if (!e4m3_nan(*piece) || row_of(k) >= held) continue;
            auto clean = [](uint32_t codes) { return codes & ~((e4m3_nan(codes) >> 7) * 255u); };
            *piece = make_uint4(clean(piece->x), clean(piece->y), clean(piece->z), clean(piece->w));
            bars->v_nan = 1;
          }
        }
        ok = cache_wait(&bars->v_empty[s16], ((it / C::V_STAGES) & 1) ^ 1, bars, p);
        if (!ok) break;
        constexpr int BATCH = STEPS < 8 ? STEPS : 8;  // loads in flight together
#pragma unroll 1
        for (int k0 = 0; k0 < STEPS; k0 += BATCH) {
          uint4 v[BATCH];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            v[k] = *reinterpret_cast<const uint4*>(src + cache_swizzle<D>(row_of(k0 + k), 16 * col_of(k0 + k)));
            if (row_of(k0 + k) >= held) v[k] = make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            uint4 o[2];
            chunk_f16(v[k], o);
            const int row = row_of(k0 + k);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int piece = 2 * col_of(k0 + k) + x;  // 16 bytes of the f16 row
              const uint32_t at = C::SW == 128
                                      ? (uint32_t)((piece >> 3) * C::CHUNK + row * 128 + (((piece & 7) ^ (row & 7)) << 4))
                                      : (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
              *reinterpret_cast<uint4*>(dst + at) = o[x];
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        ptx::mbar_arrive(ptx::smem_u32(&bars->v_full[s16]));
        ptx::mbar_arrive(ptx::smem_u32(&bars->v8_empty[s8]));
      }
    }
    __syncwarp();
    finish();
    return;
  }
  if (warp >= 8) {
    if (warp == 8) {
      // ---------------------------------------------------------- producer --
      if (lane == 0) {
        ptx::tma_prefetch_desc(&p.tm_k);
        ptx::tma_prefetch_desc(&p.tm_v);
      }
      const int page = p.c.page, ppt = kCacheTile / page, batch = 32 / ppt;
      uint32_t it = 0, skipped = 0xffffffffu;
      bool ok = true;
      CachePages pages;
      while (ok && walk.next(sg)) {
        const int npages = sg.len == 0 ? 0 : (sg.len - 1) / page + 1;
        // The unit's rows of Q on their way to L2 while the last unit is finished.
#pragma unroll 1
        for (int r = sg.rt * kChunkRows + (int)lane; r < min(p.rows.R, (sg.rt + 1) * kChunkRows); r += 32) {
          const char* q = reinterpret_cast<const char*>(p.q + p.row_at(sg.b, sg.h, r) * D);
          for (int x = 0; x < D * 2; x += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + x));
        }
        for (int j = 0; j < sg.ntiles; ++j, ++it) {
          const int in_batch = j % batch;
          if (in_batch == 0) pages.fetch(p, sg, j, lane);
          const uint32_t s = it % C::K_STAGES, ph = ((it / C::K_STAGES) & 1) ^ 1, meta = it % kChunkMeta;
          ok = cache_wait(&bars->k_empty[s], ph, bars, p) && cache_wait(&bars->v8_empty[s], ph, bars, p);
          if (!ok) break;
          if (p.inject_stall && blockIdx.x == 0 && it == 1) {  // nothing arrives: consumers time out
            skipped = it;
            continue;
          }
          const int my_id = __shfl_sync(0xffffffffu, pages.id, in_batch * ppt + (int)(lane % ppt));
          const int n = max(0, min(ppt, npages - (sg.tile0 + j) * ppt));  // pages that hold tokens
          const uint32_t kf = ptx::smem_u32(&bars->k_full[s]), vf = ptx::smem_u32(&bars->v8_full[s]);
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(kf, (uint32_t)(n * page * D));
            ptx::mbar_arrive_expect_tx(vf, (uint32_t)(n * page * D));
          }
          __syncwarp();
          if ((int)lane < n) {
            const uint32_t off = s * C::T8 + lane * page * D;
            const int at = my_id * p.c.H + sg.h;
            ptx::tma_load_3d(ptx::smem_u32(sK) + off, &p.tm_k, kf, 0, 0, at);
            ptx::tma_load_3d(ptx::smem_u32(sV8) + off, &p.tm_v, vf, 0, 0, at);
          }
          // The scales, for which the copies do not wait.  Their slot was last
          // used kChunkMeta tiles ago; the V slot that is free now means that
          // tile it - K_STAGES - V_STAGES is through the softmax.
          const int g = in_batch * ppt + (int)(lane & 3) * 32 / page;  // page of this lane's 32 tokens
          const float my_ks = __shfl_sync(0xffffffffu, pages.ks, g), my_vs = __shfl_sync(0xffffffffu, pages.vs, g);
          if (lane < 4) {
            bars->ks[meta][lane] = my_ks;
            bars->vs[meta][lane] = my_vs;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->meta_full[meta]));
        }
      }
      if (!ok && lane == 0) {
        // Drain: every copy issued has landed once its stage's last phase is complete.
        for (int s = 0; s < C::K_STAGES; ++s) {
          uint32_t n = it > (uint32_t)s ? (it - 1 - s) / C::K_STAGES + 1 : 0;
          if (skipped < it && skipped % C::K_STAGES == (uint32_t)s) --n;
          if (n) {
            cache_drain(&bars->k_full[s], (n - 1) & 1, p);
            cache_drain(&bars->v8_full[s], (n - 1) & 1, p);
          }
        }
      }
    } else if (warp == 9) {
      // --------------------------------------------------------------- MMA --
      constexpr uint32_t IDESC_S = (1u << 4) | (16u << 17) | (8u << 24);  // e4m3, 128 x 128
      constexpr uint32_t IDESC_PV = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                    (8u << 24);                           // f16, 128 x D, B transposed
      constexpr uint32_t kVStep = (16 * C::SW) >> 4;                      // 16 keys of V
      const uint64_t dq = cache_desc(ptx::smem_u32(sQ), 16, 8 * D, C::LAYOUT8);
      const uint64_t dk = cache_desc(ptx::smem_u32(sK), 16, 8 * D, C::LAYOUT8);
      const uint64_t dv = cache_desc(ptx::smem_u32(sV), C::CHUNK, 8 * C::SW, C::LAYOUT16);
      const uint32_t q_hi = (uint32_t)(dq >> 32), k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
      auto issue_s = [&](int t, uint32_t stage) {
        const uint32_t d = tmem + C::COL_S + t * 128, b = (uint32_t)dk + stage * (C::T8 >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // hi, then lo on top
          const uint32_t a = (uint32_t)dq + (2 * (PAIR ? 0 : t) + part) * (C::T8 >> 4);
          if constexpr (D == 128)
            ptx::mma_ss_f8_x4_el<2, 4, 6>(d, a, q_hi, b, k_hi, IDESC_S, part);
          else if constexpr (D == 64)
            ptx::mma_ss_f8_x2_el<2>(d, a, q_hi, b, k_hi, IDESC_S, part);
          else
            ptx::mma_ss_f8_x1_el(d, a, q_hi, b, k_hi, IDESC_S, part);
        }
        ptx::mma_commit_el(ptx::smem_u32(&bars->s_full[t]));
      };
      uint32_t it = 0, pc[2] = {0, 0}, qc[2] = {0, 0};
      // O_t += P_t V in two halves of 64 keys, each as soon as its P is there.
      auto issue_pv = [&](int t, uint32_t stage, bool first, uint32_t parity) -> bool {
        const uint32_t b = (uint32_t)dv + stage * (C::T16 >> 4), d = tmem + C::COL_O + t * D;
        const uint32_t a = tmem + C::COL_S + t * 128;
        if (!cache_wait(&bars->p_half[t], parity, bars, p)) return false;
        ptx::tc_fence_after_sync();
        ptx::mma_ts_x4_el<kVStep>(d, a, b, v_hi, IDESC_PV, first ? 0u : 1u);
        if (!cache_wait(&bars->p_ready[t], parity, bars, p)) return false;
        ptx::tc_fence_after_sync();
        ptx::mma_ts_x4_el<kVStep>(d, a + 32, b + 4 * kVStep, v_hi, IDESC_PV, 1u);
        return true;
      };
      auto take_k = [&](uint32_t n) -> bool {
        const bool r = cache_wait(&bars->k_full[n % C::K_STAGES], (n / C::K_STAGES) & 1, bars, p);
        ptx::tc_fence_after_sync();
        return r;
      };
      bool ok = true;
      while (ok && walk.next(sg)) {
        const bool two = sg.rt * kChunkRows + 128 < p.rows.R;
        ok = take_k(it) && cache_wait(&bars->q_ready[0], qc[0] & 1, bars, p);
        if (!ok) break;
        ++qc[0];
        ptx::tc_fence_after_sync();
        issue_s(0, it % C::K_STAGES);
        if constexpr (PAIR) {
          // S of tile j + 2 follows P V of tile j, in the same columns.
          const uint32_t end = it + (uint32_t)sg.ntiles, first = it;
          ptx::mma_commit_el(ptx::smem_u32(&bars->k_empty[it % C::K_STAGES]));
          auto next_s = [&](uint32_t n) -> bool {
            if (!take_k(n)) return false;
            issue_s((int)((n - first) & 1), n % C::K_STAGES);
            ptx::mma_commit_el(ptx::smem_u32(&bars->k_empty[n % C::K_STAGES]));
            return true;
          };
          if (first + 1 < end) ok = next_s(first + 1);
          for (; ok && it < end; ++it) {
            const int t = (int)((it - first) & 1);
            const uint32_t sv = it % C::V_STAGES;
            ok = cache_wait(&bars->v_full[sv], (it / C::V_STAGES) & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            ok = issue_pv(t, sv, it < first + 2, pc[t] & 1);
            if (!ok) break;
            ++pc[t];
            ptx::mma_commit_el(ptx::smem_u32(&bars->v_empty[sv]));
            if (it + 2 < end)
              ok = next_s(it + 2);
            else
              ptx::mma_commit_el(ptx::smem_u32(&bars->o_full[t]));
          }
          continue;
        }
        if (two) {
          ok = cache_wait(&bars->q_ready[1], qc[1] & 1, bars, p);
          if (!ok) break;
          ++qc[1];
          ptx::tc_fence_after_sync();
          issue_s(1, it % C::K_STAGES);
        }
        ptx::mma_commit_el(ptx::smem_u32(&bars->k_empty[it % C::K_STAGES]));
        for (int j = 0; j < sg.ntiles; ++j, ++it) {
          const bool more = j + 1 < sg.ntiles;
          const uint32_t sv = it % C::V_STAGES, sk = (it + 1) % C::K_STAGES;
          ok = cache_wait(&bars->v_full[sv], (it / C::V_STAGES) & 1, bars, p);
          if (!ok) break;
          ptx::tc_fence_after_sync();
          ok = issue_pv(0, sv, j == 0, pc[0] & 1);
          if (!ok) break;
          ++pc[0];
          if (more) {
            ok = take_k(it + 1);
            if (!ok) break;
            issue_s(0, sk);
          } else {
            ptx::mma_commit_el(ptx::smem_u32(&bars->o_full[0]));
          }
          if (two) {
            ok = issue_pv(1, sv, j == 0, pc[1] & 1);
            if (!ok) break;
            ++pc[1];
            if (!more) ptx::mma_commit_el(ptx::smem_u32(&bars->o_full[1]));
          }
          ptx::mma_commit_el(ptx::smem_u32(&bars->v_empty[sv]));
          if (more) {
            if (two) issue_s(1, sk);
            ptx::mma_commit_el(ptx::smem_u32(&bars->k_empty[sk]));
          }
        }
      }
      ptx::mma_commit_el(ptx::smem_u32(&bars->drain));
      cache_drain(&bars->drain, 0, p);
    }
    __syncwarp();
    finish();
    return;
  }

  // ---------------------------------------------------------------- softmax --
  const int t = warp / 4;
  const int in_tile = (warp % 4) * 32 + (int)lane;  // row of the tile, lane of tensor memory
  const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
  const uint32_t tS = tmem + lane_base + C::COL_S + t * 128, tO = tmem + lane_base + C::COL_O + t * D;
  const int qt = PAIR ? 0 : t;  // row tile
  uint8_t* q_hi = sQ + 2 * qt * C::T8;
  uint8_t* q_lo = q_hi + C::T8;
  constexpr int STEP = PAIR ? 2 : 1;
  uint32_t it = 0, sc = 0, oc = 0, jc = 0;
  bool ok = true;
  while (ok && walk.next(sg)) {
    const int row0 = sg.rt * kChunkRows + qt * 128;
    // (tile 1 of a unit cut short; the second of a pair where there is one key tile)
    if (row0 >= p.rows.R || (PAIR && t >= sg.ntiles)) {
      it += (uint32_t)sg.ntiles;
      continue;
    }
    const int row = row0 + in_tile;
    const bool valid = row < p.rows.R;
    const long long at = p.row_at(sg.b, sg.h, valid ? row : row0);
    // The warp's 32 rows of Q as s (hi + lo), D / 8 lanes to a row.  The MMAs
    // that read the last unit's Q are done: their S has been read.
    float c = 0.f;
    {
      // (Rolled up, four steps' loads in flight: this code runs once a unit.
      // Unrolled it cost more time in instruction misses than in work; with one
      // load in flight, in waiting for memory.)
      constexpr int LPR = D / 8, RPS = 32 / LPR;  // lanes of a row, rows of a step
      constexpr int BATCH = 4;
      const float sign = p.scale_log2 < 0.f ? -1.f : 1.f;  // a negative scale turns the row round
      uint4 next[BATCH];
      auto fetch = [&](int k0) {
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
          const long long from = __shfl_sync(0xffffffffu, at, (k0 + x) * RPS + (int)lane / LPR);
          next[x] = __ldg(reinterpret_cast<const uint4*>(p.q + from * D) + lane % LPR);
        }
      };
      fetch(0);
#pragma unroll 1
      for (int k0 = 0; k0 < LPR; k0 += BATCH) {
        uint4 v[BATCH];
#pragma unroll
        for (int x = 0; x < BATCH; ++x) v[x] = next[x];
        if (k0 + BATCH < LPR) fetch(k0 + BATCH);
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
          const int k = k0 + x;
          const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
          const uint32_t two = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                        __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
          uint32_t amax = max(two << 16, two & 0xffff0000u);  // magnitude as fp32 bits
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const int e2 = max((int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
          const float inv = __int_as_float((127 - e2) << 23) * sign;
          uint32_t h[4], l[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = __fmul2_rn(make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)),
                                        make_float2(inv, inv));
            h[e] = e4m3x2_bits(a.x, a.y);
            const float2 left = __ffma2_rn(e4m3x2_value(h[e]), make_float2(-1.f, -1.f), a);
            l[e] = e4m3x2_bits(left.x, left.y);
          }
          const uint32_t off = cache_swizzle<D>((warp % 4) * 32 + k * RPS + (int)lane / LPR, 8 * ((int)lane % LPR));
          if (qt == t) {  // (the second of a pair needs the rows' scales only)
            *reinterpret_cast<uint2*>(q_hi + off) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
            *reinterpret_cast<uint2*>(q_lo + off) = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
          }
          // a row that holds a number that is not finite gives NaN
          const float cr = amax >= 0x7f800000u ? __int_as_float(0x7fc00000)
                                               : __int_as_float((e2 + 127) << 23) * fabsf(p.scale_log2);
          const float mine = __shfl_sync(0xffffffffu, cr, ((int)lane % RPS) * LPR);
          if ((int)lane / RPS == k) c = mine;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (qt == t) ptx::mbar_arrive(ptx::smem_u32(&bars->q_ready[t]));
    }
    const int lim = p.rows.limit(sg.len, sg.first, (int)p.rows.by_g.div((uint32_t)(valid ? row : row0)));
    if (lim < 0) c = 0.f;  // a row of q that sees no key counts for nothing, NaN or not
    const int wlim = __reduce_min_sync(0xffffffffu, lim);
    float m = -INFINITY, l = 0.f;
    float v_ref = 0.f;  // the largest scale of V that the row has seen so far: the unit of O
    const int j0 = PAIR ? t : 0;
    for (int j = j0; j < sg.ntiles; j += STEP) {
      const int kbase = (sg.tile0 + j) * kCacheTile;
      const uint32_t n = it + (uint32_t)j, meta = n % kChunkMeta;
      // On a stretch's first tile, S before the scales: it is issued after K of the
      // tile was announced, so every earlier tile's scales have come, and the
      // parity of the tile's own names one phase only.  A warpgroup that skipped
      // a stretch has waited for nothing of it: the slot could still be at the
      // phase of tile n - 32, whose parity is the same.  (From one tile of a
      // stretch to the next the waits that are there suffice.  S first on every
      // tile costs 5 %: the chain from S to P is the bound.)
      if (j == j0) {
        ok = cache_wait(&bars->s_full[t], sc & 1, bars, p);
        if (!ok) break;
      }
      ok = cache_wait(&bars->meta_full[meta], (n / kChunkMeta) & 1, bars, p);
      if (!ok) break;
      constexpr int G = ONE ? 1 : 4;  // groups of keys with scales of their own
      float sl[G];  // multipliers of the raw scores: positive, or NaN
      int ve[G];    // exponents of the scales of V, less that of the unit (0 at most)
      float ks[G], vs[G], v_new = v_ref;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        ks[g] = bars->ks[meta][g];
        vs[g] = bars->vs[meta][g];
        // (pages past the row's last key leave its unit alone)
        if (kbase + g * (128 / G) <= lim) v_new = fmaxf(v_new, vs[g]);
      }
      const int v_down = max((__float_as_int(v_ref) >> 23) - (__float_as_int(v_new) >> 23), -100);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        sl[g] = c * ks[g];
        if (sl[g] < 1.17549435e-38f) sl[g] = 1.17549435e-38f;
        ve[g] = min(max((__float_as_int(vs[g]) >> 23) - (__float_as_int(v_new) >> 23), -100), 0);
      }
      v_ref = v_new;
      ok = cache_wait(&bars->s_full[t], sc & 1, bars, p);
      if (!ok) break;
      ++sc;
      ptx::tc_fence_after_sync();
      float s[128];
      {
        uint32_t r[128];
        ptx::tmem_ld32x32b_x128(tS, r);
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(r[i]);
      }
      if (kbase + kCacheTile - 1 > wlim) {  // some row does not see every key
        const int hi = lim - kbase;
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = i <= hi ? s[i] : -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        constexpr int N = 128 / G;
        float a[4] = {s[N * g], s[N * g + 1], s[N * g + 2], s[N * g + 3]};
#pragma unroll
        for (int i = 4; i < N; i += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (i + 2 * x < N) a[x] = ptx::fmax3(a[x], s[N * g + i + 2 * x], s[N * g + i + 2 * x + 1]);
        mx = fmaxf(mx, fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * sl[g]);
      }
      // The reference moves only when the maximum grew by more than 8 (exact:
      // O, l and LSE use the same one).
      const float m_new = fmaxf(m, mx);
      const bool grow = m_new - m > 8.f;  // -inf - -inf: NaN, false
      float alpha = 1.f;
      if (grow) {
        alpha = ptx::ex2(m - m_new);
        m = m_new;
      }
      const float m_use = m == -INFINITY ? 0.f : m;
      l *= alpha;
      const bool rescale = j > j0 && __any_sync(0xffffffffu, grow || v_down < 0);
      alpha *= __int_as_float((v_down + 127) << 23);  // for O, which is in units of v_ref
      auto release = [&](uint64_t* bar) {
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        ptx::mbar_arrive(ptx::smem_u32(bar));
      };
      // p carries the ratio of its page's scale of V to v_ref: a shift of the
      // exponent, taken back from the sum.
      float2 lsum = make_float2(0.f, 0.f);
#pragma unroll
      for (int cb = 0; cb < 128; cb += 32) {
        const int g = cb * G / 128;
        const float shift = (float)ve[g] - m_use;
        const float2 nm2 = make_float2(shift, shift), sl2 = make_float2(sl[g], sl[g]);
        uint32_t packed[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 x = __ffma2_rn(make_float2(s[cb + i], s[cb + i + 1]), sl2, nm2);
          const float2 e = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
          lsum = __fadd2_rn(lsum, e);
          packed[i / 2] = pack_f16x2(e.x, e.y);
        }
        ptx::tmem_st32x32b_x16(tS + cb / 2, packed);
        if (!ONE || cb == 96) {
          l = fmaf(lsum.x + lsum.y, __int_as_float((127 - ve[g]) << 23), l);
          lsum = make_float2(0.f, 0.f);
        }
        if (cb == 32 && !rescale) release(&bars->p_half[t]);
      }
      if (rescale) {
        // P V of the last tile is done: the S just read was issued after it.
#pragma unroll 1
        for (int cb = 0; cb < D; cb += 32) {
          uint32_t r[32];
          ptx::tmem_ld32x32b_x32(tO + cb, r);
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
          ptx::tmem_st32x32b_x32(tO + cb, r);
        }
        release(&bars->p_half[t]);
      }
      release(&bars->p_ready[t]);
    }
    if (!ok) break;
    it += (uint32_t)sg.ntiles;
    ok = cache_wait(&bars->o_full[t], oc & 1, bars, p);
    if (!ok) break;
    ++oc;
    ptx::tc_fence_after_sync();
    // Partial O four channels at a time, the rows of a warp side by side.  The
    // second of a pair leaves its results in the upper rows of the CTA's slot
    // (128 rows or fewer leave them free), where the first takes them.
    const bool whole = sg.ntiles == sg.total, join = PAIR && sg.ntiles > 1;
    const long long slot = whole ? 2LL * blockIdx.x : cache_slot((int)blockIdx.x, bars->plan.t0, sg.unit_t0);
    const int in_unit = t * 128 + in_tile;
    float4* part = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * kChunkRows;
    float2* part_ml = reinterpret_cast<float2*>(p.part_ml) + slot * kChunkRows;
    if (p.part_o && !p.check_slot(slot)) break;
    if (!p.check_row(at)) break;
    float own = v_ref, other = 0.f;
    if (join && t == 0) {
      ok = cache_wait(&bars->joined, jc & 1, bars, p);
      if (!ok) break;
      ++jc;
      const float2 ml = part_ml[128 + in_tile];
      const float m_all = fmaxf(l == 0.f ? -INFINITY : m, ml.y == 0.f ? -INFINITY : ml.x);
      const float w = l == 0.f ? 0.f : ptx::ex2(m - m_all);
      other = ml.y == 0.f ? 0.f : ptx::ex2(ml.x - m_all);
      own *= w;
      l = fmaf(w, l, other * ml.y);
      m = m_all;
    }
    if (bars->v_nan) {  // the tiles that were looked through, as far as this row sees
      const int from = max(sg.tile0, (chunk_least(p.rows, sg) + 1) / kCacheTile) * kCacheTile;
      const int to = min(lim, (sg.tile0 + sg.ntiles - 1) * kCacheTile + (kCacheTile - 1));
      if (chunk_sees_nan<D>(p.c, sg.b, sg.h, from, to)) own = __int_as_float(0x7fc00000);
    }
    const bool out = whole && t == qt;
    if (out) {
      own = l == 0.f ? 0.f : own / l;
      other = l == 0.f ? 0.f : other / l;
    }
#pragma unroll 1
    for (int cb = 0; cb < D; cb += 32) {
      uint32_t r[32];
      ptx::tmem_ld32x32b_x32(tO + cb, r);
      float o[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(r[i]) * own;
      if (join && t == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 x = part[(cb / 4 + k) * kChunkRows + 128 + in_tile];
          o[4 * k] = fmaf(other, x.x, o[4 * k]);
          o[4 * k + 1] = fmaf(other, x.y, o[4 * k + 1]);
          o[4 * k + 2] = fmaf(other, x.z, o[4 * k + 2]);
          o[4 * k + 3] = fmaf(other, x.w, o[4 * k + 3]);
        }
      }
      if (out) {
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + cb);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(ptx::pack_bf16x2(o[8 * k], o[8 * k + 1]), ptx::pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                ptx::pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), ptx::pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          part[(cb / 4 + k) * kChunkRows + in_unit] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
    if (out) {
      if (valid) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    } else {
      part_ml[in_unit] = make_float2(m, l);
      if (t != qt)
        ptx::mbar_arrive(ptx::smem_u32(&bars->joined));
      else if (threadIdx.x == 0)
        p.note_cut(sg, bars->plan);
    }
    ptx::tc_fence_before_sync();  // O has been read: the next unit's products may overwrite it
  }
  ptx::tc_fence_before_sync();
  finish();
}

// Joins the pieces of the units cut between CTAs, as fa_cache_merge_kernel;
// one block for 16 channels of a unit's 256 rows, thread = row.
template <int D>
__global__ void __launch_bounds__(kChunkRows) fa_cache_chunk_merge_kernel(const __grid_constant__ CacheAttnParams p) {
  constexpr int PARTS = D / 16;
  const int c0 = blockIdx.x / PARTS, part = blockIdx.x - c0 * PARTS;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // see fa_cache_merge_kernel
  const int4 cut = p.cut[c0];
  const int row = cut.z * kChunkRows + (int)threadIdx.x, c1 = cut.w >> 1;
  if (cut.x < 0 || row >= p.rows.R || !p.check_slot(2LL * c1)) return;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + threadIdx.x;
  auto slot = [&](int c) { return 2LL * c + (c == c0 ? (cut.w & 1) : 0); };
  float m = -INFINITY, l = 0.f;
  for (int c = c0; c <= c1; ++c) {
    const float2 x = ml[slot(c) * kChunkRows];
    if (x.y != 0.f) m = fmaxf(m, x.x);
  }
  float4 o[4] = {};
  for (int c = c0; c <= c1; ++c) {
    const float2 x = ml[slot(c) * kChunkRows];
    if (x.y == 0.f) continue;
    const float w = ptx::ex2(x.x - m);
    l = fmaf(w, x.y, l);
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + (slot(c) * (D / 4) + part * 4) * kChunkRows + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = src[k * kChunkRows];
      o[k].x = fmaf(w, v.x, o[k].x);
      o[k].y = fmaf(w, v.y, o[k].y);
      o[k].z = fmaf(w, v.z, o[k].z);
      o[k].w = fmaf(w, v.w, o[k].w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long long at = p.row_at(cut.x, cut.y, row);
  if (!p.check_row(at)) return;
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[2 * k] = ptx::pack_bf16x2(o[k].x * inv, o[k].y * inv);
    w[2 * k + 1] = ptx::pack_bf16x2(o[k].z * inv, o[k].w * inv);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + part * 16);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (part == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace fa
