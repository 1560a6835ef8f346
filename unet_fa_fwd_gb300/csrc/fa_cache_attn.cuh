// fa_cache_attn.cuh — attention of bf16 queries to the paged e4m3 cache:
//   t_ij = scale * q_i . k_j,  O_i = sum_j softmax_j(t_ij) v_j,
//   LSE_i = ln sum_j e^(t_ij),
// over the keys j < len[b], with `causal` j <= q_start[b] + i too.  Query head
// hq reads key head hq / (Hq / H).  A row that sees no key gives O = 0 and
// LSE = -inf.
//
// The rows of a key head's queries (its Hq / H query heads times Nq rows) are
// few here, so the products are taken the other way round: the 128 keys of a
// tile are the M side of the MMA and the rows the N side,
//   S^T [128 keys, rows] = K Q^T,   O^T [D channels, rows] = V^T P^T,
// and the codes go from HBM to the tensor cores as they are: TMA copies pages
// into shared memory and kind::f8f6f4 reads them as its A operand (K with the
// channels contiguous, V transposed).  No thread ever touches a code.
//
// What the e4m3 side cannot hold in one number is split over several N
// columns, each the rounding of what the one before left, scaled up by 16:
//   q = s (hi + lo / 16)               (s: a power of two a row; exact for
//     elements above 2^-14 of the row's largest, bf16 having 8 bits and e4m3
//     four; below, off by 2^-23 of it),
//   p = hi + mid / 16 + lo / 256       (12 bits, or 2^-25 of the row's largest p).
// The columns are extra work for the tensor cores only, which have time: the
// kernel is HBM bound.  Sums are fp32 throughout; each tile's O^T is added to
// fp32 registers (so a page's scale of V is applied outside the MMA, and O is
// rescaled there when the running maximum moves).
//
// A row must not get anything from keys that it does not see, but on the tensor
// cores 0 times NaN is NaN.  So in the tiles of which some row does not see
// every key (with causal, one or two a unit) a key whose V holds a NaN goes in
// as zeros; the rows that do see it are noted and give NaN at the end.
//
// Within a tile pages may differ in their scale of V: p carries the ratio of
// the page's scale to the tile's largest (a power of two <= 1), so the 2^-25
// above is relative to the largest V of the 128 tokens.  Where some row does not
// see every key, the largest is each row's own, of the pages that it sees.
//
// All units' tiles (fa_cache_geom.h) are cut into equal ranges, one per CTA, so
// ragged lengths and few heads balance alike; a unit cut between CTAs leaves
// fp32 partial results that fa_cache_merge_kernel joins in a fixed order.
//
// HBM bound: one query of 24 heads of 128 on 119056 keys takes 110 us, 6.7 TB/s;
// 64 sequences of up to 8192 tokens, 32 query heads to 8 key heads, 126 us,
// 6.5 TB/s, both with the join of the pieces.  Two CTAs an SM at D = 128 keep 96
// KB of codes in flight each (one CTA an SM: 130 and 160 us).
//
// Warps: 0-3 softmax (thread = key of the tile, and channel of O), 4 producer
// (page numbers, scales, TMA), 5 MMA issuer and owner of tensor memory.  Waits
// are bounded as in the forward kernel.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <climits>
#include <cstdint>

#include "fa_cache_geom.h"
#include "fa_cache_quant.cuh"
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kCacheStatusTimeout = 4;  // == FA_ERR_TIMEOUT
constexpr int kCacheMaxGrid = 1024;     // partial results are sized for this many CTAs
constexpr int kCacheThreads = 192;
constexpr int kCacheStagesMax = 8;

// A CTA's range of tiles.
struct CacheRange {
  long long total, t0, t1, base0;  // tiles in all; the range; first tile of entry b0
  int grid, b0;                    // CTAs with a range; the batch entry that holds t0
};

struct CacheAttnParams {
  CUtensorMap tm_k, tm_v;  // [num_pages * H][page][D] bytes
  CacheView c;
  CacheRows rows;
  const __nv_bfloat16* q;  // [B][Hq][Nq][D]
  __nv_bfloat16* out;      // [B][Hq][Nq][D]
  float* lse;              // [B][Hq][Nq]
  float* part_o;           // [2 * ctas][RT][D]
  float* part_ml;          // [2 * ctas][RT][2]: maximum (log2 domain), sum
  int4* cut;               // [ctas]: the unit that starts in a CTA's range and goes on past it
  int ctas;                // of the attention kernel's launch
  float scale_log2;
  int* status;
  int* debug_record;       // debug builds: first failed check
  unsigned long long timeout_ns;
  int inject_stall;        // test hook: CTA 0 withholds its second tile

  // Debug builds: an output row or a slot of partial results outside its array
  // is recorded and not accessed (release builds compile the checks to true).
  __device__ __forceinline__ bool check(bool ok, int id, long long a, long long b) const {
#ifdef FA_DEBUG
    if (!ok) {
      atomicCAS(status, 0, 5);  // FA_ERR_DEBUG_CHECK
      if (atomicCAS(&debug_record[0], 0, id) == 0) {
        debug_record[1] = (int)blockIdx.x;
        debug_record[2] = (int)threadIdx.x;
        debug_record[3] = (int)a;
        debug_record[4] = (int)b;
      }
      atomicAdd(&debug_record[7], 1);
    }
    return ok;
#else
    (void)ok; (void)id; (void)a; (void)b;
    return true;
#endif
  }
  __device__ __forceinline__ bool check_row(long long at) const {
    return check(at >= 0 && at < (long long)rows.B * rows.H * rows.g * rows.Nq, 6, at, rows.Nq);
  }
  __device__ __forceinline__ bool check_slot(long long slot) const {
    return check(slot >= 0 && slot < 2LL * ctas, 7, slot, ctas);
  }

  // cut[c]: batch entry (-1: no such unit), key head, row tile, and the CTA that
  // holds its last tile times two, plus one if its first piece is in slot 1.
  __device__ __forceinline__ void note_cut(const CacheSegment& s, const CacheRange& range) const {
    if (s.tile0 != 0 || s.ntiles == s.total) return;
    const int last = cache_range_owner(range.total, range.grid, s.unit_t0 + s.total - 1);
    cut[blockIdx.x] = make_int4(s.b, s.h, s.rt, 2 * last + (s.unit_t0 > range.t0 ? 1 : 0));
  }
  // Row of q, out and lse of row r of a key head.
  __device__ __forceinline__ long long row_at(int b, int h, int r) const {
    const int i = (int)rows.by_g.div((uint32_t)r);
    return (((long long)b * rows.H + h) * rows.g + (r - i * rows.g)) * rows.Nq + i;
  }
};

template <int D, int RT>
struct CacheCfg {
  static constexpr int TILE_BYTES = kCacheTile * D;      // 128 tokens of K or V
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int NS = (2 * RT + 15) / 16 * 16;     // N of S^T: hi and lo of each row
  static constexpr int NO = (3 * RT + 15) / 16 * 16;     // N of O^T: hi, mid, lo
  static constexpr uint32_t LAYOUT = D == 128 ? 2u : (D == 64 ? 4u : 6u);  // swizzle over a token's D bytes
  static constexpr int SBO = 8 * D;
  static constexpr int STAGES = D == 128 ? 3 : (D == 64 ? 3 : 4);
  static constexpr int SMEM_Q = (NS * D + 1023) / 1024 * 1024;
  static constexpr int SMEM_P = NO * kCacheTile;         // K-major: 128 keys of a column contiguous
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SMEM_Q + SMEM_P + 2048;
  static constexpr int COL_S = 0, COL_O = 2 * NS;
  static constexpr int TMEM_COLS = 2 * NS + NO <= 64 ? 64 : 128;
  static_assert(2 * NS + NO <= 128, "tensor memory");
  // CTAs that an SM is to hold (the compiler's register bound): two at D = 128,
  // by shared memory; the rows' registers decide below that.
  static constexpr int RESIDENT = D == 128 ? 2 : (RT == 4 ? 4 : (RT == 8 ? 3 : 2));
  static_assert(STAGES <= kCacheStagesMax, "ring barriers");
};

struct CacheBars {
  uint64_t kv_full[kCacheStagesMax], kv_empty[kCacheStagesMax];
  uint64_t s_full[2], p_ready, pv_done, q_ready, drain;
  CacheRange plan;
  uint32_t tmem_base;
  volatile int abort_flag;
  int wg_fail;
  uint32_t nan_rows;  // rows of the unit that see a key of which a NaN in V was taken out
  float ks[kCacheStagesMax][4];
  alignas(16) float vs[kCacheStagesMax][4];  // scales of a tile's 32-token groups
  alignas(16) float c[16];  // row: multiplier of the raw product, times the page's scale of K
  alignas(16) int lim[16];  // row: its last visible key
  float red[4][16];
  // A warp's copies: the largest scale of V that a row sees of the last tile, and
  // the ratio of the warp's page's to it.
  alignas(16) float row_vs[4][16], row_ratio[4][16];
};
static_assert(sizeof(CacheBars) <= 2048, "barrier space");

__device__ __forceinline__ uint64_t cache_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}

// Four e4m3 MMAs of one product, operand A stepping by AS and B by BS (16-byte
// units) each; the first overwrites the accumulator.  Issued by one elected
// lane of a converged warp.
template <int AS, int BS>
__device__ __forceinline__ void cache_mma4(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                           uint32_t idesc) {
  asm volatile(
      "{\n"
      ".reg .pred n, y, e;\n"
      ".reg .b32 el, al, bl;\n"
      ".reg .b64 da, db;\n"
      "elect.sync el|e, 0xffffffff;\n"
      "setp.ne.u32 n, 0, 0;\n"
      "setp.eq.u32 y, 0, 0;\n"
      "mov.b64 da, {%1, %2};\n"
      "mov.b64 db, {%3, %4};\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, n;\n"
      "add.u32 al, %1, %6;\n"
      "add.u32 bl, %3, %7;\n"
      "mov.b64 da, {al, %2};\n"
      "mov.b64 db, {bl, %4};\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, y;\n"
      "add.u32 al, %1, %8;\n"
      "add.u32 bl, %3, %9;\n"
      "mov.b64 da, {al, %2};\n"
      "mov.b64 db, {bl, %4};\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, y;\n"
      "add.u32 al, %1, %10;\n"
      "add.u32 bl, %3, %11;\n"
      "mov.b64 da, {al, %2};\n"
      "mov.b64 db, {bl, %4};\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, y;\n"
      "}\n"
      ::"r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(AS), "n"(BS), "n"(2 * AS), "n"(2 * BS),
        "n"(3 * AS), "n"(3 * BS)
      : "memory");
}

// Byte (row, col) of a K-major operand of W-byte rows, swizzled over W bytes.
template <int W>
__device__ __forceinline__ uint32_t cache_swizzle(int row, int col) {
  const int x = W == 128 ? (row & 7) : (W == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1));
  return (uint32_t)(row * W + ((((col >> 4) ^ x) << 4) | (col & 15)));
}

// The bytes of four e4m3 codes that are NaN (0x7f or 0xff): their highest bits.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t e4m3_nan(const uint4& v) {
  return e4m3_nan(v.x) | e4m3_nan(v.y) | e4m3_nan(v.z) | e4m3_nan(v.w);
}

// The rest of a wait whose phase has not come at the first look.  (Out of line:
// the kernels have a dozen waits, and the loop of the one for many rows is near
// the instruction cache's size.  With it inline 2048 rows on 16896 keys take 4 us
// more at D = 128 and 18 more at D = 32.)
static __device__ __noinline__ bool cache_wait_on(uint32_t a, uint32_t parity, volatile int* abort_flag, int* status,
                                                  unsigned long long timeout_ns) {
  bool ok = false;
  const uint64_t t0 = ptx::global_timer_ns();
  while (true) {
    if (ptx::mbar_try_wait_sleep(a, parity, 20000u)) {
      ok = true;
      break;
    }
    if (*abort_flag) break;
    if (ptx::global_timer_ns() - t0 > timeout_ns) {
      *abort_flag = 1;
      atomicCAS(status, 0, kCacheStatusTimeout);
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Bounded wait of a whole warp; false once the CTA is giving up.
template <typename Bars>
__device__ __forceinline__ bool cache_wait(uint64_t* bar, uint32_t parity, Bars* bars, const CacheAttnParams& p) {
  const uint32_t a = ptx::smem_u32(bar);
  if (__all_sync(0xffffffffu, ptx::mbar_try_wait(a, parity))) return true;
  return cache_wait_on(a, parity, &bars->abort_flag, p.status, p.timeout_ns);
}

// Wait (bounded) for copies or MMAs in flight before the CTA ends.
__device__ __forceinline__ void cache_drain(uint64_t* bar, uint32_t parity, const CacheAttnParams& p) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(ptx::smem_u32(bar), parity) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
  }
}

// OR of a predicate over the four softmax warps (also a barrier among them).
__device__ __forceinline__ bool cache_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 2, 128, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// The tile range of this CTA and the batch entry it starts in (one warp).
__device__ __forceinline__ void cache_plan(const CacheRows& rows, int ctas, int* status, uint32_t lane,
                                           CacheRange* out) {
  bool bad = false;
  auto tiles = [&](int b) -> long long {
    if (b >= rows.B) return 0;
    const int len = rows.len(b, bad);
    return rows.head_tiles(len, rows.first(b, len)) * rows.H;
  };
  long long total = 0;
  const long long mine = tiles((int)lane);  // of the first 32 entries, used again below
  for (int b = (int)lane; b < rows.B; b += 32) total += b < 32 ? mine : tiles(b);
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int grid = cache_active(total, ctas), c = (int)blockIdx.x;
  const long long q = cache_div(total, grid);
  const int left = (int)(total - q * grid);
  const long long t0 = c < grid ? q * c + left * c / grid : total;  // cache_range_begin
  const long long t1 = c < grid ? q * (c + 1) + left * (c + 1) / grid : total;
  long long base = 0, base0 = 0;
  int b0 = 0;
  for (int b = 0; b < rows.B && t0 < total; b += 32) {
    const int i = b + (int)lane;
    const long long n = b == 0 ? mine : tiles(i);
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if ((int)lane >= o) incl += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, i < rows.B && base + incl > t0);
    if (past) {
      const int src = __ffs(past) - 1;
      b0 = b + src;
      base0 = base + __shfl_sync(0xffffffffu, incl - n, src);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) atomicCAS(status, 0, kStatusIndex);
  if (lane == 0) *out = CacheRange{total, t0, t1, base0, grid, b0};
}

// The producer warp's view of a stretch's pages: each lane holds the number and
// scales of one of 32 pages.  (Fetching the next 32 ahead of their use measured
// no faster: the ring of tiles covers the two trips to memory.)
struct CachePages {
  int id;
  float ks, vs;

  // The 32 pages from tile j of the stretch on.
  __device__ __forceinline__ void fetch(const CacheAttnParams& p, const CacheSegment& s, int j, uint32_t lane) {
    const int ppt = kCacheTile / p.c.page;
    const int held = s.len == 0 ? 0 : (s.len - 1) / p.c.page + 1;  // pages with tokens
    const int idx = (s.tile0 + j) * ppt + (int)lane;
    bool bad = false;
    id = 0;
    ks = vs = 0.f;
    if (idx < held && idx < (s.tile0 + s.ntiles) * ppt) {
      id = cache_page(p.c.table[(long long)s.b * p.c.width + idx], p.c.num_pages, bad);
      const long long at = (long long)id * p.c.H + s.h;
      ks = p.c.scale[0][at];
      vs = p.c.scale[1][at];
    }
    if (bad) atomicCAS(p.status, 0, kStatusIndex);
  }
};

template <int D, int RT>
__global__ void __launch_bounds__(kCacheThreads, CacheCfg<D, RT>::RESIDENT) fa_cache_attn_kernel(const __grid_constant__ CacheAttnParams p) {
  using C = CacheCfg<D, RT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sRing = smem;
  uint8_t* sQ = sRing + C::STAGES * C::STAGE_BYTES;
  uint8_t* sP = sQ + C::SMEM_Q;
  CacheBars* bars = reinterpret_cast<CacheBars*>(sP + C::SMEM_P);
  const int warp = threadIdx.x / 32, tid = threadIdx.x;
  const uint32_t lane = threadIdx.x % 32;

  if (tid == 0) {
    if (p.cut) p.cut[blockIdx.x].x = -1;
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->kv_full[s]), 2);  // the copies; the scales
      ptx::mbar_init(ptx::smem_u32(&bars->kv_empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->s_full[0]), 1);
    ptx::mbar_init(ptx::smem_u32(&bars->s_full[1]), 1);
    ptx::mbar_init(ptx::smem_u32(&bars->p_ready), 128);
    ptx::mbar_init(ptx::smem_u32(&bars->q_ready), 128);
    ptx::mbar_init(ptx::smem_u32(&bars->pv_done), 1);
    ptx::mbar_init(ptx::smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    bars->wg_fail = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 4) cache_plan(p.rows, p.ctas, p.status, lane, &bars->plan);
  if (warp == 5) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  CacheWalk walk;
  walk.start(p.rows, bars->plan.t0, bars->plan.t1, bars->plan.b0, bars->plan.base0);
  CacheSegment sg;

  if (warp == 4) {
    // ------------------------------------------------------------ producer --
    if (lane == 0) {
      ptx::tma_prefetch_desc(&p.tm_k);
      ptx::tma_prefetch_desc(&p.tm_v);
    }
    const int page = p.c.page, ppt = kCacheTile / page;  // pages of a tile
    const int batch = 32 / ppt;                          // tiles whose pages the lanes hold
    uint32_t it = 0, skipped = 0xffffffffu;
    bool ok = true;
    CachePages pages;
    while (ok && walk.next(sg)) {
      const int npages = sg.len == 0 ? 0 : (sg.len - 1) / page + 1;
      for (int j = 0; j < sg.ntiles; ++j, ++it) {
        const int in_batch = j % batch;
        if (in_batch == 0) pages.fetch(p, sg, j, lane);
        const uint32_t s = it % C::STAGES;
        ok = cache_wait(&bars->kv_empty[s], ((it / C::STAGES) & 1) ^ 1, bars, p);
        if (!ok) break;
        if (p.inject_stall && blockIdx.x == 0 && it == 1) {  // nothing arrives: consumers time out
          skipped = it;
          continue;
        }
        const int my_id = __shfl_sync(0xffffffffu, pages.id, in_batch * ppt + (int)(lane % ppt));
        const int n = max(0, min(ppt, npages - (sg.tile0 + j) * ppt));  // pages of this tile that hold tokens
        const uint32_t full = ptx::smem_u32(&bars->kv_full[s]);
        if (lane == 0) ptx::mbar_arrive_expect_tx(full, (uint32_t)(2 * n * page * D));
        __syncwarp();
        if ((int)lane < n) {
          const uint32_t dst = ptx::smem_u32(sRing + s * C::STAGE_BYTES) + lane * page * D;
          const int at = my_id * p.c.H + sg.h;
          ptx::tma_load_3d(dst, &p.tm_k, full, 0, 0, at);
          ptx::tma_load_3d(dst + C::TILE_BYTES, &p.tm_v, full, 0, 0, at);
        }
        // The scales, for which the copies do not wait.
        const int group = in_batch * ppt + (int)(lane & 3) * 32 / page;  // page of this lane's 32 tokens
        const float my_ks = __shfl_sync(0xffffffffu, pages.ks, group), my_vs = __shfl_sync(0xffffffffu, pages.vs, group);
        if (lane < 4) {
          bars->ks[s][lane] = my_ks;
          bars->vs[s][lane] = my_vs;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full);
      }
    }
    if (!ok && lane == 0) {
      // Drain: every copy issued has landed once its stage's last phase is complete.
      for (int s = 0; s < C::STAGES; ++s) {
        uint32_t n = it > (uint32_t)s ? (it - 1 - s) / C::STAGES + 1 : 0;
        if (skipped < it && skipped % C::STAGES == (uint32_t)s) --n;
        if (n) cache_drain(&bars->kv_full[s], (n - 1) & 1, p);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // ----------------------------------------------------------------- MMA --
    constexpr uint32_t kIdesc = (1u << 4) | (8u << 24);  // e4m3 x e4m3, fp32 sums, M = 128
    constexpr uint32_t IDESC_S = kIdesc | ((uint32_t)(C::NS >> 3) << 17);
    constexpr uint32_t IDESC_O = kIdesc | ((uint32_t)(C::NO >> 3) << 17) | (1u << 15);  // A = V, transposed
    const uint64_t dk = cache_desc(ptx::smem_u32(sRing), 16, C::SBO, C::LAYOUT);
    // V as the transposed A: 8 tokens x D channels per swizzle atom.  M is 128
    // whatever D is: with a leading offset of 0 the channels repeat (their
    // lanes of O^T are not read).
    const uint64_t dv = cache_desc(ptx::smem_u32(sRing) + C::TILE_BYTES, 0, C::SBO, C::LAYOUT);
    const uint64_t dq = cache_desc(ptx::smem_u32(sQ), 16, C::SBO, C::LAYOUT);
    const uint64_t dp = cache_desc(ptx::smem_u32(sP), 16, 1024, 2u);
    auto issue_s = [&](uint32_t stage, uint32_t buf) {
      const uint32_t a = (uint32_t)dk + stage * (C::STAGE_BYTES >> 4), d = tmem + C::COL_S + buf * C::NS;
      if constexpr (D == 128)
        ptx::mma_ss_f8_x4_el<2, 4, 6>(d, a, (uint32_t)(dk >> 32), (uint32_t)dq, (uint32_t)(dq >> 32), IDESC_S, 0);
      else if constexpr (D == 64)
        ptx::mma_ss_f8_x2_el<2>(d, a, (uint32_t)(dk >> 32), (uint32_t)dq, (uint32_t)(dq >> 32), IDESC_S, 0);
      else
        ptx::mma_ss_f8_x1_el(d, a, (uint32_t)(dk >> 32), (uint32_t)dq, (uint32_t)(dq >> 32), IDESC_S, 0);
    };
    auto issue_o = [&](uint32_t stage) {
      const uint32_t a = (uint32_t)dv + stage * (C::STAGE_BYTES >> 4);
      cache_mma4<(32 * D >> 4), 2>(tmem + C::COL_O, a, (uint32_t)(dv >> 32), (uint32_t)dp, (uint32_t)(dp >> 32),
                                   IDESC_O);  // 32 keys each
    };
    uint32_t it = 0, seg = 0;  // tiles and segments so far
    bool ok = true;
    // P of tile n is ready: its product, which also frees its stage.
    auto finish_tile = [&](uint32_t n) -> bool {
      if (!cache_wait(&bars->p_ready, n & 1, bars, p)) return false;
      ptx::tc_fence_after_sync();
      issue_o(n % C::STAGES);
      ptx::mma_commit_el(ptx::smem_u32(&bars->kv_empty[n % C::STAGES]));
      ptx::mma_commit_el(ptx::smem_u32(&bars->pv_done));
      return true;
    };
    while (ok && walk.next(sg)) {
      ok = cache_wait(&bars->q_ready, seg & 1, bars, p);
      ++seg;
      if (!ok) break;
      for (int j = 0; j < sg.ntiles; ++j, ++it) {
        ok = cache_wait(&bars->kv_full[it % C::STAGES], (it / C::STAGES) & 1, bars, p);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        // The other S buffer was read before P of tile it - 2 was released.
        issue_s(it % C::STAGES, it & 1);
        ptx::mma_commit_el(ptx::smem_u32(&bars->s_full[it & 1]));
        if (j > 0) ok = finish_tile(it - 1);
        if (!ok) break;
      }
      if (ok) ok = finish_tile(it - 1);
    }
    ptx::mma_commit_el(ptx::smem_u32(&bars->drain));
    cache_drain(&bars->drain, 0, p);
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax --
    // p is kept between 2^-25 and 2^8.75 (e4m3's largest is 448) by a running
    // reference m: on the first tile, and whenever a score passes m + 8.75, m
    // becomes the row's maximum less 7.
    constexpr float kTop = 7.f, kLimit = 8.75f, kNone = -3.402823466e38f;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + lane_base + C::COL_S, tO = tmem + lane_base + C::COL_O;
    // Byte of key tid in column n of P (128-byte rows, swizzled over them).
    auto p_byte = [&](int n) -> uint8_t& { return sP[(tid ^ ((n & 7) << 4)) + n * kCacheTile]; };
    uint32_t it = 0;
    uint32_t stage = 0, stage_phase = 0;
    bool fail = false;
    while (walk.next(sg)) {
      const int row0 = sg.rt * RT, rows = min(RT, p.rows.R - row0);
      // Q: each warp splits rows warp, warp + 4, ... into hi and lo columns.
      {
        constexpr int PER = D / 32;
        for (int r = warp; r < RT; r += 4) {
          float x[PER];
          uint32_t amax = 0;
          const bool in = r < rows;
          if (in) {
            const __nv_bfloat16* src = p.q + p.row_at(sg.b, sg.h, row0 + r) * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
              x[e] = __bfloat162float(src[e]);
              amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
            }
          } else {
#pragma unroll
            for (int e = 0; e < PER; ++e) x[e] = 0.f;
          }
          amax = __reduce_max_sync(0xffffffffu, amax);
          // 2^e: the least power of two with amax <= 448 * 2^e (not below 2^-100)
          const int e2 = max((int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
          const float inv = __int_as_float((127 - e2) << 23);
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const float v = x[e] * inv;
            const uint32_t hi = e4m3x2_bits(v, 0.f);
            const float left = (v - e4m3x2_value(hi).x) * 16.f;
            const uint32_t lo = e4m3x2_bits(left, 0.f);
            sQ[cache_swizzle<D>(2 * r, (int)lane * PER + e)] = (uint8_t)hi;
            sQ[cache_swizzle<D>(2 * r + 1, (int)lane * PER + e)] = (uint8_t)lo;
          }
          if (lane == 0) {
            // a row that holds a number that is not finite gives NaN
            bars->c[r] = amax >= 0x7f800000u ? __int_as_float(0x7fc00000)
                                             : __int_as_float((e2 + 127) << 23) * p.scale_log2;
            bars->lim[r] = p.rows.limit(sg.len, sg.first, (int)p.rows.by_g.div((uint32_t)(row0 + r)));
          }
        }
        if (tid == 0) bars->nan_rows = 0;
        // (limits grow with the row: the first row's is the least)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        ptx::mbar_arrive(ptx::smem_u32(&bars->q_ready));
        ptx::named_barrier_sync(3, 128);
      }
      const int least = bars->lim[0];
      float m[RT], l[RT], o[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        m[r] = kNone;
        l[r] = o[r] = 0.f;
      }
      float v_scale = 0.f;   // of the tile whose O^T is still to be added
      bool pending = false;
      auto tile_unit = [&](int) { return v_scale; };
      // Adds the last tile's O^T, in units of the current m and of unit(r), to o.
      auto take_o = [&](auto unit) {
        if (!cache_wait(&bars->pv_done, (it - 1) & 1, bars, p)) fail = true;
        ptx::tc_fence_after_sync();
        [[maybe_unused]] uint32_t r0[16];
        if constexpr (RT == 4) {
          ptx::tmem_ld32x32b_x16(tO, r0);
#pragma unroll
          for (int r = 0; r < RT; ++r)
            o[r] += unit(r) * (__uint_as_float(r0[3 * r]) + 0.0625f * __uint_as_float(r0[3 * r + 1]) +
                               0.00390625f * __uint_as_float(r0[3 * r + 2]));
        } else {
          uint32_t r1[32];
          float f[48];
          ptx::tmem_ld32x32b_x32(tO, r1);
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r1[i]);
          if constexpr (RT == 16) {
            ptx::tmem_ld32x32b_x16(tO + 32, r0);
#pragma unroll
            for (int i = 0; i < 16; ++i) f[32 + i] = __uint_as_float(r0[i]);
          }
#pragma unroll
          for (int r = 0; r < RT; ++r)
            o[r] += unit(r) * (f[3 * r] + 0.0625f * f[3 * r + 1] + 0.00390625f * f[3 * r + 2]);
        }
        pending = false;
      };

      bool stop = false;
      for (int j = 0; j < sg.ntiles; ++j) {
        const int key0 = (sg.tile0 + j) * kCacheTile;
        if (!cache_wait(&bars->kv_full[stage], stage_phase, bars, p)) fail = true;
        // This warp's 32 keys are in one page.
        const float ks = bars->ks[stage][warp], vs = bars->vs[stage][warp];
        const float4 v4 = *reinterpret_cast<const float4*>(bars->vs[stage]);
        const float vt = fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w));  // (0 where a page has no tokens)
        if (!cache_wait(&bars->s_full[it & 1], (it >> 1) & 1, bars, p)) fail = true;
        ptx::tc_fence_after_sync();
        float t[RT];
        {
          auto scores = [&](const uint32_t* sv) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
              t[r] = fmaf(__uint_as_float(sv[2 * r + 1]), 0.0625f, __uint_as_float(sv[2 * r])) * (bars->c[r] * ks);
          };
          if constexpr (C::NS == 16) {
            uint32_t sv[16];
            ptx::tmem_ld32x32b_x16(tS + (it & 1) * C::NS, sv);
            scores(sv);
          } else {
            uint32_t sv[32];
            ptx::tmem_ld32x32b_x32(tS + (it & 1) * C::NS, sv);
            scores(sv);
          }
        }
        if (key0 + kCacheTile - 1 > least) {  // some row does not see the whole tile
#pragma unroll
          for (int r = 0; r < RT; ++r) t[r] = key0 + tid <= bars->lim[r] ? t[r] : -INFINITY;
        }
        float above = -INFINITY;
#pragma unroll
        for (int r = 0; r < RT; ++r) above = fmaxf(above, t[r] - m[r]);
        const bool need = above > kLimit;
        if (cache_any(need || fail)) {
          if (pending) take_o(tile_unit);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            float x = t[r];
#pragma unroll
            for (int k = 16; k; k >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
            if (lane == 0) bars->red[warp][r] = x;
          }
          if (fail) bars->wg_fail = 1;
          ptx::named_barrier_sync(3, 128);
          if (bars->wg_fail) {
            stop = true;
            break;
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const float x = fmaxf(fmaxf(bars->red[0][r], bars->red[1][r]), fmaxf(bars->red[2][r], bars->red[3][r]));
            if (x - m[r] > kLimit) {
              const float alpha = ptx::ex2(m[r] - (x - kTop));
              m[r] = x - kTop;
              l[r] *= alpha;
              o[r] *= alpha;
            }
          }
        }
        const int held = sg.len - key0;
        const bool mixed = least < key0 + min(held, kCacheTile) - 1;  // some row does not see every key
        // vs / vt, a power of two (below, for each row's own vt)
        auto exponent = [&](float unit) { return max((__float_as_int(vs) >> 23) - (__float_as_int(unit) >> 23), -100); };
        const float ratio = __int_as_float(((mixed ? 0 : exponent(vt)) + 127) << 23);
        float2 pr[RT / 2];
#pragma unroll
        for (int r = 0; r < RT; r += 2) {
          const float2 e = make_float2(ptx::ex2(t[r] - m[r]), ptx::ex2(t[r + 1] - m[r + 1]));
          l[r] += e.x;
          l[r + 1] += e.y;
          pr[r / 2] = __fmul2_rn(e, make_float2(ratio, ratio));
        }
        if (pending) take_o(tile_unit);  // P and O^T are free once the last tile's product is done
        uint8_t* sV = sRing + stage * C::STAGE_BYTES + C::TILE_BYTES;
        if (mixed) {
          if ((int)lane < RT) {
            const int groups = (bars->lim[lane] - key0) >> 5;  // the last group of 32 keys that the row sees
            float x = groups >= 0 ? v4.x : 0.f;
            if (groups >= 1) x = fmaxf(x, v4.y);
            if (groups >= 2) x = fmaxf(x, v4.z);
            if (groups >= 3) x = fmaxf(x, v4.w);
            bars->row_vs[warp][lane] = x;
            bars->row_ratio[warp][lane] = __int_as_float((min(exponent(x), 0) + 127) << 23);
          }
          __syncwarp();
#pragma unroll
          for (int r = 0; r < RT; r += 2)
            pr[r / 2] = __fmul2_rn(pr[r / 2], *reinterpret_cast<const float2*>(&bars->row_ratio[warp][r]));
          // NaN in V: this thread's key.  (Rolled up: cold code costs its instruction misses.)
          uint32_t nan = 0;
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i)
            nan |= e4m3_nan(*reinterpret_cast<const uint4*>(sV + tid * D + (i + tid) % (D / 16) * 16));
          if (nan) {
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) *reinterpret_cast<uint4*>(sV + tid * D + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            uint32_t see = 0;
#pragma unroll 1
            for (int r = 0; r < RT; ++r) see |= (key0 + tid <= bars->lim[r] ? 1u : 0u) << r;
            atomicOr(&bars->nan_rows, see);
          }
        }
        const float2 up = make_float2(16.f, 16.f), down = make_float2(-16.f, -16.f);
#pragma unroll
        for (int r = 0; r < RT; r += 2) {
          const uint32_t hi = e4m3x2_bits(pr[r / 2].x, pr[r / 2].y);
          const float2 a = __ffma2_rn(e4m3x2_value(hi), down, __fmul2_rn(pr[r / 2], up));
          const uint32_t mid = e4m3x2_bits(a.x, a.y);
          const float2 c = __ffma2_rn(e4m3x2_value(mid), down, __fmul2_rn(a, up));
          const uint32_t lo = e4m3x2_bits(c.x, c.y);
          p_byte(3 * r) = (uint8_t)hi;
          p_byte(3 * r + 1) = (uint8_t)mid;
          p_byte(3 * r + 2) = (uint8_t)lo;
          p_byte(3 * r + 3) = (uint8_t)(hi >> 8);
          p_byte(3 * r + 4) = (uint8_t)(mid >> 8);
          p_byte(3 * r + 5) = (uint8_t)(lo >> 8);
        }
        // Rows of V past the length may hold anything, NaN among it: zero them.
        if (held < kCacheTile) {
          for (int i = max(held, 0) * D + tid * 16; i < C::TILE_BYTES; i += 128 * 16)
            *reinterpret_cast<uint4*>(sV + i) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        ptx::tc_fence_before_sync();
        ptx::mbar_arrive(ptx::smem_u32(&bars->p_ready));
        v_scale = vt;
        pending = true;
        ++it;
        if (++stage == (uint32_t)C::STAGES) {
          stage = 0;
          stage_phase ^= 1u;
        }
        // (At once, so that the tiles that all rows see whole have one unit.  16 rows
        // at D = 64, where an instruction more a tile shows: 146 us for 64 sequences
        // of 8192 keys and 8 heads, 148 with a choice of units in every tile.)
        if (mixed) take_o([&](int r) { return bars->row_vs[warp][r]; });
      }
      if (!stop && pending) take_o(tile_unit);
      if (cache_any(fail || stop)) break;

      if (const uint32_t nan = bars->nan_rows) {
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r] = (nan >> r) & 1u ? __int_as_float(0x7fc00000) : o[r];
      }
      // The row's sum over the 128 threads.
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float x = l[r];
#pragma unroll
        for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        if (lane == 0) bars->red[warp][r] = x;
      }
      ptx::named_barrier_sync(3, 128);
#pragma unroll
      for (int r = 0; r < RT; ++r) l[r] = bars->red[0][r] + bars->red[1][r] + bars->red[2][r] + bars->red[3][r];
      if (sg.ntiles == sg.total) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (r >= rows) break;
          const long long at = p.row_at(sg.b, sg.h, row0 + r);
          if (!p.check_row(at)) continue;
          if (tid < D) p.out[at * D + tid] = __float2bfloat16_rn(l[r] == 0.f ? 0.f : o[r] / l[r]);
          if (tid == r) p.lse[at] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * 0.6931471805599453f;
        }
      } else {
        const long long slot = cache_slot((int)blockIdx.x, bars->plan.t0, sg.unit_t0);
        if (tid == 0) p.note_cut(sg, bars->plan);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (r >= rows || !p.check_slot(slot)) break;
          if (tid < D) p.part_o[(slot * RT + r) * D + tid] = o[r];
          if (tid == r) {
            p.part_ml[(slot * RT + r) * 2] = m[r];
            p.part_ml[(slot * RT + r) * 2 + 1] = l[r];
          }
        }
      }
    }
    ptx::tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == 5) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the partial results of the units that were cut between CTAs: for each
// row, over its pieces s in order, m = max m_s, l = sum 2^(m_s - m) l_s,
// O = sum 2^(m_s - m) O_s / l.  One block for each row of the unit that is cut
// at the end of a CTA's range: its threads first take a piece each (maxima,
// sums, weights), then four channels of every G-th piece.
template <int D, int RT>
__global__ void __launch_bounds__(128) fa_cache_merge_kernel(const __grid_constant__ CacheAttnParams p) {
  constexpr int LANES = D / 4, G = 128 / LANES;  // threads of a row of O; pieces read at a time
  __shared__ float weight[kCacheMaxGrid], red[4], part[G][D];
  const int tid = threadIdx.x;
  const int c0 = blockIdx.x / RT, in_tile = blockIdx.x - c0 * RT;
  // Launched while the attention kernel still runs (programmatic dependent
  // launch): every block waits for it, those with nothing to join too, so that
  // this kernel's end stands for both.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 cut = p.cut[c0];
  const int r = cut.z * RT + in_tile, c1 = cut.w >> 1;
  if (cut.x < 0 || r >= p.rows.R) return;
  // The unit is the first stretch of every CTA but c0.
  auto slot = [&](int c) { return (2LL * c + (c == c0 ? (cut.w & 1) : 0)) * RT + in_tile; };
  const int pieces = c1 - c0 + 1;
  if (!p.check_slot(2LL * c1)) return;
  auto block = [&](float x, bool max) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      x = max ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = x;
    __syncthreads();
    return max ? fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])) : (red[0] + red[1]) + (red[2] + red[3]);
  };
  float m = -INFINITY, l = 0.f;
  for (int i = tid; i < pieces; i += 128) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot(c0 + i) * 2);
    if (ml.y != 0.f) m = fmaxf(m, ml.x);  // a piece with no visible key has sum 0
  }
  m = block(m, true);
  for (int i = tid; i < pieces; i += 128) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot(c0 + i) * 2);
    const float w = ml.y != 0.f ? ptx::ex2(ml.x - m) : 0.f;
    weight[i] = w;
    l = fmaf(w, ml.y, l);
  }
  l = block(l, false);  // (its barriers also publish the weights)
  const int lane = tid % LANES, g = tid / LANES;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = g; i < pieces; i += G) {
    const float w = weight[i];  // (of a piece with no visible key: 0, and its O is 0)
    const float4 x = *reinterpret_cast<const float4*>(p.part_o + slot(c0 + i) * D + lane * 4);
    o.x = fmaf(w, x.x, o.x);
    o.y = fmaf(w, x.y, o.y);
    o.z = fmaf(w, x.z, o.z);
    o.w = fmaf(w, x.w, o.w);
  }
  *reinterpret_cast<float4*>(&part[g][lane * 4]) = o;
  __syncthreads();
  const long long at = p.row_at(cut.x, cut.y, r);
  if (!p.check_row(at)) return;
  if (tid < D) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) x += part[i][tid];
    p.out[at * D + tid] = __float2bfloat16_rn(l == 0.f ? 0.f : x / l);
  }
  if (tid == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace fa
