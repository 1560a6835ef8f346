// fa_cache_geom.h — index arithmetic of the paged e4m3 cache, shared by the
// kernels and a host-side check: the power-of-two scale rule, the bounds
// checks of page numbers, lengths and positions that come from device memory,
// and the split of the cached attention's key tiles over the grid.
#pragma once

#include <cstdint>

#include "fa_fastdiv.h"  // FA_HD

namespace fa {

// Scale exponents: 2^-117 keeps code * scale a normal bf16 number down to
// e4m3's least value 2^-9; 448 * 2^119 is finite in bf16.
constexpr int kCacheExpMin = -117, kCacheExpMax = 119;

// Least e in [kCacheExpMin, kCacheExpMax] with amax <= 448 * 2^e, from the
// bits of a finite amax >= 0 (448 = 1.75 * 2^8, so the mantissa decides
// between exponent - 8 and exponent - 7).
FA_HD int cache_scale_exp(uint32_t amax_bits) {
  const int x = (int)((amax_bits >> 23) & 255u) - 127;  // subnormals: -127, clamped below
  const int e = x - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kCacheExpMin ? kCacheExpMin : (e > kCacheExpMax ? kCacheExpMax : e);
}

// A length (or position) read from device memory, kept inside [0, most].
FA_HD int cache_clamp(int n, int most, bool& bad) {
  if (n < 0) {
    bad = true;
    return 0;
  }
  if (n > most) {
    bad = true;
    return most;
  }
  return n;
}

// A page number from the table: one outside the cache is read as page 0.
FA_HD int cache_page(int id, int num_pages, bool& bad) {
  if (id < 0 || id >= num_pages) {
    bad = true;
    return 0;
  }
  return id;
}

// ---- the attention's work ----
// The rows of a key head are its g = Hq / H query heads' Nq rows each, taken
// position by position (row r: position r / g of query head r % g), so that a
// tile of RT rows covers few positions.  A unit is one (batch entry, key head,
// row tile); it has the 128-key tiles that some row of it sees, at least one
// (so that an empty row still gets its outputs written).  The tiles of all
// units in order are cut into equal ranges, one per CTA; no range is empty, so
// with fewer tiles than CTAs the last CTAs have none.
constexpr int kCacheTile = 128;

FA_HD int cache_tiles(int len) { return len <= 0 ? 1 : (len - 1) / kCacheTile + 1; }

// Lengths and positions may hold anything: lengths are kept inside
// [0, max_len], positions are added in 64 bits.
struct CacheRows {
  const int* lens;     // [B]
  const int* q_start;  // [B] or nullptr: len - Nq
  int B, H, g, Nq, R, RT, row_tiles, causal, max_len;
  FastDiv by_g;        // division by g

  FA_HD int len(int b, bool& bad) const { return cache_clamp(lens[b], max_len, bad); }
  FA_HD long long first(int b, int len) const { return q_start ? (long long)q_start[b] : (long long)len - Nq; }
  // Last key that the row at position i sees, -1 for none.
  FA_HD int limit(int len, long long first, int i) const {
    long long last = len - 1;
    if (causal && first + i < last) last = first + i;
    return last < -1 ? -1 : (int)last;
  }
  // Tiles of row tile rt of a batch entry of this length and first position.
  FA_HD int tiles(int len, long long first, int rt) const {
    if (!causal) return cache_tiles(len);
    const int rows = (rt + 1) * (long long)RT < R ? (rt + 1) * RT : R;
    return cache_tiles(limit(len, first, (int)by_g.div((uint32_t)(rows - 1))) + 1);
  }
  // Tiles of all row tiles of a key head.
  FA_HD long long head_tiles(int len, long long first) const {
    if (!causal || row_tiles == 1) return (long long)tiles(len, first, 0) * row_tiles;
    long long n = 0;
    for (int rt = 0; rt < row_tiles; ++rt) n += tiles(len, first, rt);
    return n;
  }
};

FA_HD int cache_active(long long total, int ctas) { return total < ctas ? (int)total : ctas; }

// a / b for a >= 0, b > 0 (a 64-bit division costs a kernel's start some half a
// microsecond, so it is taken only where it is needed).
FA_HD long long cache_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// `grid` below is cache_active(total, ctas): at most a few thousand.
FA_HD long long cache_range_begin(long long total, int grid, int cta) {
  const long long q = cache_div(total, grid);
  return q * cta + (int)(total - q * grid) * cta / grid;  // floor(total * cta / grid)
}

// The CTA whose range holds tile t.
FA_HD int cache_range_owner(long long total, int grid, long long t) {
  int c = (int)((double)t * grid / (double)total);
  if (c >= grid) c = grid - 1;
  while (c > 0 && cache_range_begin(total, grid, c) > t) --c;
  while (c + 1 < grid && cache_range_begin(total, grid, c + 1) <= t) ++c;
  return c;
}

// One stretch of a unit's tiles inside a CTA's range.
struct CacheSegment {
  int b, h, rt;        // the unit
  int len;             // its batch entry's checked length
  long long first;     // position of the first query row
  long long unit_t0;   // the unit's first tile
  int tile0, ntiles;   // this stretch
  int total;           // tiles of the unit
};

// Walks a CTA's range of tiles.
struct CacheWalk {
  const CacheRows* r;
  long long t, end, base;    // next tile, end of the range, first tile of the current unit
  long long first;
  int b, h, rt, len, nt;

  // `b0`, `base0`: the batch entry that holds tile t0, and its first tile.
  FA_HD void start(const CacheRows& rows, long long t0, long long t1, int b0, long long base0) {
    r = &rows;
    t = t0;
    end = t1;
    base = base0;
    b = b0;
    h = rt = 0;
    load();
    if (t >= end) return;
    const long long per_head = r->head_tiles(len, first);
    h = (int)cache_div(t - base, per_head);
    base += h * per_head;
    unit();
    while (t >= base + nt) {
      base += nt;
      ++rt;
      unit();
    }
  }
  FA_HD void load() {
    bool bad = false;
    len = b < r->B ? r->len(b, bad) : 0;
    first = b < r->B ? r->first(b, len) : 0;
  }
  FA_HD void unit() { nt = r->tiles(len, first, rt); }
  FA_HD bool next(CacheSegment& s) {
    if (t >= end) return false;
    if (t >= base + nt) {  // the range goes on with the next unit
      base += nt;
      if (++rt == r->row_tiles) {
        rt = 0;
        if (++h == r->H) {
          h = 0;
          ++b;
          load();
        }
      }
      unit();
    }
    s.b = b;
    s.h = h;
    s.rt = rt;
    s.len = len;
    s.first = first;
    s.unit_t0 = base;
    s.tile0 = (int)(t - base);
    s.total = nt;
    const long long left = end - t;
    s.ntiles = nt - s.tile0 < left ? nt - s.tile0 : (int)left;
    t += s.ntiles;
    return true;
  }
};

// ---- the rings of the kernel for many rows ----
// Tile n of a CTA's range uses stage n % chunk_k_stages of the K and V codes,
// stage n % kChunkVStages of V in f16 and slot n % kChunkMeta of the scales.
constexpr int kChunkRows = 256;    // rows of a unit: two row tiles of 128 (one of them with PAIR)
constexpr int kChunkVStages = 2;
constexpr int kChunkMeta = 16;     // more than the pipeline's depth
constexpr int chunk_k_stages(int D, bool pair) { return pair || D == 128 ? 3 : 6; }

// Partial results: a CTA has at most two stretches that are not whole units,
// its first (slot 0) and its last (slot 1 when the unit starts inside the range).
FA_HD int cache_slot(int c, long long range_t0, long long unit_t0) { return 2 * c + (unit_t0 > range_t0 ? 1 : 0); }

}  // namespace fa
