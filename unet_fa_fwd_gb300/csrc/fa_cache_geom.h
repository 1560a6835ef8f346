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
// A unit is one (batch entry, key head, row tile); it has as many 128-key
// tiles as its batch entry's length (at least one, so that an empty sequence
// still gets its outputs written).  The tiles of all units in order are cut
// into equal ranges, one per CTA; no range is empty, so with fewer tiles than
// CTAs the last CTAs have none.
constexpr int kCacheTile = 128;

FA_HD int cache_tiles(int len) { return len <= 0 ? 1 : (len - 1) / kCacheTile + 1; }

FA_HD int cache_active(long long total, int ctas) { return total < ctas ? (int)total : ctas; }

// `grid` below is cache_active(total, ctas).
FA_HD long long cache_range_begin(long long total, int grid, int cta) {
  return total / grid * cta + total % grid * cta / grid;  // floor(total * cta / grid)
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
  int b, unit;         // batch entry; (key head, row tile) within it
  int len;             // its checked length
  int tile0, ntiles;   // this stretch
  int total;           // tiles of the unit
};

// Walks a CTA's range of tiles.  `lens` may hold anything; lengths are kept
// inside [0, max_len].
struct CacheWalk {
  const int* lens;
  int B, units, max_len;     // batch entries; units per entry
  long long t, end, base;    // next tile, end of the range, first tile of entry b
  int b, len, nt;

  // `b0`, `base0`: the batch entry that holds tile t0, and its first tile.
  FA_HD void start(const int* l, int B_, int units_, int max_len_, long long t0, long long t1, int b0,
                   long long base0) {
    lens = l;
    B = B_;
    units = units_;
    max_len = max_len_;
    t = t0;
    end = t1;
    base = base0;
    b = b0;
    load();
  }
  FA_HD void load() {
    bool bad = false;
    len = b < B ? cache_clamp(lens[b], max_len, bad) : 0;
    nt = cache_tiles(len);
  }
  FA_HD bool next(CacheSegment& s) {
    if (t >= end) return false;
    while (t >= base + (long long)nt * units) {
      base += (long long)nt * units;
      ++b;
      load();
    }
    const long long rel = t - base;
    s.b = b;
    s.unit = (int)(rel / nt);
    s.tile0 = (int)(rel - (long long)s.unit * nt);
    s.len = len;
    s.total = nt;
    const long long left = end - t;
    s.ntiles = nt - s.tile0 < left ? nt - s.tile0 : (int)left;
    t += s.ntiles;
    return true;
  }
};

// Partial results: a CTA has at most two stretches that are not whole units,
// its first (slot 0) and its last (slot 1).  The slot that CTA c uses for the
// unit whose first tile is unit_t0:
FA_HD int cache_slot(long long total, int grid, int c, long long unit_t0) {
  return 2 * c + (unit_t0 > cache_range_begin(total, grid, c) ? 1 : 0);
}

}  // namespace fa
