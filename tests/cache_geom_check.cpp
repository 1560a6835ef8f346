// Index arithmetic of the paged e4m3 cache (fa_cache_geom.h) against its
// definitions: the scale rule, the checks of numbers that come from device
// memory, and the split of the attention's tiles over a grid.  Prints "ok" or
// the first mismatch.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "fa_cache_geom.h"

static int scales() {
  for (uint32_t bits = 0; bits < 0x7f80u; ++bits) {  // every finite bf16 >= 0
    const uint32_t w = bits << 16;
    float a;
    std::memcpy(&a, &w, 4);
    int e = fa::kCacheExpMin;
    while (e < fa::kCacheExpMax && (double)a > std::ldexp(448.0, e)) ++e;
    if (fa::cache_scale_exp(w) != e) {
      std::printf("scale of %g: %d != %d\n", a, fa::cache_scale_exp(w), e);
      return 1;
    }
  }
  return 0;
}

static int checks() {
  const int n[] = {INT_MIN, -1, 0, 1, 99, 100, 101, INT_MAX};
  for (int x : n) {
    bool bad = false;
    const int got = fa::cache_clamp(x, 100, bad);
    if (got < 0 || got > 100 || bad != (x < 0 || x > 100) || (!bad && got != x)) {
      std::printf("clamp %d: %d %d\n", x, got, bad);
      return 1;
    }
    bad = false;
    const int id = fa::cache_page(x, 100, bad);
    if (id < 0 || id >= 100 || bad != (x < 0 || x >= 100) || (!bad && id != x)) {
      std::printf("page %d: %d %d\n", x, id, bad);
      return 1;
    }
  }
  return 0;
}

// Every tile of every unit is walked once, by one CTA, in order; a CTA has at
// most two stretches that are not whole units, in different slots; tiles past
// a unit's last visible key are left out.
static int walk(const std::vector<int>& lens, const std::vector<int>& starts, int H, int g, int Nq, int RT, int causal,
                int max_len, int ctas) {
  const int B = (int)lens.size();
  fa::CacheRows rows{lens.data(), starts.empty() ? nullptr : starts.data(), B, H, g, Nq, g * Nq, RT,
                     (g * Nq + RT - 1) / RT, causal, max_len, fa::FastDiv::make((uint32_t)g)};
  struct Unit { int b, h, rt; long long t0; int nt; };
  std::vector<Unit> units;
  std::vector<long long> base(B + 1, 0);
  long long total = 0;
  for (int b = 0; b < B; ++b) {
    const long long len = lens[b] < 0 ? 0 : (lens[b] > max_len ? max_len : lens[b]);
    const long long first = starts.empty() ? len - Nq : starts[b];
    for (int h = 0; h < H; ++h)
      for (int rt = 0; rt < rows.row_tiles; ++rt) {
        long long keys = len;
        if (causal) {  // the largest count of keys that a row of the tile sees
          keys = 0;
          for (int r = rt * RT; r < (rt + 1) * RT && r < g * Nq; ++r) {
            const long long n = first + r / g + 1;
            if (n > keys) keys = n;
          }
          if (keys > len) keys = len;
        }
        const int nt = keys <= 0 ? 1 : (int)((keys + 127) / 128);
        units.push_back({b, h, rt, total, nt});
        total += nt;
      }
    base[b + 1] = total;
  }
  const int grid = fa::cache_active(total, ctas);
  long long seen = 0;
  size_t u = 0;
  for (int c = 0; c < grid; ++c) {
    const long long t0 = fa::cache_range_begin(total, grid, c), t1 = fa::cache_range_begin(total, grid, c + 1);
    if (t0 != seen || t1 <= t0) return std::printf("range %d\n", c), 1;
    int b0 = 0;
    while (b0 + 1 < B && base[b0 + 1] <= t0) ++b0;
    fa::CacheWalk w;
    w.start(rows, t0, t1, b0, base[b0]);
    fa::CacheSegment s;
    int used = 0;
    while (w.next(s)) {
      while (seen >= units[u].t0 + units[u].nt) ++u;
      const Unit& x = units[u];
      if (s.b != x.b || s.h != x.h || s.rt != x.rt || s.unit_t0 != x.t0 || s.total != x.nt || s.ntiles < 1 ||
          s.tile0 < 0 || s.tile0 + s.ntiles > s.total || s.unit_t0 + s.tile0 != seen)
        return std::printf("segment\n"), 1;
      // (a long stretch: its two ends only)
      for (long long t = seen; t < seen + s.ntiles; t += s.ntiles > 5000 ? s.ntiles - 1 : 1)
        if (fa::cache_range_owner(total, grid, t) != c) return std::printf("owner\n"), 1;
      seen += s.ntiles;
      if (s.ntiles < s.total) {
        const int slot = fa::cache_slot(c, t0, s.unit_t0) - 2 * c;
        if (slot != (s.unit_t0 > t0 ? 1 : 0) || (used >> slot) & 1) return std::printf("slot\n"), 1;
        used |= 1 << slot;
      }
    }
    if (seen != t1) return std::printf("end\n"), 1;
  }
  return seen == total ? 0 : (std::printf("total\n"), 1);
}

int main() {
  if (scales() || checks()) return 1;
  std::mt19937 r(7);
  for (int i = 0; i < 3000; ++i) {
    const int B = 1 + r() % 9, H = 1 + r() % 5, g = 1 + r() % 5, max_len = 1 + r() % 4000;
    const int Nq = r() % 3 ? 1 + r() % 8 : 1 + r() % 300, RT = 4 << r() % 7;
    std::vector<int> lens(B), starts;
    for (int& n : lens) n = r() % 10 == 0 ? (r() % 2 ? -5 : INT_MAX) : (int)(r() % (max_len + 1));
    if (r() % 3 == 0)
      for (int b = 0; b < B; ++b)
        starts.push_back(r() % 8 == 0 ? (r() % 2 ? INT_MIN : INT_MAX) : (int)(r() % (max_len + 1)) - 50);
    if (walk(lens, starts, H, g, Nq, RT, r() % 2, max_len, 1 + r() % 400)) return 1;
  }
  // 2^31 tokens a sequence, many heads: the tile count needs 64 bits
  if (fa::cache_range_begin(1LL << 45, 304, 304) != 1LL << 45) return std::printf("wide\n"), 1;
  if (walk({INT_MAX, 5, 0}, {}, 3, 2, 1, 4, 1, INT_MAX, 37)) return 1;
  std::printf("ok\n");
  return 0;
}
