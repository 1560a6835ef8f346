// fa_bwd_geom.h — which work each CTA of the attention's gradient kernels does.
// Host and device; checked on the CPU against a plain enumeration.
//
// A unit is 128 rows of one side (keys for dK and dV, queries for dQ) of one
// head; it walks the other side's 128-row tiles, one iteration each (for keys
// that several query heads share, the tiles of all of them).  Units are dealt
// whole to the persistent CTAs in rounds, in snake order; those that would not
// fill a last round evenly are cut into ranges of iterations that level the
// CTAs' totals.  A unit that is cut leaves partial sums, which a second kernel
// joins in a fixed order.
#pragma once

#include <cstdint>

#include "fa_fastdiv.h"

namespace fa {

constexpr int kBwdMaxCtas = 192;  // CTAs (one per SM) that the cuts are sized for

// The units of one kernel.
struct BwdUnits {
  int heads;   // B x heads of the unit's side
  int tiles;   // 128-row tiles of a head
  int other;   // 128-row tiles of the other side
  int group;   // heads of the other side that a unit walks (shared key heads; 1 for dQ)
  int causal;  // query i sees keys 0 .. i
  int rows_q;  // the unit's rows are queries (dQ), else keys
  int spread;  // units of equal weight next to each other (heads inner), else head by head
  FastDiv div_heads, div_tiles;

  int count() const { return heads * tiles; }
  // Causal: heaviest units first (key tiles ascending, query tiles descending).
  FA_HD void locate(int u, int& head, int& tile) const {
    int level;
    if (spread) {
      level = (int)div_heads.div((uint32_t)u);
      head = u - level * heads;
    } else {
      head = (int)div_tiles.div((uint32_t)u);
      level = u - head * tiles;
    }
    tile = causal && rows_q ? tiles - 1 - level : level;
  }
  // Tiles of the other side, of one head, that the unit's tile meets: first .. first + n - 1.
  FA_HD void range(int tile, int& first, int& n) const {
    first = 0;
    n = other;
    if (causal) {
      if (rows_q) {
        n = tile + 1 < other ? tile + 1 : other;
      } else {
        first = tile;
        n = other > tile ? other - tile : 0;
      }
    }
  }
  // Iterations of a unit (0: no query sees its keys; it still writes its zeros).
  FA_HD int iterations(int tile) const {
    int first, n;
    range(tile, first, n);
    return n * group;
  }
  // What a unit counts for in the plan: its iterations, one at least.
  FA_HD int weight(int u) const {
    int head, tile;
    locate(u, head, tile);
    const int n = iterations(tile);
    return n > 0 ? n : 1;
  }
};

// A place between iterations: before iteration `it` of unit `unit`.
struct BwdCut {
  int unit, it;
};

struct BwdPlan {
  BwdUnits units;
  int ctas;   // CTAs of the launch
  int whole;  // units [0, whole) are dealt whole; the others are cut at cut[1 .. ctas - 1]
  int joins;  // cuts that fall inside a unit
  BwdCut cut[kBwdMaxCtas + 1];
};

// One stretch of a CTA's work.
struct BwdPiece {
  int head, tile;
  int it0, it1;  // iterations (none: the unit has none, write zeros)
  int slot;      // where its partial sums go, -1: it is a whole unit
};

// Unit of round r of CTA c in snake order.
FA_HD long long bwd_snake(int r, int c, int ctas) { return (long long)r * ctas + ((r & 1) ? ctas - 1 - c : c); }

// A CTA's pieces, in order.
struct BwdWalk {
  int r = 0, u = -1, first = 1;

  FA_HD bool next(const BwdPlan& p, int c, BwdPiece& out) {
    if (r >= 0) {
      const long long v = bwd_snake(r, c, p.ctas);
      if (v < p.whole) {
        ++r;
        p.units.locate((int)v, out.head, out.tile);
        out.it0 = 0;
        out.it1 = p.units.iterations(out.tile);
        out.slot = -1;
        return true;
      }
      r = -1;
      u = p.cut[c].unit;
    }
    const BwdCut from = p.cut[c], to = p.cut[c + 1];
    if (u > to.unit || (u == to.unit && (to.it == 0 || (u == from.unit && from.it == to.it)))) return false;
    p.units.locate(u, out.head, out.tile);
    const int n = p.units.iterations(out.tile), w = n > 0 ? n : 1;
    const int a = u == from.unit ? from.it : 0, b = u == to.unit ? to.it : w;
    out.it0 = a;
    out.it1 = n > 0 ? b : a;
    out.slot = a == 0 && b == w ? -1 : 2 * c + (first ? 0 : 1);
    first = 0;
    ++u;
    return true;
  }
};

// The pieces of the unit whose first piece ends at cut[c + 1], inside it, for
// the kernel that joins them, in order: first_slot of CTA c, then slots 2 k of
// CTAs k = c + 1 .. last whose range is not empty; false when no unit starts in
// CTA c's range and goes past it.
FA_HD bool bwd_join(const BwdPlan& p, int c, int& unit, int& last, int& first_slot) {
  const BwdCut from = p.cut[c], to = p.cut[c + 1];
  if (to.it == 0) return false;
  unit = to.unit;
  if (from.unit == unit && from.it > 0) return false;  // it started in an earlier range
  first_slot = 2 * c + (from.unit == unit ? 0 : 1);
  last = c + 1;
  while (p.cut[last + 1].unit == unit) ++last;  // (cut[ctas] lies behind the last unit)
  return true;
}

// ---- host ----

// Weights of units dealt to CTAs in snake order, from unit 0 on.  Runs of units of one
// weight count by rounds, in which each CTA has one unit: a plan takes the time of its
// levels, not of its units, where these are many (short sequences of many heads).
struct BwdDeal {
  int ctas;
  long long unit = 0, all = 0;          // next unit; what full rounds gave every CTA
  long long extra[kBwdMaxCtas] = {};    // what a CTA has besides
  long long most = 0;                   // the largest `extra`

  explicit BwdDeal(int c) : ctas(c) {}
  long long longest() const { return all + most; }
  long long of(int c) const { return all + extra[c]; }
  void one(long long w) {
    const int r = (int)(unit / ctas), at = (int)(unit - (long long)r * ctas), c = (r & 1) ? ctas - 1 - at : at;
    extra[c] += w;
    most = extra[c] > most ? extra[c] : most;
    ++unit;
  }
  // Units up to `end`, each of weight w.
  void run(long long end, long long w) {
    while (unit < end && unit % ctas) one(w);
    const long long rounds = end > unit ? (end - unit) / ctas : 0;
    all += rounds * w;
    unit += rounds * ctas;
    while (unit < end) one(w);
  }
};

// Units from u on that are known to have u's weight: the end of the run.
inline int bwd_run_end(const BwdUnits& units, int u) {
  if (!units.causal) return units.count();
  return units.spread ? (u / units.heads + 1) * units.heads : u + 1;
}

// Deals the units out to at most `sms` CTAs.  `join_cost`: iterations that a
// partial result and its join cost; units are cut only where that makes the
// longest CTA shorter by more.
inline BwdPlan bwd_plan(const BwdUnits& units, int sms, int join_cost) {
  BwdPlan p{};
  p.units = units;
  const int n = units.count();
  if (sms > kBwdMaxCtas) sms = kBwdMaxCtas;
  // All units whole.
  const int few = n < sms ? n : sms;
  long long total = 0;
  BwdDeal whole_deal(few);
  for (int u = 0; u < n;) {
    const int end = bwd_run_end(units, u);
    const long long w = units.weight(u);
    total += w * (end - u);
    whole_deal.run(end, w);
    u = end;
  }
  const long long longest = whole_deal.longest();
  // Cut: no CTA gets less than join_cost iterations.
  long long ctas = total / join_cost;
  ctas = ctas < 1 ? 1 : (ctas > sms ? sms : ctas);
  const long long target = (total + ctas - 1) / ctas;
  if (longest <= target + join_cost) {
    p.ctas = few;
    p.whole = n;
    for (int c = 0; c <= few; ++c) p.cut[c] = BwdCut{n, 0};
    return p;
  }
  p.ctas = (int)ctas;
  // Full rounds of whole units as long as no CTA passes the target.
  BwdDeal deal(p.ctas);
  int whole = 0;
  while ((long long)whole + ctas <= n) {
    const int end = bwd_run_end(units, whole);
    const long long w = units.weight(whole);
    long long rounds = (end - whole) / ctas;
    if (rounds > 0) {  // of one weight
      const long long fit = (target - deal.longest()) / w;
      if (target < deal.longest() || fit == 0) break;
      rounds = rounds < fit ? rounds : fit;
      deal.run(whole + rounds * ctas, w);
    } else {
      const int r = whole / p.ctas;
      bool fits = true;
      for (int c = 0; c < p.ctas; ++c)
        fits = fits && deal.of(c) + units.weight((int)bwd_snake(r, c, p.ctas)) <= target;
      if (!fits) break;
      for (int i = 0; i < p.ctas; ++i) deal.one(units.weight(whole + i));
      rounds = 1;
    }
    whole += (int)(rounds * ctas);
  }
  p.whole = whole;
  int u = whole, it = 0;
  for (int c = 0; c < p.ctas; ++c) {
    p.cut[c] = BwdCut{u, it};
    long long left = target - deal.of(c);
    while (left > 0 && u < n) {
      const int w = units.weight(u) - it;
      if (w <= left) {
        left -= w;
        ++u;
        it = 0;
      } else {
        it += (int)left;
        left = 0;
      }
    }
  }
  p.cut[p.ctas] = BwdCut{n, 0};
  for (int c = 1; c < p.ctas; ++c) p.joins += p.cut[c].it > 0;
  return p;
}

}  // namespace fa
