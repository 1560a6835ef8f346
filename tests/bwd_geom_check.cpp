// Checks fa_bwd_geom.h against a plain enumeration: every iteration of every unit
// is in exactly one piece, pieces lie inside their units, whole units have no slot,
// slots are distinct, and the joins list the pieces of each cut unit in order.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "fa_bwd_geom.h"

using namespace fa;

#define REQUIRE(x, ...)                                     \
  do {                                                      \
    if (!(x)) {                                             \
      std::printf("failed: %s  ", #x);                      \
      std::printf(__VA_ARGS__);                             \
      std::printf("\n");                                    \
      std::exit(1);                                         \
    }                                                       \
  } while (0)

static long long checked = 0, cut_units = 0, empty_units = 0;

static void check(int heads, int tiles, int other, int group, int causal, int rows_q, int spread, int sms, int cost) {
  BwdUnits u{};
  u.heads = heads;
  u.tiles = tiles;
  u.other = other;
  u.group = group;
  u.causal = causal;
  u.rows_q = rows_q;
  u.spread = spread;
  u.div_heads = FastDiv::make((uint32_t)heads);
  u.div_tiles = FastDiv::make((uint32_t)tiles);
  const BwdPlan p = bwd_plan(u, sms, cost);
  char what[200];
  std::snprintf(what, sizeof what, "heads %d tiles %d other %d group %d causal %d rows_q %d spread %d sms %d cost %d",
                heads, tiles, other, group, causal, rows_q, spread, sms, cost);
  REQUIRE(p.ctas >= 1 && p.ctas <= sms && p.ctas <= kBwdMaxCtas, "%s", what);
  const int n = u.count();
  // units <-> (head, tile)
  std::vector<int> unit_of((size_t)n, -1);
  for (int i = 0; i < n; ++i) {
    int h, t;
    u.locate(i, h, t);
    REQUIRE(h >= 0 && h < heads && t >= 0 && t < tiles && unit_of[(size_t)h * tiles + t] < 0, "%s", what);
    unit_of[(size_t)h * tiles + t] = i;
    int first, len, want = 0, lo = -1;
    u.range(t, first, len);
    for (int o = 0; o < other; ++o) {
      const bool seen = !causal || (rows_q ? o <= t : o >= t);
      if (seen && lo < 0) lo = o;
      want += seen;
    }
    REQUIRE(len == want && (len == 0 || first == lo) && u.iterations(t) == want * group, "%s tile %d", what, t);
  }
  struct Seen {
    int it0, it1, slot, cta;
  };
  std::vector<std::vector<Seen>> pieces((size_t)n);
  std::set<int> slots;
  long long longest = 0, total = 0;
  for (int c = 0; c < p.ctas; ++c) {
    BwdWalk w;
    BwdPiece pc;
    long long load = 0;
    int guard = 0;
    while (w.next(p, c, pc)) {
      REQUIRE(++guard < 10000000, "%s", what);
      const int i = unit_of[(size_t)pc.head * tiles + pc.tile];
      const int it = u.iterations(pc.tile);
      REQUIRE(pc.it0 >= 0 && pc.it1 <= it && (it == 0 ? pc.it0 == pc.it1 : pc.it0 < pc.it1), "%s unit %d [%d, %d) of %d",
              what, i, pc.it0, pc.it1, it);
      const bool is_whole = pc.it0 == 0 && pc.it1 == it;
      REQUIRE((pc.slot < 0) == is_whole, "%s", what);
      if (pc.slot >= 0) REQUIRE(pc.slot / 2 == c && slots.insert(pc.slot).second, "%s slot %d", what, pc.slot);
      pieces[(size_t)i].push_back(Seen{pc.it0, pc.it1, pc.slot, c});
      load += it > 0 ? pc.it1 - pc.it0 : 1;
    }
    REQUIRE(!w.next(p, c, pc), "%s", what);
    longest = load > longest ? load : longest;
    total += load;
  }
  std::map<int, std::vector<int>> joined;  // unit -> slots
  for (int c = 0; c < p.ctas; ++c) {
    int unit, last, slot;
    if (!bwd_join(p, c, unit, last, slot)) continue;
    REQUIRE(unit >= 0 && unit < n && last < p.ctas && joined.count(unit) == 0, "%s", what);
    auto& list = joined[unit];
    for (int k = c; k <= last; ++k) {
      if (k > c) {
        slot = 2 * k;
        if (p.cut[k].unit == p.cut[k + 1].unit && p.cut[k].it == p.cut[k + 1].it) continue;
      }
      list.push_back(slot);
    }
  }
  REQUIRE((p.joins > 0) == !joined.empty(), "%s joins %d", what, p.joins);
  for (int i = 0; i < n; ++i) {
    int h, t;
    u.locate(i, h, t);
    const int it = u.iterations(t);
    auto& s = pieces[(size_t)i];
    REQUIRE(!s.empty(), "%s unit %d has no piece", what, i);
    int at = 0;
    std::vector<int> order;
    for (auto& x : s) {  // (CTAs ascending: iterations ascending)
      REQUIRE(x.it0 == at, "%s unit %d", what, i);
      at = x.it1;
      if (x.slot >= 0) order.push_back(x.slot);
    }
    REQUIRE(at == it, "%s unit %d covers %d of %d", what, i, at, it);
    if (s.size() > 1 || s[0].slot >= 0) {
      REQUIRE(joined.count(i) && joined[i] == order, "%s unit %d joins", what, i);
      ++cut_units;
    } else {
      REQUIRE(!joined.count(i), "%s unit %d joined though whole", what, i);
      REQUIRE(it > 0 || s.size() == 1, "%s", what);
      empty_units += it == 0;
    }
  }
  if (p.joins) REQUIRE(longest <= (total + p.ctas - 1) / p.ctas, "%s longest %lld of %lld", what, longest, total);
  ++checked;
}

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (uint32_t)(hi - lo + 1)); };
  for (int sms : {1, 2, 7, 152, 192})
    for (int causal : {0, 1})
      for (int rows_q : {0, 1})
        for (int heads : {1, 3, 16, 48})
          for (int tiles : {1, 2, 9, 36})
            for (int other : {1, 5, 36}) check(heads, tiles, other, rows_q ? 1 : 4, causal, rows_q, causal, sms, 4);
  for (int i = 0; i < 6000; ++i) {
    const int causal = pick(0, 1), rows_q = pick(0, 1);
    check(pick(1, 40), pick(1, 40), pick(1, 60), rows_q ? 1 : pick(1, 8), causal, rows_q, pick(0, 1), pick(1, 192), pick(1, 8));
  }
  check(24, 931, 931, 1, 0, 0, 0, 152, 4);
  check(24, 931, 931, 1, 1, 1, 0, 152, 4);
  check(1, 1, 4000, 1, 0, 1, 0, 152, 4);
  check(70000, 1, 1, 1, 0, 1, 0, 152, 4);
  if (cut_units < 1000 || empty_units < 1000) {
    std::printf("too few cases: %lld cut, %lld empty\n", cut_units, empty_units);
    return 1;
  }
  std::printf("ok\n");
  return 0;
}
