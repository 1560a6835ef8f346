// The barriers and rings of the cached attention's kernel for many rows
// (fa_cache_chunk.cuh) as a model on the host: its warps' waits, arrivals,
// copies and products, over the stretches that fa_cache_geom.h gives each CTA,
// run in random orders in which some of the warps are much slower than others.
// Barriers are what the hardware has: a wait names a parity, and passes
// whenever the phase under way has the other one.  Every buffer holds the
// number of the tile that it was last written for, and every use is checked.
//
// `scales_first` plants a mistake in the model: the softmax reads the scales of
// a stretch's first tile after a wait for their own barrier alone.  A warpgroup
// that has skipped a stretch then takes another tile's.
//
//   cache_ring_check kernel    the kernel's order: prints "ok" or the first error
//   cache_ring_check planted   prints "stale" if the planted mistake is seen
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <deque>
#include <random>
#include <vector>

#include "fa_cache_geom.h"

namespace {

enum Buffer { K = 0, V8 = 8, V = 16, META = 18, S = 34, P = 36, Q = 38, BUFFERS = 40 };
enum Bar {
  K_FULL = 0, K_EMPTY = 8, V8_FULL = 16, V8_EMPTY = 24, V_FULL = 32, V_EMPTY = 34, META_FULL = 36, Q_READY = 52,
  S_FULL = 54, P_HALF = 56, P_READY = 58, O_FULL = 60, JOINED = 62, BARS = 63
};
enum Kind { WAIT, ARRIVE, WRITE, READ, COPY, PRODUCT, COMMIT };

// WAIT bar parity; ARRIVE bar; WRITE / READ buffer tile; COPY (asynchronous:
// buffer, tile, then an arrival on bar); PRODUCT (in order on the tensor
// pipe: reads `a` and `buffer`, which must hold `tile` and `ta`, writes S if `out`
// is given); COMMIT (an arrival on bar when all products before it are done).
struct Op {
  Kind kind;
  int bar = 0, parity = 0, buffer = 0;
  int64_t tile = 0;
  int a = -1, out = -1;
  int64_t ta = 0;
};
Op wait(int bar, uint64_t phase) { Op o{WAIT}; o.bar = bar; o.parity = (int)(phase & 1); return o; }
Op arrive(int bar) { Op o{ARRIVE}; o.bar = bar; return o; }
Op write(int buffer, int64_t tile) { Op o{WRITE}; o.buffer = buffer; o.tile = tile; return o; }
Op read(int buffer, int64_t tile) { Op o{READ}; o.buffer = buffer; o.tile = tile; return o; }
Op copy(int buffer, int64_t tile, int bar) { Op o{COPY}; o.buffer = buffer; o.tile = tile; o.bar = bar; return o; }
Op product(int buffer, int64_t tile, int a, int64_t ta, int out) {
  Op o{PRODUCT}; o.buffer = buffer; o.tile = tile; o.a = a; o.ta = ta; o.out = out; return o;
}
Op commit(int bar) { Op o{COMMIT}; o.bar = bar; return o; }

struct Case {
  std::vector<int> lens, starts;
  int H, g, Nq, D, causal, max_len, ctas;
};

struct Cta {
  std::vector<fa::CacheSegment> stretches;
  std::vector<Op> warp[5];  // producer, conversion, MMA, softmax 0 and 1
};

// The kernel's warps, op by op.
void programs(Cta& c, int R, int D, bool scales_first) {
  const bool pair = R <= 128;
  const int KS = fa::chunk_k_stages(D, pair), VS = fa::kChunkVStages, MS = fa::kChunkMeta;
  auto &prod = c.warp[0], &conv = c.warp[1], &mma = c.warp[2];
  auto k_of = [&](int64_t n) { return (int)(n % KS); };
  auto v_of = [&](int64_t n) { return (int)(n % VS); };
  int64_t it = 0;
  for (const auto& sg : c.stretches)
    for (int j = 0; j < sg.ntiles; ++j, ++it) {
      const int s = k_of(it), m = (int)(it % MS);
      prod.insert(prod.end(), {wait(K_EMPTY + s, (it / KS & 1) ^ 1), wait(V8_EMPTY + s, (it / KS & 1) ^ 1),
                               copy(K + s, it, K_FULL + s), copy(V8 + s, it, V8_FULL + s), write(META + m, it),
                               arrive(META_FULL + m)});
      conv.insert(conv.end(), {wait(V8_FULL + s, it / KS), wait(V_EMPTY + v_of(it), (it / VS & 1) ^ 1),
                               read(V8 + s, it), write(V + v_of(it), it), arrive(V_FULL + v_of(it)),
                               arrive(V8_EMPTY + s)});
    }

  // MMA.  Q is tagged with the number of the stretch, S and P with the tile's.
  it = 0;
  uint64_t pc[2] = {0, 0}, qc[2] = {0, 0};
  int64_t unit = 0;
  auto take_k = [&](int64_t n) { mma.push_back(wait(K_FULL + k_of(n), n / KS)); };
  auto issue_s = [&](int t, int64_t n) {
    mma.push_back(product(K + k_of(n), n, Q + (pair ? 0 : t), unit, S + t));
    mma.push_back(commit(S_FULL + t));
  };
  auto issue_pv = [&](int t, int64_t n) {
    mma.push_back(wait(P_HALF + t, pc[t]));
    mma.push_back(wait(P_READY + t, pc[t]));
    mma.push_back(product(V + v_of(n), n, P + t, n, -1));
    ++pc[t];
  };
  for (const auto& sg : c.stretches) {
    const bool two = sg.rt * fa::kChunkRows + 128 < R;
    take_k(it);
    mma.push_back(wait(Q_READY, qc[0]++));
    issue_s(0, it);
    if (pair) {
      const int64_t first = it, end = it + sg.ntiles;
      mma.push_back(commit(K_EMPTY + k_of(it)));
      auto next_s = [&](int64_t n) {
        take_k(n);
        issue_s((int)((n - first) & 1), n);
        mma.push_back(commit(K_EMPTY + k_of(n)));
      };
      if (first + 1 < end) next_s(first + 1);
      for (; it < end; ++it) {
        const int t = (int)((it - first) & 1);
        mma.push_back(wait(V_FULL + v_of(it), it / VS));
        issue_pv(t, it);
        mma.push_back(commit(V_EMPTY + v_of(it)));
        if (it + 2 < end)
          next_s(it + 2);
        else
          mma.push_back(commit(O_FULL + t));
      }
    } else {
      if (two) {
        mma.push_back(wait(Q_READY + 1, qc[1]++));
        issue_s(1, it);
      }
      mma.push_back(commit(K_EMPTY + k_of(it)));
      for (int j = 0; j < sg.ntiles; ++j, ++it) {
        const bool more = j + 1 < sg.ntiles;
        mma.push_back(wait(V_FULL + v_of(it), it / VS));
        issue_pv(0, it);
        if (more) {
          take_k(it + 1);
          issue_s(0, it + 1);
        } else {
          mma.push_back(commit(O_FULL));
        }
        if (two) {
          issue_pv(1, it);
          if (!more) mma.push_back(commit(O_FULL + 1));
        }
        mma.push_back(commit(V_EMPTY + v_of(it)));
        if (more) {
          if (two) issue_s(1, it + 1);
          mma.push_back(commit(K_EMPTY + k_of(it + 1)));
        }
      }
    }
    ++unit;
  }

  for (int t = 0; t < 2; ++t) {
    auto& w = c.warp[3 + t];
    const int qt = pair ? 0 : t, step = pair ? 2 : 1;
    uint64_t sc = 0, oc = 0, jc = 0;
    it = unit = 0;
    for (const auto& sg : c.stretches) {
      const int row0 = sg.rt * fa::kChunkRows + qt * 128;
      if (row0 >= R || (pair && t >= sg.ntiles)) {
        it += sg.ntiles;
        ++unit;
        continue;
      }
      if (qt == t) {
        w.push_back(write(Q + t, unit));
        w.push_back(arrive(Q_READY + t));
      }
      for (int j = pair ? t : 0; j < sg.ntiles; j += step) {
        const int64_t n = it + j;
        const int m = (int)(n % MS);
        const Op s = wait(S_FULL + t, sc++);
        if (!scales_first && j < step) w.push_back(s);
        w.insert(w.end(), {wait(META_FULL + m, n / MS), read(META + m, n), s, read(S + t, n), write(P + t, n),
                           arrive(P_HALF + t), arrive(P_READY + t)});
      }
      w.push_back(wait(O_FULL + t, oc++));
      if (pair && sg.ntiles > 1) w.push_back(t == 0 ? wait(JOINED, jc++) : arrive(JOINED));
      it += sg.ntiles;
      ++unit;
    }
  }
}

const char* kError[] = {"", "stale scales", "wrong tile", "a score was lost", "no warp can go on"};

// One CTA in a random order; the number of the error seen, 0 for none.
int run(const Cta& c, std::mt19937& r) {
  int64_t held[BUFFERS];
  for (auto& h : held) h = -1;
  uint64_t done[BARS] = {};
  bool unread[2] = {};
  size_t at[5] = {};
  std::vector<Op> copies;
  std::deque<Op> pipe;
  double slow[7];  // five warps, the copies, the tensor pipe
  for (auto& s : slow) s = r() % 3 ? 1.0 : (r() % 2 ? 0.03 : 0.001);
  while (true) {
    int can[7], n = 0;
    double sum = 0;
    auto offer = [&](int e) { can[n++] = e; sum += slow[e]; };
    bool left = !copies.empty() || !pipe.empty();
    for (int e = 0; e < 5; ++e) {
      if (at[e] == c.warp[e].size()) continue;
      left = true;
      const Op& o = c.warp[e][at[e]];
      if (o.kind != WAIT || (int)(done[o.bar] & 1) != o.parity) offer(e);
    }
    if (!copies.empty()) offer(5);
    if (!pipe.empty()) offer(6);
    if (!left) return 0;
    if (!n) return 4;
    double x = sum * (r() / 4294967296.0);
    int e = can[n - 1];
    for (int i = 0; i < n; ++i)
      if ((x -= slow[can[i]]) < 0) {
        e = can[i];
        break;
      }
    if (e == 5) {
      const size_t i = r() % copies.size();
      held[copies[i].buffer] = copies[i].tile;
      ++done[copies[i].bar];
      copies.erase(copies.begin() + (long)i);
    } else if (e == 6) {
      const Op o = pipe.front();
      pipe.pop_front();
      if (o.kind == COMMIT) {
        ++done[o.bar];
      } else {
        if (held[o.buffer] != o.tile || held[o.a] != o.ta) return 2;
        if (o.out >= 0) {
          if (unread[o.out - S]) return 3;
          held[o.out] = o.tile;
          unread[o.out - S] = true;
        }
      }
    } else {
      const Op& o = c.warp[e][at[e]++];
      switch (o.kind) {
        case ARRIVE: ++done[o.bar]; break;
        case WRITE: held[o.buffer] = o.tile; break;
        case READ:
          if (held[o.buffer] != o.tile) return o.buffer >= META && o.buffer < S ? 1 : 2;
          if (o.buffer >= S && o.buffer < P) unread[o.buffer - S] = false;
          break;
        case COPY: copies.push_back(o); break;
        case PRODUCT:
        case COMMIT: pipe.push_back(o); break;
        default: break;
      }
    }
  }
}

// Errors of all CTAs of a case, `orders` random orders each; the number of the
// last one seen.
int check(const Case& x, bool scales_first, int orders, std::mt19937& r) {
  const int B = (int)x.lens.size(), R = x.g * x.Nq;
  fa::CacheRows rows{x.lens.data(), x.starts.empty() ? nullptr : x.starts.data(), B, x.H, x.g, x.Nq, R, fa::kChunkRows,
                     (R + fa::kChunkRows - 1) / fa::kChunkRows, x.causal, x.max_len,
                     fa::FastDiv::make((uint32_t)x.g)};
  std::vector<long long> base(B + 1, 0);
  for (int b = 0; b < B; ++b) base[b + 1] = base[b] + rows.head_tiles(x.lens[b], rows.first(b, x.lens[b])) * x.H;
  const int grid = fa::cache_active(base[B], x.ctas);
  int bad = 0, seen = 0;
  for (int i = 0; i < grid; ++i) {
    const long long t0 = fa::cache_range_begin(base[B], grid, i), t1 = fa::cache_range_begin(base[B], grid, i + 1);
    int b0 = 0;
    while (b0 + 1 < B && base[b0 + 1] <= t0) ++b0;
    fa::CacheWalk w;
    w.start(rows, t0, t1, b0, base[b0]);
    Cta c;
    fa::CacheSegment s;
    while (w.next(s)) c.stretches.push_back(s);
    programs(c, R, x.D, scales_first);
    int e = 0;
    for (int k = 0; k < orders && !e; ++k) e = run(c, r);
    if (e) {
      seen = e;
      ++bad;
    }
  }
  if (bad && !scales_first)
    std::printf("%s: %d of %d CTAs, B %d H %d g %d Nq %d D %d causal %d, %d keys\n", kError[seen], bad, grid, B, x.H, x.g,
                x.Nq, x.D, x.causal, x.lens[0]);
  return seen;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 2) return 2;
  const bool planted = std::strcmp(argv[1], "planted") == 0;
  std::mt19937 r(11);
  // Many row tiles whose last is half empty; grouped heads; a prompt; whole
  // units; runs of one-tile units before longer ones, with 128 rows or fewer.
  std::vector<Case> cases = {
      {{16896}, {}, 24, 1, 300, 128, 1, 16896, 152}, {{16896}, {}, 24, 1, 2100, 128, 1, 16896, 152},
      {std::vector<int>(8, 8192), {}, 8, 4, 75, 64, 0, 8192, 152}, {{10800}, {}, 24, 1, 10800, 32, 1, 10800, 152},
      {{16896}, {}, 24, 1, 512, 128, 0, 16896, 152}};
  std::vector<int> ragged;
  for (int i = 0; i < 60; ++i) ragged.push_back(i % 4 == 3 ? 700 : 100);
  cases.push_back({ragged, {}, 8, 1, 20, 128, 1, 704, 19});
  cases.push_back({ragged, {}, 8, 1, 128, 64, 0, 704, 13});
  if (planted) {
    for (size_t i = 0; i < cases.size(); ++i)
      if (i != 4 && check(cases[i], true, 20, r) != 1) return std::printf("case %zu: not seen\n", i), 1;
    std::printf("stale\n");
    return 0;
  }
  for (const Case& c : cases)
    if (check(c, false, 6, r)) return 1;
  for (int i = 0; i < 400; ++i) {
    Case c{};
    const int B = 1 + r() % 30;
    c.max_len = 1 << (7 + r() % 6);
    for (int b = 0; b < B; ++b) c.lens.push_back((int)(r() % (c.max_len + 1)) >> (r() % 3 ? 0 : 4));
    c.H = 1 + r() % 6;
    c.g = 1 + r() % 4;
    c.Nq = 1 + r() % (r() % 2 ? 40 : 700);
    if (c.g * c.Nq <= 16) c.Nq = 17;
    c.D = 32 << r() % 3;
    c.causal = r() % 2;
    c.ctas = 1 + r() % 12;
    if (r() % 4 == 0)
      for (int b = 0; b < B; ++b) c.starts.push_back((int)(r() % (c.max_len + 1)) - 50);
    if (check(c, false, 4, r)) return 1;
  }
  std::printf("ok\n");
  return 0;
}
