// Goes through all pieces of shared-prefix calls of random shapes with the library's
// own arithmetic (csrc/shared_plan.cuh), as its load warps do, and checks: every key
// tile of every segment is in one piece; no two pieces have a slot in common; each
// slot lies in the workspace whose size the host reckons; the merge finds exactly the
// slots of a row's pieces.  Arguments: seed, number of calls.  Exit status 0: all well.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "shared_plan.cuh"

using namespace pa::shared;

static void fail(const char* what, const Plan& p) {
  std::fprintf(stderr, "%s: B %d Hq %d Hkv %d Nq %d Np %d Nt %d ctas %d\n", what, p.B, p.Hq, p.Hkv, p.Nq, p.Np, p.Nt,
               p.ctas);
  std::exit(1);
}

// Pieces of one kind: slots in use and, for each segment, its tiles and slots.
struct Kind {
  long long slots;
  std::set<long long> used;
  std::map<long long, std::vector<int>> tiles;      // segment -> times each tile was taken
  std::map<long long, std::set<long long>> of;      // segment -> slots
  void piece(const Plan& p, long long segment, int n_tiles, int t0, int t1, long long slot) {
    if (t0 < 0 || t1 > n_tiles || t0 >= t1) fail("tiles of a piece", p);
    if (slot < 0 || slot >= slots) fail("slot outside the workspace", p);
    if (!used.insert(slot).second) fail("slot used twice", p);
    auto& v = tiles[segment];
    v.resize(n_tiles);
    for (int t = t0; t < t1; ++t) ++v[t];
    of[segment].insert(slot);
  }
};

static void check_call(Plan p) {
  int tiles = 0, some = 0;
  for (int b = 0; b < p.B; ++b) {
    const int n = Plan::tiles_of(p.len(b));
    tiles += n;
    some += n > 0;
  }
  const int pair_ctas = p.pair_ctas(tiles, some), start = p.start_units(tiles);
  if (pair_ctas < 0 || pair_ctas > p.ctas) fail("CTAs of the pairs", p);
  Kind pair{p.pair_slots(), {}, {}, {}}, odd{p.odd_slots(), {}, {}, {}}, tail{p.tail_slots(), {}, {}, {}};
  for (int block = 0; block < p.ctas; ++block) {
    if (block < pair_ctas) {
      const int lanes = p.lanes(pair_ctas), l = block % lanes, c = block / lanes;
      const Cut cut = p.pair_line(pair_ctas, lanes, l);
      const int u0 = c < cut.parts ? cut.begin(c) : 0, u1 = c < cut.parts ? cut.begin(c + 1) : 0;
      for (int u = u0; u < u1;) {
        const int s = u / p.prefix_tiles, t0 = u - s * p.prefix_tiles;
        const int t1 = std::min(p.prefix_tiles, t0 + u1 - u);
        const int which = l + s / p.Hkv * lanes;  // the pair
        if (which >= p.pairs()) fail("pair out of range", p);
        pair.piece(p, static_cast<long long>(which) * p.Hkv + s % p.Hkv, p.prefix_tiles, t0, t1,
                   Plan::pair_slot(s, c, lanes, l));
        u += t1 - t0;
      }
    } else {
      for (int stream = 0; stream < 2; ++stream) {
        const int singles = p.ctas - pair_ctas, c = stream * singles + block - pair_ctas;
        const Cut cut = p.single_line(pair_ctas, tiles, some);
        const int u0 = c < cut.parts ? cut.begin(c) : 0, u1 = c < cut.parts ? cut.begin(c + 1) : 0;
        for (int u = u0; u < std::min(u1, p.odd_units());) {
          const int s = u / p.prefix_tiles, t0 = u - s * p.prefix_tiles;
          const int t1 = std::min(p.prefix_tiles, t0 + u1 - u);
          odd.piece(p, s, p.prefix_tiles, t0, t1, Plan::single_slot(s, c));
          u += t1 - t0;
        }
        int at = p.odd_units();
        for (int b = 0; b < p.B; ++b) {
          const int n = Plan::tiles_of(p.len(b));
          if (n == 0) continue;
          for (int hk = 0; hk < p.Hkv; ++hk) {
            const int a = at + start, t0 = std::max(u0 - a, 0), t1 = std::min(u1 - a, n);
            if (t0 < t1) tail.piece(p, p.tail_segment(b, hk), n, t0, t1, Plan::single_slot(p.tail_segment(b, hk), c));
            at += n + start;
          }
        }
      }
    }
  }
  for (const Kind* k : {&pair, &odd, &tail})
    for (const auto& s : k->tiles)
      for (int n : s.second)
        if (n != 1) fail("a key tile not taken once", p);
  if (p.row_tiles > 0 && (static_cast<long long>(pair.tiles.size()) != static_cast<long long>(p.pairs()) * p.Hkv ||
                          static_cast<int>(odd.tiles.size()) != (p.odd() ? p.Hkv : 0)))
    fail("a prefix segment left out", p);
  if (static_cast<long long>(tail.tiles.size()) != static_cast<long long>(some) * p.Hkv) fail("a tail left out", p);

  int tiles_before = 0, some_before = 0;
  for (int b = 0; b < p.B; ++b) {
    for (int hk = 0; hk < p.Hkv; ++hk) {
      const Plan::Parts x = p.parts(b, hk, tiles, some, tiles_before, some_before);
      const int mt = b / p.tile_reqs;
      std::set<long long> got, want;
      const int copies_p = x.pair ? 1 : Plan::copies(p.tile_rows()), copies_t = Plan::copies(p.rows);
      for (int k = 0; k < x.n_p; ++k) got.insert(x.base_p + static_cast<long long>(k) * x.step_p);
      if (p.row_tiles > 0) {
        if (x.pair != (mt < 2 * p.pairs())) fail("kind of a row tile", p);
        if (x.pair)
          for (long long s : pair.of[static_cast<long long>(mt / 2) * p.Hkv + hk]) want.insert(2 * s + (mt & 1));
        else
          for (long long s : odd.of[hk])
            for (int u = 0; u < copies_p; ++u) want.insert(s * copies_p + u);
      }
      if (got != want || static_cast<int>(got.size()) != x.n_p) fail("the merge's slots of the prefix", p);
      got.clear();
      want.clear();
      for (int k = 0; k < x.n_t; ++k) got.insert(x.base_t + k);
      if (p.len(b) > 0)
        for (long long s : tail.of[p.tail_segment(b, hk)])
          for (int u = 0; u < copies_t; ++u) want.insert(s * copies_t + u);
      if (got != want) fail("the merge's slots of a tail", p);
    }
    const int n = Plan::tiles_of(p.len(b));
    tiles_before += n;
    some_before += n > 0;
  }
  // The regions of the workspace hold the slots counted above and do not overlap.
  for (int d : {64, 128}) {
    const Workspace w = workspace(p, d);
    const uint64_t pr = p.pair_slots() * 2 * p.tile_rows();
    const uint64_t od = p.odd_slots() * Plan::copies(p.tile_rows()) * p.tile_rows();
    const uint64_t tl = p.tail_slots() * Plan::copies(p.rows) * p.rows;
    if (w.pair_o + pr * d * 4 > w.pair_ml || w.pair_ml + pr * 8 > w.odd_o || w.odd_o + od * d * 4 > w.odd_ml ||
        w.odd_ml + od * 8 > w.tail_o || w.tail_o + tl * d * 4 > w.tail_ml || w.tail_ml + tl * 8 > w.end ||
        (w.pair_o | w.pair_ml | w.odd_o | w.odd_ml | w.tail_o | w.tail_ml) % 256)
      fail("regions of the workspace", p);
  }
}

int main(int argc, char** argv) {
  std::mt19937 rng(argc > 1 ? std::atoi(argv[1]) : 1);
  const int calls = argc > 2 ? std::atoi(argv[2]) : 1000;
  auto pick = [&](std::initializer_list<int> v) { return v.begin()[rng() % v.size()]; };
  for (int i = 0; i < calls; ++i) {
    const int G = pick({1, 1, 2, 3, 4, 7, 8, 25, 40, 128}), Nq = pick({1, 1, 1, 2, 3, 14}), Hkv = pick({1, 2, 3, 8});
    const int B = pick({1, 2, 3, 5, 17, 32, 64, 100, 130, 257, 700});
    const int Np = pick({0, 1, 100, 128, 129, 1000, 5000, 33000, 119056}), Nt = pick({0, 1, 16, 128, 129, 500, 2100});
    Plan p;
    if (!make_plan(B, G * Hkv, Hkv, Nq, Np, Nt, pick({2, 3, 7, 20, 132, 148, 160}),
                   pair_cost(rng() % 2, rng() % 2), &p)) continue;
    std::vector<int> lens(B);
    const int most = pick({0, 1, 2}), third = static_cast<int>(rng() % 3);
    for (int& n : lens) {
      n = most == 0 || Nt == 0 ? Nt : static_cast<int>(rng() % (Nt + 1));
      if (third == 0 && rng() % 4 == 0) n = 0;
      if (third == 1 && rng() % 50) n = 0;
    }
    lens[rng() % B] = pick({-5, 0, Nt, 1 << 30});  // clamped
    p.tail_lens = lens.data();
    check_call(p);
  }
  for (int Np : {0, 128, 300}) {  // as many requests as there may be
    Plan p;
    std::vector<int> lens(65535);
    for (int& n : lens) n = static_cast<int>(rng() % 9);
    if (!make_plan(65535, 1, 1, 1, Np, 8, 148, pair_cost(false, false), &p)) return 1;
    p.tail_lens = lens.data();
    check_call(p);
  }
  std::puts("slots checked");
  return 0;
}
