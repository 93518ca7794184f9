// How the work of a shared-prefix call (attn_shared.cuh) is cut into pieces, and
// where the partial results of each lie in the caller's workspace: plain integer
// arithmetic, the same in both kernels, on the host that sizes the workspace, and in
// a test that goes through all pieces with a C++ compiler alone.
#pragma once

#include <cmath>
#include <cstdint>

#ifdef __CUDACC__
#define PA_HD __host__ __device__
#else
#define PA_HD
#endif

namespace pa {

constexpr int kPlanRows = 128, kPlanKeys = 128;  // a row tile, a key tile

namespace shared {

constexpr int kMaxCtas = 160;  // sizes the workspace; the grid is one CTA an SM, at most this many
// What a pair's key tile and a unit of the singles cost, in parts of one another:
// how the CTAs are dealt to the two kinds.  Both the cap and the bias lengthen the
// softmax that bounds pairs, and hide behind the loads of singles.  Five shapes (64 to
// 256 requests, groups of 2 to 8 heads, prefixes of 8192 to 32768 keys, tails of 64 to
// 1024), each at 9, 12, 15, 18, 22 and 27 : 6, d 128 and 64, relative to 15 : 6 in the
// geometric mean:
//   plain   1.09 1.03 1 1.07 1.17 1.31     1.13 1.04 1 1.01 1.10 1.20
//   capped  1.12 1.04 1 1.04 1.13 1.26     1.14 1.05 1 1.04 1.12 1.24
//   biased  1.13 1.05 1 1.00 1.08 1.20     1.14 1.06 1 0.99 1.02 1.13
//   both    1.16 1.06 1 0.99 0.94 0.95     1.16 1.07 1 0.99 0.95 0.95
constexpr int kSingleCost = 6;
inline int pair_cost(bool cap, bool bias) { return cap && bias ? 22 : 15; }

PA_HD inline int clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }
PA_HD inline float to_float(long long x) { return static_cast<float>(x); }
PA_HD inline int round_int(float x) { return static_cast<int>(rintf(x)); }
PA_HD inline int load(const int* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}

// A line of n units cut into `parts` parts, none empty, sizes differing by one.
struct Cut {
  int n, parts, q, r;
  PA_HD Cut(int n_, int most)
      : n(n_), parts(n_ < most ? (n_ > 1 ? n_ : 1) : (most > 1 ? most : 1)), q(n_ / parts), r(n_ - q * parts) {}
  PA_HD int begin(int c) const { return c * q + (c < r ? c : r); }
  PA_HD int holder(int u) const { return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q; }
};

// Shapes of a call.
struct Plan {
  int B, Hq, Hkv, G, Nq;
  int rows;          // rows of one request under one K/V head: G * Nq
  int tile_reqs;     // requests in a row tile: 128 / rows, at most B
  int row_tiles;     // ceil(B / tile_reqs); 0 without a prefix
  int Np, Nt;
  int prefix_tiles;  // key tiles of the prefix
  int ctas;
  int pair_cost;     // see pair_cost()
  const int* tail_lens;

  PA_HD int tile_rows() const { return tile_reqs * rows; }
  PA_HD int pairs() const { return row_tiles / 2; }
  PA_HD bool odd() const { return (row_tiles & 1) != 0; }
  PA_HD int pair_units() const { return Hkv * pairs() * prefix_tiles; }
  // Pairs side by side, lane l of them taken by the CTAs c with c mod lanes = l;
  // with more pairs than CTAs a lane has several, l, l + lanes, ..
  PA_HD int lanes(int pair_ctas) const { return pairs() < pair_ctas ? pairs() : pair_ctas; }
  PA_HD int lane_pairs(int lanes, int l) const { return (pairs() - l + lanes - 1) / lanes; }
  PA_HD int odd_units() const { return odd() ? Hkv * prefix_tiles : 0; }
  // Copies of a row tile's rows.
  PA_HD static int copies(int n) { return n <= 32 ? 4 : n <= 64 ? 2 : 1; }
  PA_HD int len(int b) const { return clamp(load(tail_lens + b), 0, Nt); }
  PA_HD static int tiles_of(int keys) { return (keys + kPlanKeys - 1) / kPlanKeys; }
  // CTAs that take pairs, given the key tiles (under one K/V head) of all tails
  // and the number of tails that have any; a tail's start costs about a tile.
  PA_HD int pair_ctas(int tiles, int tails) const {
    const long long p = static_cast<long long>(pair_units()) * pair_cost;
    const long long s = (odd_units() + (tiles + tails) * static_cast<long long>(Hkv)) * kSingleCost;
    if (p == 0) return 0;
    if (s == 0) return ctas <= pairs() ? ctas : ctas - ctas % pairs();
    // One division and one product, each rounded once: the same in both kernels.
    const float share = to_float(p) / to_float(p + s);
    const int n = clamp(round_int(static_cast<float>(ctas) * share), 1, ctas - 1);
    return n <= pairs() ? n : n - n % pairs();  // as many for every pair
  }
  // Units of the line before a tail's own tiles, for its start: one where the prefix
  // has more row tiles x key tiles than the tails (`tiles` of them).  Counted and
  // not: 7 requests of 119056 + 333 keys 234 and 258 us, 32 of 32768 + 300 52 and 57,
  // 128 on pairs of 32768 + 1024 132 and 142.  Where tails are most of the work,
  // HBM evens out their starts, and a coarser line only costs: 100 requests of
  // 1000 + 600 47 and 41, 128 of 100 + 2000 75 and 73, 32 of 4608 + 1152 35 and 33.
  PA_HD int start_units(int tiles) const { return row_tiles * prefix_tiles >= tiles ? 1 : 0; }

  // Where the partial results of a piece lie: segment + part, no two pieces alike
  // since both only grow along a line, none at or past the number of segments and
  // parts.  Pairs: segment s = (pair of the lane) * Hkv + K/V head, part c of lane l.
  PA_HD int pair_segment(int mt, int hk, int lanes) const { return mt / 2 / lanes * Hkv + hk; }
  PA_HD int tail_segment(int req, int hk) const { return req * Hkv + hk; }
  PA_HD static int pair_slot(int s, int c, int lanes, int l) { return (s + c) * lanes + l; }
  PA_HD static int single_slot(int s, int c) { return s + c; }
  // Slots of each kind, for any number of CTAs up to kMaxCtas and of lanes up to the pairs.
  PA_HD long long pair_slots() const { return pairs() > 0 ? 2ll * Hkv * pairs() + kMaxCtas : 0; }
  PA_HD long long odd_slots() const { return odd() ? Hkv + 2ll * kMaxCtas : 0; }
  PA_HD long long tail_slots() const { return Nt > 0 ? static_cast<long long>(B) * Hkv + 2ll * kMaxCtas : 0; }

  // The lines, given key tiles and number of the tails that have any.
  PA_HD Cut pair_line(int pair_ctas, int lanes, int l) const {
    return Cut(lane_pairs(lanes, l) * Hkv * prefix_tiles, pair_ctas / lanes);
  }
  PA_HD Cut single_line(int pair_ctas, int tiles, int tails) const {
    return Cut(odd_units() + (tiles + start_units(tiles) * tails) * Hkv, 2 * (ctas - pair_ctas));
  }

  // Where a row's partial results lie: n_p of the prefix, slot base_p + k * step_p
  // (in row tiles; a pair's two row tiles lie side by side), n_t of the tail, from
  // slot base_t on; copies of a row side by side, too.  tiles, tails: of all requests;
  // tiles_before, tails_before: of those before req.
  struct Parts {
    bool pair;
    int base_p, step_p, n_p, base_t, n_t;
  };
  PA_HD Parts parts(int req, int hk, int tiles, int tails, int tiles_before, int tails_before) const {
    Parts x;
    const int n_tail = tiles_of(len(req)), n_pair = pair_ctas(tiles, tails), start = start_units(tiles);
    const int mt = req / tile_reqs;
    x.pair = mt < 2 * pairs();
    const Cut singles = single_line(n_pair, tiles, tails);
    x.base_p = x.n_p = x.base_t = x.n_t = 0;
    x.step_p = 1;
    if (row_tiles > 0 && x.pair) {
      const int n_lanes = lanes(n_pair), l = mt / 2 % n_lanes, s = pair_segment(mt, hk, n_lanes);
      const Cut cut = pair_line(n_pair, n_lanes, l);
      const int c = cut.holder(s * prefix_tiles);
      x.n_p = cut.holder((s + 1) * prefix_tiles - 1) + 1 - c;
      x.base_p = 2 * pair_slot(s, c, n_lanes, l) + (mt & 1);
      x.step_p = 2 * n_lanes;
    } else if (row_tiles > 0) {
      const int c = singles.holder(hk * prefix_tiles), copy = copies(tile_rows());
      x.n_p = (singles.holder((hk + 1) * prefix_tiles - 1) + 1 - c) * copy;
      x.base_p = single_slot(hk, c) * copy;
    }
    if (n_tail > 0) {
      const int at = odd_units() + (tiles_before + start * tails_before) * Hkv + hk * (n_tail + start) + start;
      const int c = singles.holder(at), copy = copies(rows);
      x.n_t = (singles.holder(at + n_tail - 1) + 1 - c) * copy;
      x.base_t = single_slot(tail_segment(req, hk), c) * copy;
    }
    return x;
  }
};

// Shapes of a call; false where the rows of one request under one K/V head do not
// fit a row tile, or the key tiles a 32-bit count.
inline bool make_plan(int B, int Hq, int Hkv, int Nq, int Np, int Nt, int ctas, int pair_cost, Plan* plan) {
  const long long rows = static_cast<long long>(Hq / Hkv) * Nq;
  if (rows < 1 || rows > kPlanRows) return false;
  plan->B = B;
  plan->Hq = Hq;
  plan->Hkv = Hkv;
  plan->G = Hq / Hkv;
  plan->Nq = Nq;
  plan->rows = static_cast<int>(rows);
  plan->tile_reqs = B < kPlanRows / plan->rows ? B : kPlanRows / plan->rows;
  plan->row_tiles = Np > 0 ? (B + plan->tile_reqs - 1) / plan->tile_reqs : 0;
  plan->Np = Np;
  plan->Nt = Nt;
  plan->prefix_tiles = Plan::tiles_of(Np);
  plan->ctas = ctas;
  plan->pair_cost = pair_cost;
  plan->tail_lens = nullptr;
  // The kernels count key tiles in 32 bits.
  const long long units = static_cast<long long>(Hkv) * (static_cast<long long>(plan->prefix_tiles) * plan->row_tiles +
                                                         static_cast<long long>(B) * Plan::tiles_of(Nt));
  return units < (1ll << 30);
}

// Byte offsets of the parts of a workspace (each on a 256-byte boundary), and their
// end.  O: fp32 rows of d; ml: a row's maximum and sum.
struct Workspace {
  uint64_t pair_o, pair_ml, odd_o, odd_ml, tail_o, tail_ml, end;
};

inline Workspace workspace(const Plan& plan, int d) {
  auto up = [](uint64_t n) { return (n + 255) & ~255ull; };
  const uint64_t rows = plan.rows, tile = plan.tile_rows();
  const uint64_t pair = plan.pair_slots() * 2 * tile;
  const uint64_t odd = plan.odd_slots() * Plan::copies(plan.tile_rows()) * tile;
  const uint64_t tail = plan.tail_slots() * Plan::copies(plan.rows) * rows;
  Workspace w;
  w.pair_o = 0;
  w.pair_ml = up(pair * d * 4);
  w.odd_o = w.pair_ml + up(pair * 8);
  w.odd_ml = w.odd_o + up(odd * d * 4);
  w.tail_o = w.odd_ml + up(odd * 8);
  w.tail_ml = w.tail_o + up(tail * d * 4);
  w.end = w.tail_ml + up(tail * 8);
  return w;
}

}  // namespace shared
}  // namespace pa
