// Attention of a few new tokens of many requests over one shared prefix and each
// request's own tail (pa_attn_shared_prefix) on sm_100a.
//
// Token t of request b (t < Nq) stands at position Np + len_b - Nq + t.  It sees
// all Np prefix keys and the tail keys j <= len_b - Nq + t.  Scores are capped
// and biased as score_mod.cuh says.  The prefix is read once for all requests:
// the rows of all of them (Nq tokens x G query heads a K/V head) are stacked
// into tiles of up to 128 rows.
//
// Work.  A segment is the keys one row tile has to go over: the prefix under one
// K/V head, or one request's tail under one K/V head.  Two row tiles over the
// same prefix make a pair, which shares its K and V tiles; what is left (the
// prefix under an odd row tile, and the tails) is single.  The singles form a line
// of key tiles (128 keys), and in some calls one more unit for the start of each
// tail (start_units), cut into equal parts, one for each of the two streams (a
// softmax warpgroup, its MMA and its load warp) of the CTAs that take singles.
// The other CTAs take pairs, as many CTAs a pair: CTA c has pair c mod (pairs), and
// the prefix, cut into equal parts, part c / (pairs) of it, so that the CTAs of
// one part read the same tiles at the same time and HBM gives them once (with
// one line of all pairs the same tile was read at two far times, and tails
// streaming through L2 drove it out in between, by chance: 100 to 130 us with
// neighbouring numbers of CTAs, where this takes 107 to 111).
// Every SM gets the same share whatever the lengths are, without counters and
// without host knowledge of them.  The part of a segment that falls to one part of the
// line is a piece; segment + part is another number for every piece, since both
// only grow along the line, and names the place of its partial results in the
// caller's workspace: O rows as the accumulators hold them, fp32, and each row's
// maximum (base 2) and sum of weights.
// shared_merge_kernel joins them, finding them by the same arithmetic.
//
// The streams of a single CTA run independently, so that one stream's loads,
// tensor work and softmax fill the other's waits.  Row tiles of few rows (32 or
// less; 64 or less) hold their rows four times (twice): every copy lies in the
// tensor-memory lanes of a warp of its own, which takes its quarter (half) of
// the tile's keys, with zero weights for the rest.  One warp working through 128
// keys a row took longer than the tile's loads: 4.5 TB/s where the copies reached
// 5.6 (24 heads, 119056 keys, 21 rows).  The copies' results are joined like those
// of different pieces.  Without starts on the line, the streams at its end had some
// forty short tails each there and finished 60 us behind the others; with them the
// kernel takes 230 us for 1.47 GB read again and again (6.4 TB/s, L2 keeps a part) and
// 260 to 280 us in a call whose buffers change (5.4 TB/s).
//
// Warps: 0-3, 4-7 softmax of stream 0 and 1 (208 registers); 8, 11 MMA issue of
// stream 0 and 1 (8 issues for both in a pair CTA); 9, 10 pieces and TMA loads
// of stream 0 and 1 (9 for both in a pair CTA).
//
// Bound: HBM (64 KB of K and V a tile at d = 128) as long as few rows share a
// tile; pairs are tensor and special-function work, their re-reads come from L2.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "attn_mod.cuh"
#include "score_mod.cuh"
#include "shared_plan.cuh"

namespace pa {
namespace shared {

using namespace mod;

using R = Roles<false>;  // warps and registers of the single-warpgroup kernel

constexpr int kMergeWarps = 8;
constexpr int kLoadWarp = 9;   // + stream
static_assert(kBM == kPlanRows && kBN == kPlanKeys, "tiles of the plan");

struct Params {
  Plan plan;
  // The operands as they lie in memory, for the merge's redo_row.
  const __nv_bfloat16* q;
  const __nv_bfloat16* kp;
  const __nv_bfloat16* vp;
  const __nv_bfloat16* kt;
  const __nv_bfloat16* vt;
  long long kp_s[2], vp_s[2];  // prefix strides: head, row (elements)
  long long kt_s[3], vt_s[3];  // tail strides: batch, head, row
  float* pair_o;               // [((segments of a lane + parts) * lanes) * 2][tile_rows][D]
  float2* pair_ml;
  float* odd_o;                // [(Hkv + 2 * ctas) * copies][tile_rows][D]
  float2* odd_ml;
  float* tail_o;               // [(B * Hkv + 2 * ctas) * copies][rows][D]
  float2* tail_ml;
  ScoreMod sm;
  int* status;
  unsigned long long timeout_ns;
};

constexpr int kEnd = -1, kTail = 0, kOdd = 1, kPair = 2;

// A piece as its load warp hands it out.
struct Piece {
  int kind;
  int hk;
  int req;     // a tail's request, or the first request of the row tile (of the first one of a pair)
  int t0, t1;  // its key tiles
  int slot;    // segment + part
  int keys;    // keys of the segment
};

template <int D>
struct SharedLayout {
  static constexpr int kStages = D == 64 ? 8 : 4;  // 128 KB of K and V; half of them a stream's own in a single CTA
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = kQOff + kQTiles * kTileBytes;
  static constexpr int kStageOff = kRingOff + kStages * kTileBytes;
  static constexpr int kStageWarpBytes = 32 * 128;
  static constexpr int kBarOff = kStageOff + 8 * kStageWarpBytes;
  // q_full[2], q_empty[2], kv_full[S], kv_empty[S], s_full[2], p_part[2],
  // p_full[2], o_full[2], drain[2], piece_full[2][2], piece_empty[2][2]
  static constexpr int kNumBars = 4 + 2 * kStages + 8 + 2 + 8;
  static constexpr int kPieceOff = kBarOff + kNumBars * 8;
  static constexpr int kTmemSlotOff = kPieceOff + 4 * static_cast<int>(sizeof(Piece));
  static constexpr int kAbortOff = kTmemSlotOff + 4;
  static constexpr int kBytes = kAbortOff + 4;
  static constexpr int kMinOneCtaPerSm = 120 * 1024;
  static constexpr int kAllocBytes = (kBytes + 1024 > kMinOneCtaPerSm) ? (kBytes + 1024) : kMinOneCtaPerSm;
};

// softmax_tile for a warp that takes kKeys keys of the tile, those from kq *
// kKeys on, of rows that have a copy in its tensor-memory lanes; the weights of
// the tile's other keys are zero in this copy.  The row sees keys j < b of the
// tile.  All exponentials on the special-function unit: a warp has few enough.
template <int D, bool kCap, bool kBias, int kKeys>
__device__ __forceinline__ void softmax_share(uint32_t tS, uint32_t tO, int kq, int b, float dist0, float slope2,
                                              const ScoreMod& sm, bool counts, bool have_o, float& m_ref, float& l,
                                              uint32_t bar_part, uint32_t bar_full, int lane) {
  constexpr bool kMod = kCap || kBias;
  const int e0 = kq * kKeys;
  uint64_t x[kKeys / 2];
  {
    uint32_t sr[kKeys];
    if constexpr (kKeys == 32)
      tmem_ld_x32(tS + e0, sr);
    else
      tmem_ld_x64(tS + e0, sr);
#pragma unroll
    for (int e = 0; e < kKeys / 2; ++e) x[e] = f2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
  }
  if constexpr (kCap) cap_scores<kKeys / 2>(x, tS + e0, sm, counts);
  if constexpr (kBias)
    bias_scores<kKeys / 2, !kCap>(x, sm.scale_log2, slope2, dist0 - static_cast<float>(e0), 0, b - e0);
  if (__any_sync(0xffffffffu, b < e0 + kKeys)) hide<kKeys / 2>(x, 0, b - e0);
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < kKeys / 2; ++e) {
    float x0, x1;
    f2_split(x[e], x0, x1);
    m4[e & 3] = max3f(m4[e & 3], x0, x1);
  }
  float mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]);
  if constexpr (!kMod) mx *= sm.scale_log2;
  float alpha = 1.f;
  bool rescale = false;
  if (mx > m_ref + kRescaleLog2) {
    alpha = ex2_approx(m_ref - mx);
    l *= alpha;
    m_ref = mx;
    rescale = have_o;
  }
  if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t orr[32];
      tmem_ld_x32(tO + ch * 32, orr);
#pragma unroll
      for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
      tmem_st_x32(tO + ch * 32, orr);
    }
  }
  const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
  uint32_t zero[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) zero[e] = 0u;
  float l2[2] = {0.f, 0.f};
  constexpr int kParts = kKeys / 32;
#pragma unroll
  for (int ch = 0; ch < kParts; ++ch) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t nm2 = f2(neg_m, neg_m), xe = x[ch * 16 + e];
      float x0, x1;
      f2_split(kMod ? f2_add(xe, nm2) : f2_fma(xe, f2(sm.scale_log2, sm.scale_log2), nm2), x0, x1);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      l2[0] += p0;
      l2[1] += p1;
      pk[e] = pack_bf16x2(p0, p1);
    }
    tmem_st_x16(tS + (kq * kParts + ch) * 16, pk);
  }
#pragma unroll
  for (int u = kParts; u < 4; ++u) tmem_st_x16(tS + ((kq * kParts + u) & 3) * 16, zero);
  l += l2[0] + l2[1];
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(bar_part);
    mbar_arrive(bar_full);
  }
}

// A thread's O row as it is, to dst, where `write`.  For a warp with few rows: no
// staging.  Kept as short as it can be, like store_raw_rows: it runs once a piece,
// and long straight code that has left the instruction cache costs more than
// its instructions (scaling and checking the row here: 4 500 clocks).
template <int D>
__device__ __noinline__ void store_raw_row(uint32_t tO, float* dst, bool write) {
  uint32_t w[D];
  if constexpr (D == 128)
    tmem_ld_x128(tO, w);
  else
    tmem_ld_x64(tO, w);
  if (write)
#pragma unroll
    for (int u = 0; u < D / 4; ++u)
      reinterpret_cast<uint4*>(dst)[u] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
}

// The O rows of a warp as they are, through its staging area (see attn_fwd.cuh):
// row r at dst + r * D, rows r >= rows_left not written.
template <int D>
__device__ __noinline__ void store_raw_rows(uint32_t tO, uint32_t stg, float* dst, int rows_left) {
  const int lane = threadIdx.x % 32;
  const int r0 = lane >> 3, c = lane & 7;
#pragma unroll 1
  for (int ch = 0; ch < D / 32; ++ch) {
    uint32_t w[32];
    tmem_ld_x32(tO + ch * 32, w);
    __syncwarp();  // the previous piece has left the staging area
#pragma unroll
    for (int u = 0; u < 8; ++u)
      st_shared_v4(stg + lane * 128 + ((u ^ (lane & 7)) << 4), w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 4 * k + r0;
      const uint4 x = ld_shared_v4(stg + r * 128 + ((c ^ (r & 7)) << 4));
      if (r < rows_left) *reinterpret_cast<uint4*>(dst + r * D + ch * 32 + c * 4) = x;
    }
  }
}

template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(R::kThreads, 1)
    attn_shared_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qt,
                       const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                       const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                       const __grid_constant__ Params p) {
  using L = SharedLayout<D>;
  constexpr int kStages = L::kStages;
  constexpr int kHalf = kStages / 2;  // ring slots of a stream in a single CTA
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);

  const uint32_t sQ = base + L::kQOff;
  const uint32_t sRing = base + L::kRingOff;
  const uint32_t bars = base + L::kBarOff;
  const uint32_t bar_q_full0 = bars, bar_q_empty0 = bars + 8 * 2;
  const uint32_t bar_kv_full0 = bars + 8 * 4;
  const uint32_t bar_kv_empty0 = bars + 8 * (4 + kStages);
  const uint32_t bar_s_full0 = bars + 8 * (4 + 2 * kStages);
  const uint32_t bar_p_part0 = bars + 8 * (6 + 2 * kStages);
  const uint32_t bar_p_full0 = bars + 8 * (8 + 2 * kStages);
  const uint32_t bar_o_full0 = bars + 8 * (10 + 2 * kStages);
  const uint32_t bar_drain0 = bars + 8 * (12 + 2 * kStages);
  const uint32_t bar_piece_full0 = bars + 8 * (14 + 2 * kStages);   // + 8 * (2 * stream + slot)
  const uint32_t bar_piece_empty0 = bars + 8 * (18 + 2 * kStages);
  volatile Piece* slots = reinterpret_cast<volatile Piece*>(gbase + L::kPieceOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kTmemSlotOff);
  volatile int* abort_word = reinterpret_cast<volatile int*>(gbase + L::kAbortOff);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint64_t lim = p.timeout_ns;
  const Plan& plan = p.plan;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_kv_full0 + 8 * s, 1);
      mbar_init(bar_kv_empty0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q_full0 + 8 * i, 1);
      mbar_init(bar_q_empty0 + 8 * i, 1);
      mbar_init(bar_s_full0 + 8 * i, 1);
      mbar_init(bar_p_part0 + 8 * i, 4);  // one arrival per softmax warp
      mbar_init(bar_p_full0 + 8 * i, 4);
      mbar_init(bar_o_full0 + 8 * i, 1);
      mbar_init(bar_drain0 + 8 * i, 1);
    }
    for (int u = 0; u < 4; ++u) {
      mbar_init(bar_piece_full0 + 8 * u, 1);
      mbar_init(bar_piece_empty0 + 8 * u, 5);  // 4 softmax warps and the MMA warp of the stream
    }
    *abort_word = 0;
    fence_barrier_init();
  }
  // The load warps reckon while the barriers and tensor memory are set up: all
  // units of tails under one K/V head, and the CTAs that take pairs.
  int tiles = 0, some = 0, pair_ctas = 0;
  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    for (int b0 = 0; b0 < plan.B; b0 += 128) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int b = b0 + u * 32 + lane;
        const int n = b < plan.B ? Plan::tiles_of(plan.len(b)) : 0;
        tiles += n;
        some += n > 0;
      }
    }
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    some = __reduce_add_sync(0xffffffffu, some);
    pair_ctas = plan.pair_ctas(tiles, some);
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&tm_qp);
    prefetch_tensormap(&tm_kp);
    prefetch_tensormap(&tm_vp);
  }
  if (warp == kLoadWarp + 1 && lane == 0) {
    prefetch_tensormap(&tm_qt);
    prefetch_tensormap(&tm_kt);
    prefetch_tensormap(&tm_vt);
  }
  if (warp == R::kMma) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // The merge may be launched as CTAs end; it waits for the last one itself.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    const bool got = mbar_wait_hint(bar, parity, abort_word, p.status, kStatusTimeout, lim, kSuspendHintNs);
    return __all_sync(0xffffffffu, got);
  };
  // The it-th piece of a stream, copied out of its slot; false at the end (or
  // where a wait gave up, with `ok` cleared).
  auto next_piece = [&](int i, int it, Piece& x, bool& ok) {
    const int u = 2 * i + (it & 1);
    if (!wait_all(bar_piece_full0 + 8 * u, (it >> 1) & 1)) {
      ok = false;
      return false;
    }
    x.kind = slots[u].kind;
    x.hk = slots[u].hk;
    x.req = slots[u].req;
    x.t0 = slots[u].t0, x.t1 = slots[u].t1;
    x.slot = slots[u].slot;
    x.keys = slots[u].keys;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_piece_empty0 + 8 * u);
    return x.kind != kEnd;
  };

  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    setmaxnreg_dec<R::kControlRegs>();
    // --------------------------------------------------- pieces and loads
    const int i = warp - kLoadWarp;
    const bool leader = elect_one();
    bool ok = true;
    int it = 0;   // pieces handed out
    int idx = 0;  // ring loads issued so far
    // Ring slots this warp fills: all of them in a pair CTA, else its half.
    int slot0 = i * kHalf, n_slots = kHalf;
    // Hands a piece to the warps of its stream (of both, for a pair).
    auto publish = [&](int kind, int hk, int req, int t0, int t1, int slot, int keys, bool both) {
      for (int s = both ? 0 : i; s <= (both ? 1 : i) && ok; ++s) {
        const int u = 2 * s + (it & 1);
        if (!wait_all(bar_piece_empty0 + 8 * u, ((it >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          slots[u].kind = kind;
          slots[u].hk = hk;
          slots[u].req = req;
          slots[u].t0 = t0;
          slots[u].t1 = t1;
          slots[u].slot = slot;
          slots[u].keys = keys;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_piece_full0 + 8 * u);
      }
      ++it;
    };
    // A piece: its Q rows, then K and V tiles from the last to the first, in
    // the order the MMA warp takes them.
    int q_loads = 0;
    auto run = [&](int kind, int hk, int req, int t0, int t1, int slot, int keys) {
      publish(kind, hk, req, t0, t1, slot, keys, kind == kPair);
      if (!ok || !wait_all(bar_q_empty0 + 8 * i, (q_loads & 1) ^ 1)) {
        ok = false;
        return;
      }
      const int q_rows = kind == kTail ? plan.rows : plan.tile_rows();
      const int copies = kind == kPair ? 2 : Plan::copies(q_rows);
      if (leader) {
        mbar_arrive_expect_tx(bar_q_full0 + 8 * i, copies * L::kBoxes * q_rows * 128);
        // Two row tiles, or the rows of one at every 128 / copies rows.
        for (int u = 0; u < copies; ++u)
#pragma unroll
          for (int bx = 0; bx < L::kBoxes; ++bx)
            tma_load_4d(kind == kPair ? sQ + u * L::kTileBytes + bx * L::kBoxBytes
                                      : sQ + i * L::kTileBytes + bx * L::kBoxBytes + u * (128 / copies) * 128,
                        kind == kTail ? &tm_qt : &tm_qp, bar_q_full0 + 8 * i, bx * 64, 0, hk,
                        kind == kPair ? req + u * plan.tile_reqs : req);
      }
      __syncwarp();
      ++q_loads;
      for (int t = t1 - 1; t >= t0; --t)
        for (int v = 0; v < 2; ++v) {
          const int s = slot0 + idx % n_slots;
          if (!wait_all(bar_kv_empty0 + 8 * s, ((idx / n_slots) & 1) ^ 1)) {
            ok = false;
            return;
          }
          if (leader) {
            const uint32_t full = bar_kv_full0 + 8 * s;
            mbar_arrive_expect_tx(full, L::kTileBytes);
            const CUtensorMap* map = kind == kTail ? (v ? &tm_vt : &tm_kt) : (v ? &tm_vp : &tm_kp);
#pragma unroll
            for (int bx = 0; bx < L::kBoxes; ++bx)
              tma_load_4d(sRing + s * L::kTileBytes + bx * L::kBoxBytes, map, full, bx * 64, t * kBN, hk,
                          kind == kTail ? req : 0);
          }
          __syncwarp();
          ++idx;
        }
    };
    if (static_cast<int>(blockIdx.x) < pair_ctas) {
      if (i == 0) {
        slot0 = 0, n_slots = kStages;
        const int lanes = plan.lanes(pair_ctas), l = blockIdx.x % lanes, c = blockIdx.x / lanes;
        const Cut cut = plan.pair_line(pair_ctas, lanes, l);
        const int u0 = c < cut.parts ? cut.begin(c) : 0, u1 = c < cut.parts ? cut.begin(c + 1) : 0;
        for (int u = u0; u < u1 && ok;) {
          const int s = u / plan.prefix_tiles, t0 = u - s * plan.prefix_tiles;
          const int t1 = min(plan.prefix_tiles, t0 + u1 - u);
          run(kPair, s % plan.Hkv, 2 * (l + s / plan.Hkv * lanes) * plan.tile_reqs, t0, t1,
              Plan::pair_slot(s, c, lanes, l), plan.Np);
          u += t1 - t0;
        }
        if (ok) publish(kEnd, 0, 0, 0, 0, 0, 0, true);
      }
    } else {
      const int singles = plan.ctas - pair_ctas;
      const int start = plan.start_units(tiles);
      const Cut cut = plan.single_line(pair_ctas, tiles, some);
      // Streams of different CTAs are neighbours on the line, so that few units
      // go to many SMs.
      const int c = i * singles + static_cast<int>(blockIdx.x) - pair_ctas;
      const int u0 = c < cut.parts ? cut.begin(c) : 0, u1 = c < cut.parts ? cut.begin(c + 1) : 0;
      int u = u0;
      for (; u < min(u1, plan.odd_units()) && ok;) {
        const int s = u / plan.prefix_tiles, t0 = u - s * plan.prefix_tiles;
        const int t1 = min(plan.prefix_tiles, t0 + u1 - u);
        run(kOdd, s, (plan.row_tiles - 1) * plan.tile_reqs, t0, t1, Plan::single_slot(s, c), plan.Np);
        u += t1 - t0;
      }
      int at = plan.odd_units();  // place of request b0's first unit
      for (int b0 = 0; b0 < plan.B && at < u1 && ok; b0 += 32) {
        const int n = b0 + lane < plan.B ? plan.len(b0 + lane) : 0;
        const int nt = Plan::tiles_of(n);
        const int nu = nt > 0 ? nt + start : 0;
        int upto = nu;  // inclusive scan
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        const int mine0 = at + (upto - nu) * plan.Hkv, mine1 = at + upto * plan.Hkv;
        at += __shfl_sync(0xffffffffu, upto, 31) * plan.Hkv;
        // Requests of these 32 that have a unit in this part.
        unsigned todo = __ballot_sync(0xffffffffu, nu > 0 && mine0 < u1 && mine1 > u0);
        while (todo != 0u && ok) {
          const int k = __ffs(todo) - 1;
          todo &= todo - 1;
          const int a0 = __shfl_sync(0xffffffffu, mine0, k);
          const int kn = __shfl_sync(0xffffffffu, n, k), knt = __shfl_sync(0xffffffffu, nt, k);
          for (int hk = max(u0 - a0, 0) / (knt + start); hk < plan.Hkv && ok; ++hk) {
            const int a = a0 + hk * (knt + start) + start;  // the first tile's place
            if (a >= u1) break;
            if (a + knt > u0)
              run(kTail, hk, b0 + k, max(u0 - a, 0), min(u1 - a, knt),
                  Plan::single_slot(plan.tail_segment(b0 + k, hk), c), kn);
          }
        }
      }
      if (ok) publish(kEnd, 0, 0, 0, 0, 0, 0, false);
    }
    if (!ok) {  // every copy issued has landed before the CTA exits
      if (q_loads > 0) mbar_wait(bar_q_full0 + 8 * i, (q_loads - 1) & 1, nullptr, p.status, kStatusTimeout, lim);
      for (int s = 0; s < n_slots && s < idx; ++s) {
        const int cnt = (idx - s + n_slots - 1) / n_slots;
        mbar_wait(bar_kv_full0 + 8 * (slot0 + s), (cnt - 1) & 1, nullptr, p.status, kStatusTimeout, lim);
      }
    }
    __syncwarp();
  } else if (warp >= R::kMma) {
    setmaxnreg_dec<R::kControlRegs>();
    // ----------------------------------------------------------- MMA issue
    const int me = warp == R::kMma ? 0 : 1;  // stream
    const bool leader = elect_one();
    constexpr uint32_t kIdS = idesc_bf16(128, kBN, false, false);
    constexpr uint32_t kIdPV = idesc_bf16(128, D, false, true);
    constexpr uint64_t kTileDesc = L::kTileBytes >> 4;
    const uint32_t tO0 = tmem + 2 * kBN;
    const uint64_t dQ = sdesc_k_sw128(sQ);
    const uint64_t dK = sdesc_k_sw128(sRing);
    const uint64_t dV = sdesc_mn_sw128(sRing, L::kBoxBytes);
    auto issue_qk = [&](int i, int slot) {
      const uint64_t dq = dQ + i * kTileDesc, dk = dK + slot * kTileDesc;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>(((kk / 4) * L::kBoxBytes + (kk % 4) * 32) >> 4);
        umma_ss(tmem + i * kBN, dq + off, dk + off, kIdS, kk > 0);
      }
      umma_commit(bar_s_full0 + 8 * i);
    };
    auto issue_pv = [&](int i, int slot, bool acc, int part, int steps) {
      const uint64_t dv = dV + slot * kTileDesc;
      constexpr int kPer = kBN / 16 / kPParts;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int kk = part * kPer + u;
        if (kk < steps)
          umma_ts(tO0 + i * D, tmem + i * kBN + kk * 8, dv + static_cast<uint64_t>(kk * 128), kIdPV,
                  (acc || kk > 0) ? 1u : 0u);
      }
    };
    bool ok = true;
    int idx = 0;  // ring position
    int g = 0;    // key tiles so far: phase of the P barriers (the same for both streams of a pair CTA)
    int q_used = 0;
    Piece x = {};
    // A piece, for the streams [i0, i1): constants, see attn_mod.cuh.
    auto work = [&](auto lo, auto hi) {
      constexpr int i0 = decltype(lo)::value, i1 = decltype(hi)::value;
      constexpr bool both = i1 - i0 == 2;
      const int slot0 = both ? 0 : me * kHalf;
      constexpr int n_slots = both ? kStages : kHalf;
      auto take = [&](int& slot) {
        slot = slot0 + idx % n_slots;
        if (!wait_all(bar_kv_full0 + 8 * slot, (idx / n_slots) & 1)) return false;
        ++idx;
        tc_fence_after();
        return true;
      };
      int slot_k = 0, slot_v = 0;
      if (!wait_all(bar_q_full0 + 8 * me, q_used & 1) || !take(slot_k)) {
        ok = false;
        return;
      }
      ++q_used;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int i = i0; i < i1; ++i) issue_qk(i, slot_k);
        umma_commit(bar_kv_empty0 + 8 * slot_k);
        if (x.t1 - 1 == x.t0) umma_commit(bar_q_empty0 + 8 * me);
      }
      __syncwarp();
      for (int t = x.t1 - 1; t >= x.t0 && ok; --t, ++g) {
        if (!take(slot_v)) {
          ok = false;
          break;
        }
        // Keys past a request's length: their weights are 0, but a value left
        // in the cache may be NaN or Inf, so the rows an instruction (16 keys)
        // would still read are cleared, and the rest left out.
        int steps = kBN / 16;
        const int valid = x.keys - t * kBN;
        if (x.kind == kTail && valid < kBN) {
          steps = (valid + 15) / 16;
          const uint32_t v0 = sRing + slot_v * L::kTileBytes;
          const int rows = steps * 16 - valid;
          for (int e = lane; e < rows * 8 * L::kBoxes; e += 32)
            st_shared_v4(v0 + (e / (rows * 8)) * L::kBoxBytes + (valid + (e / 8) % rows) * 128 + (e % 8) * 16, 0u, 0u,
                         0u, 0u);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
#pragma unroll
        for (int i = i0; i < i1; ++i) {
          if (!ok) break;
          if (!wait_all(bar_p_part0 + 8 * i, g & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) issue_pv(i, slot_v, t < x.t1 - 1, 0, steps);
          __syncwarp();
          if (!wait_all(bar_p_full0 + 8 * i, g & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) {
            issue_pv(i, slot_v, true, 1, steps);
            if (t == x.t0) umma_commit(bar_o_full0 + 8 * i);
            if (i == i1 - 1) umma_commit(bar_kv_empty0 + 8 * slot_v);
          }
          __syncwarp();
          if (t > x.t0) {
            if (i == i0 && !take(slot_k)) {
              ok = false;
              break;
            }
            if (leader) {
              issue_qk(i, slot_k);
              if (i == i1 - 1) {
                umma_commit(bar_kv_empty0 + 8 * slot_k);
                if (t - 1 == x.t0) umma_commit(bar_q_empty0 + 8 * me);  // the piece's last Q K^T
              }
            }
            __syncwarp();
          }
        }
      }
    };
    using std::integral_constant;
    for (int it = 0; ok && next_piece(me, it, x, ok); ++it) {
      if (x.kind != kPair && me == 0)
        work(integral_constant<int, 0>{}, integral_constant<int, 1>{});
      else if (x.kind != kPair)
        work(integral_constant<int, 1>{}, integral_constant<int, 2>{});
      else if (me == 0)  // warp 8 issues for both streams
        work(integral_constant<int, 0>{}, integral_constant<int, 2>{});
    }
    // Every MMA issued completes before tensor memory is freed.
    if (leader) umma_commit(bar_drain0 + 8 * me);
    __syncwarp();
    mbar_wait(bar_drain0 + 8 * me, 0, nullptr, p.status, kStatusTimeout, lim);
    __syncwarp();
  } else {
    setmaxnreg_inc<R::kSoftmaxRegs>();
    // ------------------------------------------------------------- softmax
    const int i = warp / 4;
    const int w4 = warp % 4;
    const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t tS = tmem + i * kBN + lane_off;
    const uint32_t tO = tmem + 2 * kBN + i * D + lane_off;
    bool ok = true;
    int g = 0;  // key tiles so far: phase of the S barrier
    Piece x;
    int it = 0;  // pieces so far: phase of the O barrier
    for (; ok && next_piece(i, it, x, ok); ++it) {
      const int req0 = x.kind == kPair ? x.req + i * plan.tile_reqs : x.req;
      const int rows = x.kind == kTail ? plan.rows : min(plan.tile_reqs, plan.B - req0) * plan.rows;
      const int copies = x.kind == kPair ? 1 : Plan::copies(x.kind == kTail ? plan.rows : plan.tile_rows());
      // This warp's rows of the row tile and, with copies, its share of the keys.
      const int per = 4 / copies;  // warps a copy
      const int wr = (w4 % per) * 32, r = wr + lane, kq = w4 / per;
      const bool active = wr < rows, mine = r < rows;
      // The row's request, head and token, its position (in a tail: counted
      // from the tail's start) and the keys it sees.  Rows of the tile that
      // stand for nothing have a maximum no score exceeds, and mask nothing.
      int pos = 0, seen = 0x7fffffff;
      float slope2 = 0.f;
      float m_ref = INFINITY, l = 0.f;
      if (mine) {
        const int rr = r % plan.rows, req = req0 + r / plan.rows;
        m_ref = -INFINITY;
        if (x.kind == kTail) {
          pos = x.keys - plan.Nq + rr % plan.Nq;
          seen = max(pos + 1, 0);
        } else {
          seen = plan.Np;
          if constexpr (kBias) pos = plan.Np + plan.len(req) - plan.Nq + rr % plan.Nq;
        }
        if constexpr (kBias) slope2 = __ldg(p.sm.slopes + x.hk * plan.G + rr / plan.Nq) * 1.4426950408889634f;
      }
      for (int t = x.t1 - 1; t >= x.t0; --t, ++g) {
        const bool got =
            mbar_wait_hint(bar_s_full0 + 8 * i, g & 1, abort_word, p.status, kStatusTimeout, lim, kSuspendHintNs);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        if (!active) {  // no row of this warp's counts: hand over whatever is there
          if (lane == 0) {
            mbar_arrive(bar_p_part0 + 8 * i);
            mbar_arrive(bar_p_full0 + 8 * i);
          }
          continue;
        }
        tc_fence_after();
        const int b = seen - t * kBN;
        const float dist0 = static_cast<float>(pos - t * kBN);
        const bool have_o = t < x.t1 - 1;
        if (copies == 4)
          softmax_share<D, kCap, kBias, 32>(tS, tO, kq, b, dist0, slope2, p.sm, mine, have_o, m_ref, l,
                                            bar_p_part0 + 8 * i, bar_p_full0 + 8 * i, lane);
        else if (copies == 2)
          softmax_share<D, kCap, kBias, 64>(tS, tO, kq, b, dist0, slope2, p.sm, mine, have_o, m_ref, l,
                                            bar_p_part0 + 8 * i, bar_p_full0 + 8 * i, lane);
        else
          softmax_tile<D, kCap, kBias, kCap && !kBias>(tS, tO, 0, b, dist0, slope2, p.sm, mine, have_o, m_ref, l,
                                                       bar_p_part0 + 8 * i, bar_p_full0 + 8 * i, lane);
      }
      if (!ok) break;
      {
        const bool got = mbar_wait(bar_o_full0 + 8 * i, it & 1, abort_word, p.status, kStatusTimeout, lim);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      if (!active) continue;
      const size_t row0 = x.kind == kPair ? static_cast<size_t>(2 * x.slot + i) * plan.tile_rows()
                                          : static_cast<size_t>(x.slot * copies + kq) *
                                                (x.kind == kOdd ? plan.tile_rows() : plan.rows);
      float* o = (x.kind == kPair ? p.pair_o : x.kind == kOdd ? p.odd_o : p.tail_o) + (row0 + wr) * D;
      // The merge takes m = -inf for a part in which the row saw nothing (l = 0).  A
      // maximum skips NaN, so where all scores of a part are NaN m_ref has not
      // moved while l is NaN: such a part gets a finite m, and its l reaches the row.
      if (mine)
        (x.kind == kPair ? p.pair_ml : x.kind == kOdd ? p.odd_ml : p.tail_ml)[row0 + r] =
            make_float2(l == 0.f ? -INFINITY : m_ref == -INFINITY ? 0.f : m_ref, l);
      if (copies > 1)
        store_raw_row<D>(tO, o + lane * D, mine);
      else
        store_raw_rows<D>(tO, base + L::kStageOff + warp * L::kStageWarpBytes, o, rows - wr);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Warps of a merge block.  Eight, which divide a row's partials among them, as long
// as the blocks fit on the GPU at once (four an SM); with more of them four.  From the
// first kernel's end, d = 128: 512 blocks 7.0 us with eight and 11.9 with four, 168
// blocks of 52 partials a row 10.2 and 16.4, 1024 blocks 11.7 and 7.2.
inline int merge_warps(const Plan& plan) {
  return plan.B * plan.Hkv <= 4 * plan.ctas ? kMergeWarps : kMergeWarps / 2;
}

// The columns of a row's O that are not finite once more, from the keys the row sees
// and with weights that sum to one, by its LSE.  The first kernel's matrix products
// multiply zero weights too: those of the keys that belong to another copy of the
// row and those of later tokens, and 0 * Inf is NaN; and weights against a fixed
// reference make large values overflow (cap_top).  A column with a visible value that
// is not finite needs no scores.  Rare and slow (one warp, all the row's keys); nothing
// waits for this kernel with a limit.
template <int D>
__device__ __noinline__ void redo_row(const Params& p, int rr, __nv_bfloat16* o, const float* lse) {
  constexpr int kCols = D / 32;
  const Plan& plan = p.plan;
  const int lane = threadIdx.x % 32;
  const int req = blockIdx.x / plan.Hkv, hk = blockIdx.x % plan.Hkv;
  const bool cap = p.sm.cap_log2 > 0.f, bias = p.sm.slopes != nullptr;
  const int pos = plan.len(req) - plan.Nq + rr % plan.Nq;  // counted from the tail's start
  const float slope2 = bias ? __ldg(p.sm.slopes + hk * plan.G + rr / plan.Nq) * 1.4426950408889634f : 0.f;
  const size_t row = (static_cast<size_t>(req) * plan.Hq + hk * plan.G) * plan.Nq + rr;
  const __nv_bfloat16* q = p.q + row * D;
  const float ref = lse[row] * 1.4426950408889634f;
  o += row * D + lane * kCols;
  unsigned bad = 0u;
#pragma unroll
  for (int u = 0; u < kCols; ++u)
    if (!(fabsf(__bfloat162float(o[u])) < INFINITY)) bad |= 1u << u;
  const __nv_bfloat16* kp = p.kp + hk * p.kp_s[0];
  const __nv_bfloat16* vp = p.vp + hk * p.vp_s[0];
  const __nv_bfloat16* kt = p.kt + req * p.kt_s[0] + hk * p.kt_s[1];
  const __nv_bfloat16* vt = p.vt + req * p.vt_s[0] + hk * p.vt_s[1];
  const int own = min(max(pos + 1, 0), plan.len(req));  // keys of the tail
  unsigned up = 0u, down = 0u;
  scan_values<kCols>(vp, p.vp_s[1], 0, plan.Np, up, down);
  scan_values<kCols>(vt, p.vt_s[2], 0, own, up, down);
  float qv[kCols], acc[kCols] = {};
  load_row_part<kCols>(q + lane * kCols, qv);
  if (__any_sync(0xffffffffu, (bad & ~(up | down)) != 0u)) {
    add_keys<D, kCols, 4>(qv, kp, vp, p.kp_s[1], p.vp_s[1], 0, plan.Np, plan.Np + pos, ref, slope2, p.sm, cap, bias, acc);
    add_keys<D, kCols, 4>(qv, kt, vt, p.kt_s[2], p.vt_s[2], 0, own, pos, ref, slope2, p.sm, cap, bias, acc);
  }
#pragma unroll
  for (int u = 0; u < kCols; ++u) {
    const bool a = (up >> u) & 1u, b = (down >> u) & 1u;
    if ((bad >> u) & 1u) o[u] = __float2bfloat16(a || b ? not_finite(a, b) : acc[u]);
  }
}

// Joins the partial results of every row:
//     M = max_p m_p,  w_p = 2^(m_p - M),  L = sum w_p l_p
//     o = sum w_p o_p / L,  lse = (M + log2 L) ln 2
// One block a (request, K/V head); its rows are dealt to groups of warps, the
// partials of a row to the warps of its group.  The partials lie where the
// kernel above put them: the same lines are cut into the same parts, which one
// warp reckons for its block (all of them doing so took longer than the
// joining: some 15 integer divisions).
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32, 4) shared_merge_kernel(const __grid_constant__ Params p,
                                                                        __nv_bfloat16* o, float* lse) {
  constexpr int kCols = D / 32;
  constexpr int kBatch = 4;  // partial rows a warp has on the way at once; 8 cost a third of the resident blocks
  __shared__ float part_m[kMergeWarps], part_l[kMergeWarps];
  __shared__ float part_o[kMergeWarps][D];
  // Where the partials of this block's rows lie: number k < n_p, of the prefix, in
  // place base_p + k * step_p, the others in place base_t + k - n_p.
  __shared__ int s_pair, s_base_p, s_step_p, s_n_p, s_base_t, s_n_parts;
  const Plan& plan = p.plan;
  const int warps = blockDim.x / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int req = blockIdx.x / plan.Hkv, hk = blockIdx.x % plan.Hkv;

  if (warp == 0) {
    // Key tiles of all tails (under one K/V head) and of those before req, and how
    // many of them have any.
    int all = 0, before = 0, some = 0, some_before = 0;
    for (int b0 = 0; b0 < plan.B; b0 += 128) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int b = b0 + u * 32 + lane;
        if (b >= plan.B) continue;
        const int n = Plan::tiles_of(plan.len(b));
        all += n;
        some += n > 0;
        if (b < req) before += n, some_before += n > 0;
        if (blockIdx.x == 0 && __ldg(plan.tail_lens + b) != plan.len(b)) atomicCAS(p.status, 0, kStatusBadInput);
      }
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    some = __reduce_add_sync(0xffffffffu, some);
    some_before = __reduce_add_sync(0xffffffffu, some_before);

    const Plan::Parts x = plan.parts(req, hk, all, some, before, some_before);
    if (lane == 0) {
      s_pair = x.pair;
      s_base_p = x.base_p;
      s_step_p = x.step_p;
      s_n_p = x.n_p;
      s_base_t = x.base_t;
      s_n_parts = x.n_p + x.n_t;
    }
  }
  __syncthreads();
  const int base_p = s_base_p, step_p = s_step_p, n_p = s_n_p, base_t = s_base_t, n_parts = s_n_parts;
  const float* const p_o = s_pair ? p.pair_o : p.odd_o;
  const float2* const p_ml = s_pair ? p.pair_ml : p.odd_ml;
  const int in_tile = req % plan.tile_reqs * plan.rows;

  // All of the above runs while the other kernel ends; its results are there
  // behind this.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  int group = warps;  // warps a row
  while (group > 1 && group * plan.rows > warps) group /= 2;
  const int wi = warp % group;
  unsigned redo = 0u;  // which of this warp's rows (32 at most: 128 to four warps) to do again
  for (int r0 = 0, it = 0; r0 < plan.rows; r0 += warps / group, ++it) {
    const int rr = r0 + warp / group;
    const bool row_ok = rr < plan.rows;
    // Row of the workspace that holds partial k.
    auto place = [&](int k) {
      return k < n_p ? static_cast<size_t>(base_p + k * step_p) * plan.tile_rows() + in_tile + rr
                     : static_cast<size_t>(base_t + k - n_p) * plan.rows + rr;
    };
    float m = -INFINITY, l = 0.f, acc[kCols];
#pragma unroll
    for (int u = 0; u < kCols; ++u) acc[u] = 0.f;
    for (int k0 = wi; k0 < n_parts && row_ok; k0 += 32 * group) {
      const int k = k0 + lane * group;
      float2 my = make_float2(-INFINITY, 0.f);  // m = -inf, l = 0: a part that saw nothing
      if (k < n_parts) my = __ldcg((k < n_p ? p_ml : p.tail_ml) + place(k));
      float mx = my.x;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float nm = fmaxf(m, mx);
      if (nm == -INFINITY) continue;
      const float w = (my.x == -INFINITY) ? 0.f : exp2f(my.x - nm);
      const float keep = (m == -INFINITY) ? 0.f : exp2f(m - nm);
      m = nm;
      float lw = (my.x == -INFINITY) ? 0.f : w * my.y;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
      l = l * keep + lw;
#pragma unroll
      for (int u = 0; u < kCols; ++u) acc[u] *= keep;
      const int cnt = min(32, (n_parts - k0 + group - 1) / group);
      for (int e0 = 0; e0 < cnt; e0 += kBatch) {
        float we[kBatch], v[kBatch][kCols];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          we[e] = __shfl_sync(0xffffffffu, w, e0 + e);  // 0 behind the last part
#pragma unroll
          for (int u = 0; u < kCols; ++u) v[e][u] = 0.f;
          if (we[e] != 0.f) {  // a part of no weight may hold anything
            const int ke = k0 + (e0 + e) * group;
            const float* s = (ke < n_p ? p_o : p.tail_o) + place(ke) * D;
            if constexpr (D == 128) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(s) + lane);
              v[e][0] = x.x, v[e][1] = x.y, v[e][2] = x.z, v[e][3] = x.w;
            } else {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(s) + lane);
              v[e][0] = x.x, v[e][1] = x.y;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
#pragma unroll
          for (int u = 0; u < kCols; ++u) acc[u] = fmaf(we[e], v[e][u], acc[u]);
      }
    }
    // Warps of a group join through shared memory, in warp order.
    if (group > 1) {
      __syncthreads();
      if (lane == 0) part_m[warp] = m, part_l[warp] = l;
#pragma unroll
      for (int u = 0; u < kCols; ++u) part_o[warp][lane * kCols + u] = acc[u];
      __syncthreads();
      if (wi == 0) {
        float nm = m;
        for (int w = 1; w < group; ++w) nm = fmaxf(nm, part_m[warp + w]);
        const float ref = (nm == -INFINITY) ? 0.f : nm;
        const float keep = exp2f(m - ref);
        l *= keep;
#pragma unroll
        for (int u = 0; u < kCols; ++u) acc[u] *= keep;
        for (int w = 1; w < group; ++w) {
          const float f = exp2f(part_m[warp + w] - ref);
          l = fmaf(f, part_l[warp + w], l);
#pragma unroll
          for (int u = 0; u < kCols; ++u) acc[u] = fmaf(f, part_o[warp + w][lane * kCols + u], acc[u]);
        }
        m = nm;
      }
    }
    if (row_ok && wi == 0) {
      const size_t row = (static_cast<size_t>(req) * plan.Hq + hk * plan.G) * plan.Nq + rr;
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      float top = 0.f;  // the largest magnitude, or NaN
#pragma unroll
      for (int u = 0; u < kCols; ++u) {
        acc[u] *= inv;
        top = max3_nan(top, acc[u], 0.f);
      }
      if constexpr (D == 128) {
        uint2 v;
        v.x = pack_bf16x2(acc[0], acc[1]);
        v.y = pack_bf16x2(acc[2], acc[3]);
        *reinterpret_cast<uint2*>(o + row * D + lane * kCols) = v;
      } else {
        *reinterpret_cast<uint32_t*>(o + row * D + lane * kCols) = pack_bf16x2(acc[0], acc[1]);
      }
      if (lane == 0) lse[row] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      if (__any_sync(0xffffffffu, !(top <= FLT_MAX)) && l <= FLT_MAX) redo |= 1u << it;
    }
  }
  for (; redo != 0u; redo &= redo - 1) {
    __syncwarp();  // o and lse have been written by all lanes
    redo_row<D>(p, (__ffs(redo) - 1) * (warps / group) + warp / group, o, lse);
  }
}

}  // namespace shared
}  // namespace pa
