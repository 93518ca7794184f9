// Attention of a few new tokens of many requests over one shared prefix and each
// request's own tail (pa_attn_shared_prefix) on sm_100a.
//
// Token t of request b (t < Nq) stands at position Np + len_b - Nq + t.  It sees
// all Np prefix keys and the tail keys j <= len_b - Nq + t.  Scores are capped
// and biased as score_mod.cuh says.  The prefix is read once for all requests:
// the rows of all of them (Nq tokens x G query heads a K/V head) are stacked
// into tiles of up to 128 rows.
//
// Work is a line of key tiles (128 keys): first every prefix segment (K/V head x
// pair of row tiles), then every tail segment (request x K/V head).  CTA c of C
// takes the tiles whose place on the line falls in its C-th part, so every SM
// gets the same share whatever the lengths are, without counters or host
// knowledge of them.  The part of a segment that falls to one CTA is a piece;
// segment s and CTA c name it (s + c is different for every piece, since both
// only grow along the line), and with it the place of its partial results:
// normalised fp32 O and LSE rows in the caller's workspace, which
// shared_merge_kernel joins, one row a group of warps, from the same arithmetic.
//
// A piece runs two streams, one a softmax warpgroup, so that one stream's tensor
// work overlaps the other's softmax: with a pair of row tiles each stream takes
// one tile over the same keys; with a single row tile (tails, and the prefix of
// few requests) each stream takes half of the piece's keys and leaves partial
// results of its own.  Warps as in attn_mod.cuh.
//
// Bound: HBM (64 KB of K and V a tile at d = 128) as long as few rows share a
// tile; with several row-tile pairs the prefix becomes tensor and special-
// function work and its re-reads come from L2.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "attn_mod.cuh"
#include "score_mod.cuh"

namespace pa {
namespace shared {

using namespace mod;

constexpr int kMaxCtas = 160;  // sizes the workspace; the grid is one CTA an SM, at most this many
constexpr int kMergeWarps = 8;

// The decomposition of the line, computed alike by the kernel and the merge.
struct Plan {
  int B, Hq, Hkv, G, Nq;
  int rows;          // rows of one request under one K/V head: G * Nq
  int tile_reqs;     // requests in a row tile: 128 / rows, at most B
  int row_tiles;     // ceil(B / tile_reqs)
  int pairs;         // ceil(row_tiles / 2)
  int Np, Nt;
  int prefix_tiles;  // key tiles of the prefix
  int prefix_segs;   // Hkv * pairs, 0 without a prefix
  int ctas;
  const int* tail_lens;

  __host__ __device__ long long prefix_units() const { return static_cast<long long>(prefix_segs) * prefix_tiles; }
  __device__ int len(int b) const { return min(max(__ldg(tail_lens + b), 0), Nt); }
  __device__ static int tiles_of(int keys) { return (keys + kBN - 1) / kBN; }
  // First unit of CTA c's part of a line of `total` units.
  __device__ long long part(long long total, int c) const { return total * c / ctas; }
  // Whether row tile pair `pr` is a single tile (the last one of an odd number).
  __host__ __device__ bool single(int pr) const { return 2 * pr + 1 >= row_tiles; }
};

struct Params {
  Plan plan;
  const __nv_bfloat16* q;
  const __nv_bfloat16* kt;
  const __nv_bfloat16* vt;
  long long kt_s[3], vt_s[3];  // tail strides: batch, head, row (elements)
  float* prefix_o;             // [2 * (prefix_segs + ctas)][tile_reqs * rows][D]
  float* prefix_lse;
  float* tail_o;               // [2 * (B * Hkv + ctas)][rows][D]
  float* tail_lse;
  ScoreMod sm;
  int* status;
  unsigned long long timeout_ns;
};

// A piece as the scheduler hands it out.
struct Piece {
  int kind;   // -1: no more; 0: tail; 1: prefix, one row tile; 2: prefix, two row tiles
  int hk;
  int req;    // tail: the request; prefix: the first row tile
  int t0, t1; // its key tiles
  int slot;   // segment + CTA
  int keys;   // keys of the segment
};

template <int D>
struct SharedLayout {
  static constexpr int kStages = D == 64 ? 8 : 4;  // 128 KB of K and V in flight
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = kQOff + kQTiles * kTileBytes;
  static constexpr int kStageOff = kRingOff + kStages * kTileBytes;
  static constexpr int kStageWarpBytes = 32 * 128;
  static constexpr int kBarOff = kStageOff + 8 * kStageWarpBytes;
  static constexpr int kNumBars = 2 + 2 * kStages + 8 + 1 + 4;
  static constexpr int kPieceOff = kBarOff + kNumBars * 8;
  static constexpr int kTmemSlotOff = kPieceOff + 2 * static_cast<int>(sizeof(Piece));
  static constexpr int kAbortOff = kTmemSlotOff + 4;
  static constexpr int kBytes = kAbortOff + 4;
  static constexpr int kMinOneCtaPerSm = 120 * 1024;
  static constexpr int kAllocBytes = (kBytes + 1024 > kMinOneCtaPerSm) ? (kBytes + 1024) : kMinOneCtaPerSm;
};

template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
    attn_shared_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qt,
                       const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                       const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                       const __grid_constant__ Params p) {
  using L = SharedLayout<D>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);

  const uint32_t sQ = base + L::kQOff;
  const uint32_t sRing = base + L::kRingOff;
  const uint32_t bars = base + L::kBarOff;
  const uint32_t bar_q_full = bars, bar_q_empty = bars + 8;
  const uint32_t bar_kv_full0 = bars + 8 * 2;
  const uint32_t bar_kv_empty0 = bars + 8 * (2 + kStages);
  const uint32_t bar_s_full0 = bars + 8 * (2 + 2 * kStages);
  const uint32_t bar_p_part0 = bars + 8 * (4 + 2 * kStages);
  const uint32_t bar_p_full0 = bars + 8 * (6 + 2 * kStages);
  const uint32_t bar_o_full0 = bars + 8 * (8 + 2 * kStages);
  const uint32_t bar_drain = bars + 8 * (10 + 2 * kStages);
  const uint32_t bar_piece_full0 = bars + 8 * (11 + 2 * kStages);
  const uint32_t bar_piece_empty0 = bars + 8 * (13 + 2 * kStages);
  volatile Piece* slots = reinterpret_cast<volatile Piece*>(gbase + L::kPieceOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kTmemSlotOff);
  volatile int* abort_word = reinterpret_cast<volatile int*>(gbase + L::kAbortOff);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint64_t lim = p.timeout_ns;
  const Plan& plan = p.plan;

  if (threadIdx.x == 0) {
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_kv_full0 + 8 * s, 1);
      mbar_init(bar_kv_empty0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s_full0 + 8 * i, 1);
      mbar_init(bar_p_part0 + 8 * i, 4);  // one arrival per softmax warp
      mbar_init(bar_p_full0 + 8 * i, 4);
      mbar_init(bar_o_full0 + 8 * i, 1);
      mbar_init(bar_piece_full0 + 8 * i, 1);
      mbar_init(bar_piece_empty0 + 8 * i, 10);  // 8 softmax warps, MMA, TMA
    }
    mbar_init(bar_drain, 1);
    *abort_word = 0;
    fence_barrier_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tensormap(&tm_qp);
    prefetch_tensormap(&tm_qt);
    prefetch_tensormap(&tm_kp);
    prefetch_tensormap(&tm_vp);
    prefetch_tensormap(&tm_kt);
    prefetch_tensormap(&tm_vt);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    const bool got = mbar_wait_hint(bar, parity, abort_word, p.status, kStatusTimeout, lim, kSuspendHintNs);
    return __all_sync(0xffffffffu, got);
  };
  auto next_piece = [&](int it, Piece& x, bool& ok) {
    const int s = it & 1;
    if (!wait_all(bar_piece_full0 + 8 * s, (it >> 1) & 1)) {
      ok = false;
      return false;
    }
    x.kind = slots[s].kind;
    x.hk = slots[s].hk;
    x.req = slots[s].req;
    x.t0 = slots[s].t0, x.t1 = slots[s].t1;
    x.slot = slots[s].slot;
    x.keys = slots[s].keys;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_piece_empty0 + 8 * s);
    return x.kind >= 0;
  };
  // Key tiles [a, b) of stream i of a piece: all of them with two row tiles,
  // the lower or the upper half with one.
  auto first_of = [](const Piece& x, int i) { return x.kind == 2 || i == 0 ? x.t0 : x.t0 + (x.t1 - x.t0 + 1) / 2; };
  auto last_of = [](const Piece& x, int i) { return x.kind == 2 || i == 1 ? x.t1 : x.t0 + (x.t1 - x.t0 + 1) / 2; };

  if (warp > kSchedWarp) {
    setmaxnreg_dec<kControlRegs>();
  } else if (warp == kSchedWarp) {
    setmaxnreg_dec<kControlRegs>();
    // ----------------------------------------------------------- scheduler
    int it = 0;
    bool ok = true;
    auto emit = [&](int kind, int hk, int req, int t0, int t1, int slot, int keys) {
      const int s = it & 1;
      if (!wait_all(bar_piece_empty0 + 8 * s, ((it >> 1) & 1) ^ 1)) {
        ok = false;
        return;
      }
      if (lane == 0) {
        slots[s].kind = kind;
        slots[s].hk = hk;
        slots[s].req = req;
        slots[s].t0 = t0;
        slots[s].t1 = t1;
        slots[s].slot = slot;
        slots[s].keys = keys;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_piece_full0 + 8 * s);
      ++it;
    };
    const int c = blockIdx.x;
    // All tail tiles under one K/V head.
    long long tails = 0;
    for (int b = lane; b < plan.B; b += 32) tails += Plan::tiles_of(plan.len(b));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) tails += __shfl_xor_sync(0xffffffffu, tails, off);
    const long long pre = plan.prefix_units();
    const long long total = pre + tails * plan.Hkv;
    const long long u0 = plan.part(total, c), u1 = plan.part(total, c + 1);
    if (u0 < pre) {
      for (int s = static_cast<int>(u0 / plan.prefix_tiles); s < plan.prefix_segs && ok; ++s) {
        const long long at = static_cast<long long>(s) * plan.prefix_tiles;
        if (at >= u1) break;
        const int t0 = static_cast<int>(max(u0 - at, 0ll));
        const int t1 = static_cast<int>(min(u1 - at, static_cast<long long>(plan.prefix_tiles)));
        if (t0 < t1)
          emit(plan.single(s % plan.pairs) ? 1 : 2, s / plan.pairs, 2 * (s % plan.pairs), t0, t1, s + c, plan.Np);
      }
    }
    long long at = pre;  // place of request b0's first tile
    for (int b0 = 0; b0 < plan.B && at < u1 && ok; b0 += 32) {
      const int n = b0 + lane < plan.B ? plan.len(b0 + lane) : 0;
      const int nt = Plan::tiles_of(n);
      int upto = nt;  // inclusive scan
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
      }
      const long long all = static_cast<long long>(__shfl_sync(0xffffffffu, upto, 31)) * plan.Hkv;
      // Requests of these 32 that have a tile in this CTA's part.
      const long long mine0 = at + static_cast<long long>(upto - nt) * plan.Hkv;
      const long long mine1 = mine0 + static_cast<long long>(nt) * plan.Hkv;
      unsigned todo = __ballot_sync(0xffffffffu, nt > 0 && mine0 < u1 && mine1 > u0);
      while (todo != 0u && ok) {
        const int k = __ffs(todo) - 1;
        todo &= todo - 1;
        const long long a0 = __shfl_sync(0xffffffffu, mine0, k);
        const int kn = __shfl_sync(0xffffffffu, n, k), knt = __shfl_sync(0xffffffffu, nt, k);
        for (int hk = static_cast<int>(max(u0 - a0, 0ll) / knt); hk < plan.Hkv && ok; ++hk) {
          const long long a = a0 + static_cast<long long>(hk) * knt;
          if (a >= u1) break;
          const int t0 = static_cast<int>(max(u0 - a, 0ll));
          const int t1 = static_cast<int>(min(u1 - a, static_cast<long long>(knt)));
          if (t0 < t1) emit(0, hk, b0 + k, t0, t1, (b0 + k) * plan.Hkv + hk + c, kn);
        }
      }
      at += all;
    }
    if (ok) emit(-1, 0, 0, 0, 0, 0, 0);
  } else if (warp == kTmaWarp) {
    setmaxnreg_dec<kControlRegs>();
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    bool ok = true;
    int idx = 0;      // ring loads issued so far (over all pieces)
    int q_loads = 0;  // pieces whose Q was issued
    Piece x;
    for (int it = 0; ok && next_piece(it, x, ok); ++it) {
      if (!wait_all(bar_q_empty, (q_loads & 1) ^ 1)) {
        ok = false;
        break;
      }
      if (leader) {
        const int tiles = x.kind == 2 ? 2 : 1;
        const int box_rows = x.kind == 0 ? plan.rows : plan.rows * plan.tile_reqs;
        mbar_arrive_expect_tx(bar_q_full, tiles * L::kBoxes * box_rows * 128);
        for (int i = 0; i < tiles; ++i)
#pragma unroll
          for (int bx = 0; bx < L::kBoxes; ++bx)
            tma_load_4d(sQ + i * L::kTileBytes + bx * L::kBoxBytes, x.kind == 0 ? &tm_qt : &tm_qp, bar_q_full, bx * 64,
                        0, x.hk, x.kind == 0 ? x.req : (x.req + i) * plan.tile_reqs);
      }
      __syncwarp();
      ++q_loads;
      // One K or V tile into the next ring slot.
      auto load = [&](bool is_v, int t) {
        const int s = idx % kStages;
        if (!wait_all(bar_kv_empty0 + 8 * s, ((idx / kStages) & 1) ^ 1)) {
          ok = false;
          return;
        }
        if (leader) {
          const uint32_t full = bar_kv_full0 + 8 * s;
          mbar_arrive_expect_tx(full, L::kTileBytes);
          const CUtensorMap* map = x.kind == 0 ? (is_v ? &tm_vt : &tm_kt) : (is_v ? &tm_vp : &tm_kp);
#pragma unroll
          for (int bx = 0; bx < L::kBoxes; ++bx)
            tma_load_4d(sRing + s * L::kTileBytes + bx * L::kBoxBytes, map, full, bx * 64, t * kBN, x.hk,
                        x.kind == 0 ? x.req : 0);
        }
        __syncwarp();
        ++idx;
      };
      // In the order the MMA warp takes them.
      const int streams = x.kind == 2 ? 1 : 2;
      const int n = last_of(x, 0) - first_of(x, 0);
      for (int i = 0; i < streams && ok; ++i)
        if (first_of(x, i) < last_of(x, i)) load(false, last_of(x, i) - 1);
      for (int j = 0; j < n && ok; ++j)
        for (int i = 0; i < streams && ok; ++i) {
          const int t = last_of(x, i) - 1 - j;
          if (t >= first_of(x, i)) load(true, t);
          if (ok && t - 1 >= first_of(x, i)) load(false, t - 1);
        }
    }
    if (!ok) {  // every copy issued has landed before the CTA exits
      if (q_loads > 0) mbar_wait(bar_q_full, (q_loads - 1) & 1, nullptr, p.status, kStatusTimeout, lim);
      for (int s = 0; s < kStages && s < idx; ++s) {
        const int cnt = (idx - s + kStages - 1) / kStages;
        mbar_wait(bar_kv_full0 + 8 * s, (cnt - 1) & 1, nullptr, p.status, kStatusTimeout, lim);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    setmaxnreg_dec<kControlRegs>();
    // ----------------------------------------------------------- MMA issue
    const bool leader = elect_one();
    constexpr uint32_t kIdS = idesc_bf16(128, kBN, false, false);
    constexpr uint32_t kIdPV = idesc_bf16(128, D, false, true);
    constexpr uint64_t kTileDesc = L::kTileBytes >> 4;
    const uint32_t tO0 = tmem + 2 * kBN;
    const uint64_t dQ = sdesc_k_sw128(sQ);
    const uint64_t dK = sdesc_k_sw128(sRing);
    const uint64_t dV = sdesc_mn_sw128(sRing, L::kBoxBytes);
    auto issue_qk = [&](int i, int q_tile, int slot) {
      const uint64_t dq = dQ + q_tile * kTileDesc, dk = dK + slot * kTileDesc;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>(((kk / 4) * L::kBoxBytes + (kk % 4) * 32) >> 4);
        umma_ss(tmem + i * kBN, dq + off, dk + off, kIdS, kk > 0);
      }
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
    int idx = 0;  // ring position (over all pieces)
    int g0 = 0, g1 = 0;
    int q_used = 0;
    Piece x;
    for (int it = 0; ok && next_piece(it, x, ok); ++it) {
      const bool both = x.kind == 2;  // both streams take the same keys
      int qk_left = (last_of(x, 0) - first_of(x, 0)) + (last_of(x, 1) - first_of(x, 1));
      if (!wait_all(bar_q_full, q_used & 1)) break;
      ++q_used;
      // S of stream i from the K tile in `slot`; the last of the piece frees Q.
      auto qk = [&](int i, int slot) {
        --qk_left;
        if (leader) {
          issue_qk(i, both ? i : 0, slot);
          umma_commit(bar_s_full0 + 8 * i);
          if (!both || i == 1) umma_commit(bar_kv_empty0 + 8 * slot);
          if (qk_left == 0) umma_commit(bar_q_empty);
        }
        __syncwarp();
      };
      int slot_k = 0, slot_v = 0;
      for (int i = 0; i < 2 && ok; ++i) {
        if (first_of(x, i) >= last_of(x, i)) continue;
        if (!both || i == 0) {
          slot_k = idx % kStages;
          if (!wait_all(bar_kv_full0 + 8 * slot_k, (idx / kStages) & 1)) {
            ok = false;
            break;
          }
          ++idx;
          tc_fence_after();
        }
        qk(i, slot_k);
      }
      const int n = last_of(x, 0) - first_of(x, 0);
      for (int j = 0; j < n && ok; ++j)
        for (int i = 0; i < 2 && ok; ++i) {
          const int t = last_of(x, i) - 1 - j;
          if (t < first_of(x, i)) continue;
          if (!both || i == 0) {
            slot_v = idx % kStages;
            if (!wait_all(bar_kv_full0 + 8 * slot_v, (idx / kStages) & 1)) {
              ok = false;
              break;
            }
            ++idx;
          }
          // Keys past the request's length: their weights are 0, but a value
          // left in the cache may be NaN or Inf, so the rows an instruction
          // (16 keys) would still read are cleared, and the rest left out.
          int steps = kBN / 16;
          const int valid = x.keys - t * kBN;
          if (x.kind == 0 && valid < kBN) {
            steps = (valid + 15) / 16;
            const uint32_t v0 = sRing + slot_v * L::kTileBytes;
            const int rows = steps * 16 - valid;
            for (int e = lane; e < rows * 8 * L::kBoxes; e += 32)
              st_shared_v4(v0 + (e / (rows * 8)) * L::kBoxBytes + (valid + (e / 8) % rows) * 128 + (e % 8) * 16, 0u, 0u,
                           0u, 0u);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          const uint32_t ph = (i ? g1 : g0) & 1;
          if (!wait_all(bar_p_part0 + 8 * i, ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) issue_pv(i, slot_v, j > 0, 0, steps);
          __syncwarp();
          if (!wait_all(bar_p_full0 + 8 * i, ph)) {
            ok = false;
            break;
          }
          i ? ++g1 : ++g0;
          tc_fence_after();
          if (leader) {
            issue_pv(i, slot_v, true, 1, steps);
            if (t == first_of(x, i)) umma_commit(bar_o_full0 + 8 * i);
            if (!both || i == 1) umma_commit(bar_kv_empty0 + 8 * slot_v);
          }
          __syncwarp();
          if (t > first_of(x, i)) {
            if (!both || i == 0) {
              slot_k = idx % kStages;
              if (!wait_all(bar_kv_full0 + 8 * slot_k, (idx / kStages) & 1)) {
                ok = false;
                break;
              }
              ++idx;
              tc_fence_after();
            }
            qk(i, slot_k);
          }
        }
    }
    // Every MMA issued completes before tensor memory is freed.
    if (leader) umma_commit(bar_drain);
    __syncwarp();
    mbar_wait(bar_drain, 0, nullptr, p.status, kStatusTimeout, lim);
    __syncwarp();
  } else {
    setmaxnreg_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------- softmax
    const int i = warp / 4;
    const int r = threadIdx.x % 128;  // row of the row tile
    const int wr = r - lane;          // first row of this warp
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tS = tmem + i * kBN + lane_off;
    const uint32_t tO = tmem + 2 * kBN + i * D + lane_off;
    bool ok = true;
    int g = 0;    // key tiles over all pieces: phases of the S barrier
    int n_o = 0;  // pieces with key tiles of this stream: phase of the O barrier
    Piece x;
    for (int it = 0; ok && next_piece(it, x, ok); ++it) {
      const int first = first_of(x, i), last = last_of(x, i);
      if (first >= last) continue;
      const int req0 = x.kind == 0 ? x.req : (x.req + (x.kind == 2 ? i : 0)) * plan.tile_reqs;
      const int rows = x.kind == 0 ? plan.rows : min(plan.tile_reqs, plan.B - req0) * plan.rows;
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
        if (x.kind == 0) {
          pos = x.keys - plan.Nq + rr % plan.Nq;
          seen = max(pos + 1, 0);
        } else {
          seen = plan.Np;
          if constexpr (kBias) pos = plan.Np + plan.len(req) - plan.Nq + rr % plan.Nq;
        }
        if constexpr (kBias) slope2 = __ldg(p.sm.slopes + x.hk * plan.G + rr / plan.Nq) * 1.4426950408889634f;
      }
      for (int t = last - 1; t >= first; --t, ++g) {
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
        const int k0 = t * kBN;
        softmax_tile<D, kCap, kBias>(tS, tO, 0, seen - k0, static_cast<float>(pos - k0), slope2, p.sm, t < last - 1,
                                     m_ref, l, bar_p_part0 + 8 * i, bar_p_full0 + 8 * i, lane);
      }
      if (!ok) break;
      {
        const bool got = mbar_wait(bar_o_full0 + 8 * i, n_o & 1, abort_word, p.status, kStatusTimeout, lim);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        ++n_o;
        tc_fence_after();
      }
      if (!active) continue;
      const bool empty = !mine || m_ref == -INFINITY;
      const float inv = empty ? 0.f : 1.f / l;
      const size_t row0 = x.kind == 0 ? static_cast<size_t>(2 * x.slot + i) * plan.rows
                                      : static_cast<size_t>(2 * x.slot + i) * (plan.tile_reqs * plan.rows);
      float* o = (x.kind == 0 ? p.tail_o : p.prefix_o) + (row0 + wr) * D;
      const bool bad =
          store_rows<D>(tO, base + L::kStageOff + warp * L::kStageWarpBytes, nullptr, o, D, rows - wr, inv);
      if (mine)
        (x.kind == 0 ? p.tail_lse : p.prefix_lse)[row0 + r] =
            empty ? -INFINITY : (m_ref + lg2_approx(l)) * 0.69314718055994531f;
      // A value row that is not finite among the new tokens of a request does
      // not reach the tokens before it (see repair_row).
      if (x.kind == 0 && plan.Nq > 1) {
        unsigned redo = __ballot_sync(0xffffffffu, bad && !empty && l <= FLT_MAX);
        while (redo != 0u) {
          const int k = __ffs(redo) - 1;
          redo &= redo - 1;
          __syncwarp();
          const int j0 = first * kBN, j1 = min(__shfl_sync(0xffffffffu, seen, k), last * kBN);
          const int ps = __shfl_sync(0xffffffffu, pos, k);
          const float mr = __shfl_sync(0xffffffffu, m_ref, k), iv = __shfl_sync(0xffffffffu, inv, k);
          const float sl = __shfl_sync(0xffffffffu, slope2, k);
          const size_t q_row =
              (static_cast<size_t>(x.req) * plan.Hq + x.hk * plan.G) * plan.Nq + wr + k;  // rows of a K/V head are adjacent
          repair_row<D>(p.q + q_row * D, p.kt + x.req * p.kt_s[0] + x.hk * p.kt_s[1],
                        p.vt + x.req * p.vt_s[0] + x.hk * p.vt_s[1], p.kt_s[2], p.vt_s[2], j0, j1, ps, mr, iv, sl, p.sm,
                        kCap, kBias, nullptr, o + k * D);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partial results of every row, as pa_attn_merge defines it:
//     M = max_p lse_p,  w_p = exp(lse_p - M),  o = sum w_p o_p / sum w_p
// One block a (request, K/V head); its rows are dealt to groups of warps, the
// partials of a row to the warps of its group.  The partials lie where the
// kernel above put them: the same line is cut into the same parts.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(const __grid_constant__ Params p,
                                                                        __nv_bfloat16* o, float* lse) {
  constexpr int kCols = D / 32;
  __shared__ long long sums[2][kMergeWarps];
  __shared__ float part_m[kMergeWarps], part_l[kMergeWarps];
  __shared__ float part_o[kMergeWarps][D];
  const Plan& plan = p.plan;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int req = blockIdx.x / plan.Hkv, hk = blockIdx.x % plan.Hkv;

  // Tail tiles (under one K/V head) of all requests, and of those before req.
  long long all = 0, before = 0;
  for (int b = threadIdx.x; b < plan.B; b += kMergeWarps * 32) {
    const int n = Plan::tiles_of(plan.len(b));
    all += n;
    if (b < req) before += n;
    if (blockIdx.x == 0 && __ldg(plan.tail_lens + b) != plan.len(b)) atomicCAS(p.status, 0, kStatusBadInput);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  if (lane == 0) sums[0][warp] = all, sums[1][warp] = before;
  __syncthreads();
  all = before = 0;
  for (int w = 0; w < kMergeWarps; ++w) all += sums[0][w], before += sums[1][w];

  const int n_tail = Plan::tiles_of(plan.len(req));
  const long long total = plan.prefix_units() + all * plan.Hkv;
  const int mt = req / plan.tile_reqs;
  const int seg_p = hk * plan.pairs + mt / 2, seg_t = req * plan.Hkv + hk;
  const bool single = plan.single(mt / 2);
  const long long at_p = static_cast<long long>(seg_p) * plan.prefix_tiles;
  const long long at_t = plan.prefix_units() + before * plan.Hkv + static_cast<long long>(hk) * n_tail;
  // CTAs that hold the units [at, at + n) of the line: [c0, c1).
  auto holders = [&](long long at, long long n, int& c0, int& c1) {
    auto holder = [&](long long u) {
      int c = static_cast<int>(u * plan.ctas / total);
      while (plan.part(total, c + 1) <= u) ++c;
      while (plan.part(total, c) > u) --c;
      return c;
    };
    c0 = c1 = 0;
    if (n > 0) c0 = holder(at), c1 = holder(at + n - 1) + 1;
  };
  int p0, p1, t0, t1;
  holders(at_p, plan.prefix_segs ? plan.prefix_tiles : 0, p0, p1);
  holders(at_t, n_tail, t0, t1);
  const int streams_p = single ? 2 : 1;
  const int n_p = (p1 - p0) * streams_p, n_parts = n_p + (t1 - t0) * 2;

  int group = kMergeWarps;  // warps a row
  while (group > 1 && group * plan.rows > kMergeWarps) group /= 2;
  const int wi = warp % group;
  for (int r0 = 0; r0 < plan.rows; r0 += kMergeWarps / group) {
    const int rr = r0 + warp / group;
    const bool row_ok = rr < plan.rows;
    float m = -INFINITY, l = 0.f, acc[kCols];
#pragma unroll
    for (int u = 0; u < kCols; ++u) acc[u] = 0.f;
    for (int k0 = 0; k0 < n_parts && row_ok; k0 += 32 * group) {
      const int k = k0 + lane * group + wi;
      const float* src = nullptr;
      float my = -INFINITY;
      if (k < n_parts) {
        const bool pre = k < n_p;
        const int q = pre ? k : k - n_p, st = pre ? streams_p : 2;
        const int c = (pre ? p0 : t0) + q / st;
        const long long at = pre ? at_p : at_t;
        const int n_seg = pre ? plan.prefix_tiles : n_tail;
        // The piece's tiles; its second stream has the smaller half.
        const long long a = max(plan.part(total, c) - at, 0ll);
        const long long b = min(plan.part(total, c + 1) - at, static_cast<long long>(n_seg));
        const int i = pre && !single ? (mt & 1) : q % st;
        const long long n = pre && !single ? b - a : (i == 0 ? (b - a + 1) / 2 : (b - a) / 2);
        if (n > 0) {
          const size_t row = pre ? static_cast<size_t>(2 * (seg_p + c) + i) * (plan.tile_reqs * plan.rows) +
                                       (req % plan.tile_reqs) * plan.rows + rr
                                 : static_cast<size_t>(2 * (seg_t + c) + i) * plan.rows + rr;
          my = __ldcg((pre ? p.prefix_lse : p.tail_lse) + row);
          src = (pre ? p.prefix_o : p.tail_o) + row * D;
        }
      }
      float mx = my;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float nm = fmaxf(m, mx);
      if (nm == -INFINITY && !__any_sync(0xffffffffu, my != my)) continue;
      const float w = (my == -INFINITY) ? 0.f : expf(my - nm);
      const float keep = (m == -INFINITY) ? 0.f : expf(m - nm);
      m = nm;
      float lw = w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
      l = l * keep + lw;
#pragma unroll
      for (int u = 0; u < kCols; ++u) acc[u] *= keep;
      const int cnt = min(32, (n_parts - k0 - wi + group - 1) / group);
#pragma unroll 4
      for (int e = 0; e < cnt; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, e);
        const float* s = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), e));
        if (we != 0.f) {
          if constexpr (D == 128) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + lane);
            acc[0] = fmaf(we, v.x, acc[0]);
            acc[1] = fmaf(we, v.y, acc[1]);
            acc[2] = fmaf(we, v.z, acc[2]);
            acc[3] = fmaf(we, v.w, acc[3]);
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(s) + lane);
            acc[0] = fmaf(we, v.x, acc[0]);
            acc[1] = fmaf(we, v.y, acc[1]);
          }
        }
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
        const float base = (nm == -INFINITY) ? 0.f : nm;
        const float keep = expf(m - base);
        l *= keep;
#pragma unroll
        for (int u = 0; u < kCols; ++u) acc[u] *= keep;
        for (int w = 1; w < group; ++w) {
          const float f = expf(part_m[warp + w] - base);
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
      if constexpr (D == 128) {
        uint2 v;
        v.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        v.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2*>(o + row * D + lane * kCols) = v;
      } else {
        *reinterpret_cast<uint32_t*>(o + row * D + lane * kCols) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
      }
      if (lane == 0) lse[row] = none ? -INFINITY : m + logf(l);
    }
  }
}

}  // namespace shared
}  // namespace pa
