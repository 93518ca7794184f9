// Attention with modified scores and interval masks (pa_attn_fwd_mod) on sm_100a.
//
// Row i of the call stands at position p_i = i + q_offset among the keys and
// sees one interval [lo_i, hi_i) of them:
//     no mask      [0, Nk)
//     causal       [0, max(p_i + 1, prefix))
//     documents    [start, end) of the document that holds p_i, and with
//                  causal [start, min(end, max(p_i + 1, start + prefix)))
// Scores are capped and biased as score_mod.cuh says.  A row that sees nothing
// gets O = 0 and LSE = -inf.
//
// Work: an item is 256 query rows (two tiles of 128) of one (batch, head); only
// the key tiles that some row of a tile sees are loaded, and a query tile takes
// part only in those its own rows see.  The grid has a block for every item.  A
// CTA works on its own block's item and then takes over blocks that have not
// started (cluster launch control), one ahead: the longest items, the last query
// rows under a causal mask, come first and the short ones fill up the end
// (4096 causal keys, 24 heads: 111 us, 127 us with a fixed share a CTA).  Warps:
//   0-3, 4-7   softmax of query tile 0 and 1, a row a thread (208 registers)
//   8          tcgen05.mma issue      9   TMA loads (Q of the item, K/V ring)
//   10         scheduler: the next item, its intervals' hull per query tile and
//              the documents it spans, through a slot in shared memory that is
//              free once all other warps have begun the item before
//   11         idle (completes the register split's warpgroup)
// Key tiles are walked from the last to the first: the nearest keys come
// first, so a bias that falls with distance settles the row maximum at once
// instead of moving it with every tile.
// Tensor memory and shared memory are laid out as in attn_fwd.cuh.
//
// With kWide (capped scores with the fixed reference, score_mod.cuh) two
// warpgroups share a query tile, the lower and the upper 64 keys of every tile, a
// row a thread in both: warps 0-7 and 8-15, the others at 16-19.  Four warps a
// scheduler instead of two keep its pipes busier: 37 heads x 4096 x 4096 capped
// 350 us, 471 us with one warpgroup a query tile.  Without the fixed reference
// both threads of a row would have to agree on a maximum for every tile, which
// costs more than it gains (4096 keys, 24 heads: 207 us against 181).
//
// Bound: the chain from a tile's scores to its weights, which the tensor pipe waits
// for (4608 x 4608 keys unmasked, 24 heads: 216 us, 0.73 of the matrix rate, where the
// plain forward takes 196 us, 0.80; which of the 4-D maps, the claimed items, the
// order of issue and 40 bytes of spilled registers it owes that to has not been
// measured); with a cap the FMA pipe, on which the polynomial runs (8192 capped
// causal keys, 24 heads: 421 us, FMA 56 % busy, special-function unit and tensor
// pipe 47 %); with short documents an item's start and end, some 8 000 clocks beside
// the 5 000 to 7 500 of a tile that the mask cuts (8192 keys in 24 documents, 24
// heads, biased: 109 us, tensor pipe 25 % busy); with fewer items than SMs the
// longest item, 2.2 us a key tile however few its rows (1 row of 24 heads on 8192
// keys: 107 us, its bytes 5).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "score_mod.cuh"

namespace pa {
namespace mod {

constexpr int kStages = 4;
// Warps and registers.  The split (see attn_fwd.cuh): three warpgroups of 168 at
// launch, two of 208 and one of 88 then; wide, five of 96, then four of 104 and
// one of 64.
template <bool kWide>
struct Roles {
  static constexpr int kGroups = kWide ? 4 : 2;  // softmax warpgroups
  static constexpr int kMma = 4 * kGroups, kTma = kMma + 1, kSched = kMma + 2;
  static constexpr int kThreads = 128 * (kGroups + 1);
  static constexpr int kLaunchRegs = kWide ? 96 : 168;
  static constexpr int kSoftmaxRegs = kWide ? 104 : 208;
  static constexpr int kControlRegs = kWide ? 64 : 88;
  static_assert(kControlRegs + kGroups * kSoftmaxRegs == (kGroups + 1) * kLaunchRegs,
                "register split must sum to the launch allocation");
};

struct FwdModParams {
  __nv_bfloat16* o;
  float* lse;  // [B, Hq, Nq]
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long q_s[3], k_s[3], v_s[3], o_s[3];  // element strides: batch, head, row
  int B, Hq, G;                              // G = Hq / Hkv
  int Nq, Nk;
  int items, blocks_per_bh;
  bool by_order;  // items in PairOrder's order
  int q_offset;
  int causal;
  const int* prefix;  // [B, max(n_docs, 1)] or null
  const int* docs;    // [B, n_docs + 1] or null
  int n_docs;
  ScoreMod sm;
  int* status;
  unsigned long long timeout_ns;
};

// Index of the last of off[0 .. n] that is <= pos, looked for in [t0, t1]
// (t0 is returned where none above it is; -1 stands for "none").
__device__ __forceinline__ int find_doc(const int* off, int pos, int t0, int t1) {
  while (t0 < t1) {
    const int t = t0 + (t1 - t0 + 1) / 2;
    if (__ldg(off + t) <= pos)
      t0 = t;
    else
      t1 = t - 1;
  }
  return t0;
}

// Keys [x, y) that the row at `pos` of batch b sees, its document being t.
__device__ __forceinline__ int2 row_interval(const FwdModParams& p, int b, int pos, int t) {
  int lo = 0, hi = p.Nk, pre = 0;
  if (p.docs != nullptr) {
    if (t < 0 || t >= p.n_docs) return make_int2(0, 0);
    const int* off = p.docs + static_cast<long long>(b) * (p.n_docs + 1) + t;
    lo = min(max(__ldg(off), 0), p.Nk);
    hi = min(max(__ldg(off + 1), lo), p.Nk);
    if (p.prefix != nullptr) pre = __ldg(p.prefix + static_cast<long long>(b) * p.n_docs + t);
  } else if (p.prefix != nullptr) {
    pre = __ldg(p.prefix + b);
  }
  if (p.causal) {
    pre = min(max(pre, 0), p.Nk);
    hi = max(lo, min(hi, max(pos + 1, lo + pre)));
  }
  return make_int2(lo, hi);
}

// With documents, the (row block, batch) pairs in the order of the keys their rows
// span, the most first, so that the long items start first whatever the documents
// are.  Every scheduler reckons the same order: lane l holds the ranks of pairs
// l, l + 32, ..  Without and with it, 24 heads: 8192 keys in 24 documents 115 and
// 110 us, seen in both directions 181 and 164, in 8 documents 174 and 161, 2 x 4603
// keys in 3 documents 272 and 234.  Ranking takes a microsecond or two at the start,
// which it does not give back with
//  - more than kMax pairs: there are many items a CTA then (128 pairs: 400 and 404)
//  - fewer than two items an SM (192 items: 33 and 35)
//  - more documents than row blocks: items are much alike (96 documents on 32
//    blocks: 83 and 85).
struct PairOrder {
  static constexpr int kPer = 2, kMax = 32 * kPer;
  static bool pays(int pairs, int blocks, int n_docs, int items, int sms) {
    return n_docs > 0 && pairs <= kMax && items >= 2 * sms && n_docs <= blocks;
  }
  int rank[kPer];

  __device__ __forceinline__ void reckon(const FwdModParams& p, int pairs) {
    const int lane = threadIdx.x % 32;
    int key[kPer];  // the pair's key tiles, then its place from the end: no two alike
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = u * 32 + lane;
      key[u] = -1;
      rank[u] = e < pairs ? 0 : -1;
      if (e >= pairs) continue;
      const int b = e % p.B, row0 = (p.blocks_per_bh - 1 - e / p.B) * (kQTiles * kBM);
      const int pos0 = row0 + p.q_offset, pos1 = min(row0 + kQTiles * kBM, p.Nq) - 1 + p.q_offset;
      const int* off = p.docs + static_cast<long long>(b) * (p.n_docs + 1);
      const int t0 = find_doc(off, pos0, -1, p.n_docs), t1 = find_doc(off, pos1, t0, p.n_docs);
      key[u] = kMax - 1 - e;
      if (t1 < 0 || t0 >= p.n_docs) continue;
      const int lo = row_interval(p, b, pos0, max(t0, 0)).x;
      const int hi = row_interval(p, b, pos1, min(t1, p.n_docs - 1)).y;
      key[u] += max(hi - lo, 0) / kBN * kMax;
    }
#pragma unroll
    for (int v = 0; v < kPer; ++v) {
      if (v * 32 >= pairs) break;
#pragma unroll 8
      for (int l = 0; l < 32; ++l) {
        const int other = __shfl_sync(0xffffffffu, key[v], l);
#pragma unroll
        for (int u = 0; u < kPer; ++u)
          if (key[u] >= 0) rank[u] += other > key[u];
      }
    }
  }
  // The item in the n-th place, heads of a pair side by side.
  __device__ __forceinline__ int item(int n, int Hq) const {
    const int g = n / Hq;
    int e = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const unsigned at = __ballot_sync(0xffffffffu, rank[u] == g);
      if (at != 0u) e = u * 32 + __ffs(at) - 1;
    }
    return e * Hq + n % Hq;
  }
};

// What the scheduler tells the other warps about an item (item < 0: no more).
struct ItemSlot {
  int item;
  int first[2], last[2];  // key tiles [first, last) of query tile 0 and 1
  int end;                // no row of the item sees a key at `end` or behind it
  int doc0, doc1;         // documents of the item's first and last row
};

// Cluster launch control: ask for a block of this grid that has not started, to
// work on it here.  The answer (16 bytes) is written to `resp` and counted on
// `bar`; no further request may follow one that came back empty.
__device__ __forceinline__ void clc_request(uint32_t resp, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(resp),
      "r"(bar)
      : "memory");
}

// The block of an answer, or -1.
__device__ __forceinline__ int clc_block(uint32_t resp) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}\n"
      : "=r"(x)
      : "r"(resp)
      : "memory");
  return x;
}

template <int D, bool kWide>
struct Layout {
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = kQOff + kQTiles * kTileBytes;
  static constexpr int kStageOff = kRingOff + kStages * kTileBytes;
  static constexpr int kStageWarpBytes = kWide ? 32 * 32 : 32 * 64;
  // Wide: what the two threads of a row tell each other at the end, the sums of
  // their weights; [two slots in turn][query tile][key half][row].
  static constexpr int kSumOff = kStageOff + Roles<kWide>::kGroups * 4 * kStageWarpBytes;
  static constexpr int kBarOff = kSumOff + (kWide ? 2 * 2 * 2 * 128 * 4 : 0);
  // q_full, q_empty, kv_full[S], kv_empty[S], s_full[2], p_part[2], p_full[2],
  // o_full[2], drain, item_full, item_empty, claim, swap[2][4 warps]
  static constexpr int kNumBars = 2 + 2 * kStages + 8 + 1 + 3 + 8;
  static constexpr int kClaimOff = kBarOff + kNumBars * 8;  // a claim's answer, 16 bytes
  static_assert(kClaimOff % 16 == 0, "the answer's place must be 16-byte aligned");
  static constexpr int kItemOff = kClaimOff + 16;
  static constexpr int kTmemSlotOff = kItemOff + static_cast<int>(sizeof(ItemSlot));
  static constexpr int kAbortOff = kTmemSlotOff + 4;
  static constexpr int kBytes = kAbortOff + 4;
  // Never two CTAs an SM: each takes all of tensor memory.
  static constexpr int kMinOneCtaPerSm = 120 * 1024;
  static constexpr int kAllocBytes = (kBytes + 1024 > kMinOneCtaPerSm) ? (kBytes + 1024) : kMinOneCtaPerSm;
};

// Rows `redo` of a warp once more, those of their columns in o that are not finite.
// The tensor cores multiply the zero weight of a hidden key with its value row, so
// a hidden value that is NaN or Inf reaches the accumulator; and under a fixed
// reference large values overflow it (cap_top).  Here a row takes only the keys
// [lo, hi) it sees, with weights that sum to one: ref is the log2 of the sum the
// softmax found (hidden scores never entered that).  A column with a visible value
// that is not finite needs no scores; what all rows see is looked through once for
// all of them.  lo, hi, ref: of the lane's own row; q, o: the warp's first row; k, v:
// row 0 of its head; pos: the first row's position.  kCols of the value columns
// are computed, those from v and o on.  NaN hidden from the last row block of 4096
// causal keys, 24 heads, d 128: 10 ms in all (0.12 without); visible, at every 128th
// key: 0.47 ms.
template <int D, int kCols>
__device__ __noinline__ void repair_rows(unsigned redo, const __nv_bfloat16* q, long long q_stride,
                                         const __nv_bfloat16* k, const __nv_bfloat16* v, long long k_stride,
                                         long long v_stride, int lo, int hi, int pos, float ref, float slope2,
                                         const ScoreMod& sm, bool cap, bool bias, __nv_bfloat16* o, long long o_stride) {
  constexpr int kQk = D / 32, kV = kCols / 32;
  const int lane = threadIdx.x % 32;
  const bool mine = (redo >> lane) & 1u;
  __syncwarp();  // o has been written by all lanes
  const int all0 = __reduce_max_sync(0xffffffffu, mine ? lo : 0);
  const int all1 = max(all0, __reduce_min_sync(0xffffffffu, mine ? hi : 0x7fffffff));
  unsigned all_up = 0u, all_down = 0u;
  scan_values<kV>(v, v_stride, all0, all1, all_up, all_down);
  for (; redo != 0u; redo &= redo - 1) {
    const int r = __ffs(redo) - 1;
    const int j0 = __shfl_sync(0xffffffffu, lo, r), j1 = __shfl_sync(0xffffffffu, hi, r);
    const float rr = __shfl_sync(0xffffffffu, ref, r);
    unsigned up = all_up, down = all_down;
    scan_values<kV>(v, v_stride, j0, min(all0, j1), up, down);
    scan_values<kV>(v, v_stride, max(all1, j0), j1, up, down);
    __nv_bfloat16* dst = o + r * o_stride + lane * kV;
    unsigned bad = 0u;
#pragma unroll
    for (int u = 0; u < kV; ++u)
      if (!(fabsf(__bfloat162float(dst[u])) < INFINITY)) bad |= 1u << u;
    float acc[kV] = {};
    if (__any_sync(0xffffffffu, (bad & ~(up | down)) != 0u)) {
      float qv[kQk];
      load_row_part<kQk>(q + r * q_stride + lane * kQk, qv);
      add_keys<D, kV>(qv, k, v, k_stride, v_stride, j0, j1, pos + r, rr, slope2, sm, cap, bias, acc);
    }
#pragma unroll
    for (int u = 0; u < kV; ++u) {
      const bool a = (up >> u) & 1u, b = (down >> u) & 1u;
      if ((bad >> u) & 1u) dst[u] = __float2bfloat16(a || b ? not_finite(a, b) : acc[u]);
    }
  }
}

template <int D, bool kCap, bool kBias, bool kWide>
__global__ void __launch_bounds__(Roles<kWide>::kThreads, 1)
    attn_mod_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ FwdModParams p) {
  static_assert(!kWide || (kCap && !kBias), "the fixed reference is for capped scores without a bias");
  using L = Layout<D, kWide>;
  using R = Roles<kWide>;
  constexpr int kPOff = kWide ? 64 : 32;  // columns from a tile's first weights to those of its upper 64 keys
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
  const uint32_t bar_item_full = bars + 8 * (11 + 2 * kStages);
  const uint32_t bar_item_empty = bars + 8 * (12 + 2 * kStages);
  const uint32_t bar_claim = bars + 8 * (13 + 2 * kStages);
  const uint32_t bar_swap0 = bars + 8 * (14 + 2 * kStages);  // + 8 * (4 * query tile + warp of the warpgroup)
  volatile ItemSlot* slot = reinterpret_cast<volatile ItemSlot*>(gbase + L::kItemOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kTmemSlotOff);
  volatile int* abort_word = reinterpret_cast<volatile int*>(gbase + L::kAbortOff);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint64_t lim = p.timeout_ns;

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
    }
    mbar_init(bar_item_full, 1);
    mbar_init(bar_item_empty, 4 * R::kGroups + 2);  // softmax warps, MMA, TMA
    mbar_init(bar_claim, 1);
    mbar_init(bar_drain, 1);
    for (int u = 0; u < 8; ++u) mbar_init(bar_swap0 + 8 * u, 2);  // the two warps of the same rows
    *abort_word = 0;
    fence_barrier_init();
  }
  if (warp == R::kTma && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == R::kMma) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // The scheduler reckons while the barriers and tensor memory are set up.
  PairOrder order;
  if (warp == R::kSched && p.by_order) order.reckon(p, p.blocks_per_bh * p.B);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    const bool got = mbar_wait_hint(bar, parity, abort_word, p.status, kStatusTimeout, lim, kSuspendHintNs);
    return __all_sync(0xffffffffu, got);
  };
  // The it-th item of this CTA, copied out of the slot; false at the end (or
  // where a wait gave up, with `ok` cleared).
  auto next_item = [&](int it, ItemSlot& x, bool& ok) {
    if (!wait_all(bar_item_full, it & 1)) {
      ok = false;
      return false;
    }
    x.item = slot->item;
    x.first[0] = slot->first[0], x.first[1] = slot->first[1];
    x.last[0] = slot->last[0], x.last[1] = slot->last[1];
    x.end = slot->end;
    x.doc0 = slot->doc0, x.doc1 = slot->doc1;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_item_empty);
    return x.item >= 0;
  };
  auto first_of = [](const ItemSlot& x, int i) { return i ? x.first[1] : x.first[0]; };
  auto last_of = [](const ItemSlot& x, int i) { return i ? x.last[1] : x.last[0]; };
  // Key tiles of an item: the hull of its query tiles' ranges.
  auto hull = [](const ItemSlot& x, int& a, int& b) {
    const bool has0 = x.first[0] < x.last[0], has1 = x.first[1] < x.last[1];
    a = has0 && has1 ? min(x.first[0], x.first[1]) : has0 ? x.first[0] : x.first[1];
    b = has0 && has1 ? max(x.last[0], x.last[1]) : has0 ? x.last[0] : x.last[1];
  };

  if (warp > R::kSched) {
    setmaxnreg_dec<R::kControlRegs>();
  } else if (warp == R::kSched) {
    setmaxnreg_dec<R::kControlRegs>();
    // ----------------------------------------------------------- scheduler
    const uint32_t answer = base + L::kClaimOff;
    int item = static_cast<int>(blockIdx.x);
    for (int it = 0;; ++it) {
      if (!wait_all(bar_item_empty, (it & 1) ^ 1)) break;
      if (it > 0) {
        if (lane == 0) {
          // The answer before has been read (by this warp) when it is written over.
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive_expect_tx(bar_claim, 16);
          clc_request(answer, bar_claim);
        }
        __syncwarp();
        if (!wait_all(bar_claim, (it - 1) & 1)) {
          // The answer still on its way lands before the CTA exits.
          mbar_wait(bar_claim, (it - 1) & 1, nullptr, p.status, kStatusTimeout, lim);
          break;
        }
        item = clc_block(answer);
      }
      if (item < 0) {
        if (lane == 0) slot->item = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_item_full);
        break;
      }
      // Items run from the last query rows to the first (with a causal mask the
      // long ones come first), or in the order reckoned.
      if (p.by_order) item = order.item(item, p.Hq);
      const int bh = item % (p.B * p.Hq);
      const int row0 = (p.blocks_per_bh - 1 - item / (p.B * p.Hq)) * (kQTiles * kBM);
      const int b = bh / p.Hq;
      const int rows = min(p.Nq - row0, kQTiles * kBM);
      int doc0 = 0, doc1 = 0;
      if (p.docs != nullptr) {
        const int* off = p.docs + static_cast<long long>(b) * (p.n_docs + 1);
        doc0 = find_doc(off, row0 + p.q_offset, -1, p.n_docs);
        doc1 = find_doc(off, row0 + rows - 1 + p.q_offset, doc0, p.n_docs);
      }
      int lo[2] = {0x7fffffff, 0x7fffffff}, hi[2] = {0, 0};
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = u * 32 + lane;
        if (r < rows) {
          const int pos = row0 + r + p.q_offset;
          int t = 0;
          if (p.docs != nullptr) t = find_doc(p.docs + static_cast<long long>(b) * (p.n_docs + 1), pos, doc0, doc1);
          const int2 v = row_interval(p, b, pos, t);
          if (v.x < v.y) {
            lo[u / 4] = min(lo[u / 4], v.x);
            hi[u / 4] = max(hi[u / 4], v.y);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lo[i] = __reduce_min_sync(0xffffffffu, lo[i]);
        hi[i] = __reduce_max_sync(0xffffffffu, hi[i]);
      }
      if (lane == 0) {
        slot->item = item;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          slot->first[i] = hi[i] > 0 ? lo[i] / kBN : 0;
          slot->last[i] = hi[i] > 0 ? (hi[i] + kBN - 1) / kBN : 0;
        }
        slot->end = max(hi[0], hi[1]);
        slot->doc0 = doc0;
        slot->doc1 = doc1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_item_full);
    }
  } else if (warp == R::kTma) {
    setmaxnreg_dec<R::kControlRegs>();
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    bool ok = true;
    int idx = 0;      // ring loads issued so far (over all items)
    int q_loads = 0;  // items whose Q was issued
    ItemSlot x;
    for (int it = 0; ok && next_item(it, x, ok); ++it) {
      int a, b;
      hull(x, a, b);
      if (a >= b) continue;
      const int bh = x.item % (p.B * p.Hq);
      const int q0 = (p.blocks_per_bh - 1 - x.item / (p.B * p.Hq)) * (kQTiles * kBM);
      const int bt = bh / p.Hq, hq = bh % p.Hq, hk = hq / p.G;
      if (!wait_all(bar_q_empty, (q_loads & 1) ^ 1)) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(bar_q_full, kQTiles * L::kTileBytes);
        for (int i = 0; i < kQTiles; ++i)
#pragma unroll
          for (int bx = 0; bx < L::kBoxes; ++bx)
            tma_load_4d(sQ + i * L::kTileBytes + bx * L::kBoxBytes, &tm_q, bar_q_full, bx * 64, q0 + i * kBM, hq, bt);
      }
      __syncwarp();
      ++q_loads;
      for (int j = b - 1; j >= a && ok; --j) {
        for (int t = 0; t < 2; ++t) {
          const int s = idx % kStages;
          if (!wait_all(bar_kv_empty0 + 8 * s, ((idx / kStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t full = bar_kv_full0 + 8 * s;
            mbar_arrive_expect_tx(full, L::kTileBytes);
#pragma unroll
            for (int bx = 0; bx < L::kBoxes; ++bx)
              tma_load_4d(sRing + s * L::kTileBytes + bx * L::kBoxBytes, t ? &tm_v : &tm_k, full, bx * 64, j * kBN, hk,
                          bt);
          }
          __syncwarp();
          ++idx;
        }
      }
    }
    // Every copy issued has landed before the CTA exits (where nothing went
    // wrong, the MMA warp has waited for each of them already).
    if (!ok) {
      if (q_loads > 0) mbar_wait(bar_q_full, (q_loads - 1) & 1, nullptr, p.status, kStatusTimeout, lim);
      for (int s = 0; s < kStages && s < idx; ++s) {
        const int cnt = (idx - s + kStages - 1) / kStages;
        mbar_wait(bar_kv_full0 + 8 * s, (cnt - 1) & 1, nullptr, p.status, kStatusTimeout, lim);
      }
    }
    __syncwarp();
  } else if (warp == R::kMma) {
    setmaxnreg_dec<R::kControlRegs>();
    // ----------------------------------------------------------- MMA issue
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
    };
    auto issue_pv = [&](int i, int slot, bool acc, int part) {
      const uint64_t dv = dV + slot * kTileDesc;
      constexpr int kPer = kBN / 16 / kPParts;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int kk = part * kPer + u;
        umma_ts(tO0 + i * D, tmem + i * kBN + part * kPOff + u * 8, dv + static_cast<uint64_t>(kk * 128), kIdPV,
                (acc || kk > 0) ? 1u : 0u);
      }
    };
    bool ok = true;
    int idx = 0;           // ring position (over all items)
    int g0 = 0, g1 = 0;    // key tiles of each query tile over all items: phases of the P barriers
    int q_used = 0;
    ItemSlot x;
    for (int it = 0; ok && next_item(it, x, ok); ++it) {
      int a, b;
      hull(x, a, b);
      if (a >= b) continue;
      auto in = [&](int i, int j) { return j >= first_of(x, i) && j < last_of(x, i); };
      if (!wait_all(bar_q_full, q_used & 1) ||
          !wait_all(bar_kv_full0 + 8 * (idx % kStages), (idx / kStages) & 1)) {
        ok = false;
        break;
      }
      ++q_used;
      tc_fence_after();
      if (leader) {
        for (int i = 0; i < 2; ++i)
          if (in(i, b - 1)) {
            issue_qk(i, idx % kStages);
            umma_commit(bar_s_full0 + 8 * i);
          }
        umma_commit(bar_kv_empty0 + 8 * (idx % kStages));
        if (b - 1 == a) umma_commit(bar_q_empty);
      }
      __syncwarp();
      ++idx;
      for (int j = b - 1; j >= a && ok; --j) {
        const int sv = idx % kStages;
        if (!wait_all(bar_kv_full0 + 8 * sv, (idx / kStages) & 1)) {
          ok = false;
          break;
        }
        ++idx;
        // Keys behind all that some row of the item sees (padding behind the last
        // document, the free end of a cache): their weights are 0, but a value left
        // there may be NaN or Inf, so their rows are cleared while the weights are
        // still reckoned.  Leaving out the steps of 16 keys instead made the issue of
        // all others longer (4608 keys behind a prefix: 142 and 144 us).
        const int valid = x.end - j * kBN;
        const bool cut = valid < kBN;
        if (cut) {
          // A row has 8 * kBoxes pieces of 16 bytes, one a lane.
          constexpr int kLanes = 8 * L::kBoxes;
          const uint32_t v0 = sRing + sv * L::kTileBytes + (lane % kLanes) / 8 * L::kBoxBytes + lane % 8 * 16;
          for (int r = valid + lane / kLanes; r < kBN; r += 32 / kLanes)
            st_shared_v4(v0 + r * 128, 0u, 0u, 0u, 0u);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        const bool more = j > a;
        int sk = 0;
        for (int i = 0; i < 2 && ok; ++i) {
          if (in(i, j)) {
            const bool acc = j < last_of(x, i) - 1;
            const uint32_t ph = (i ? g1 : g0) & 1;
            if (!wait_all(bar_p_part0 + 8 * i, ph)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (leader) issue_pv(i, sv, acc, 0);
            __syncwarp();
            if (!wait_all(bar_p_full0 + 8 * i, ph)) {
              ok = false;
              break;
            }
            i ? ++g1 : ++g0;
            tc_fence_after();
            if (leader) {
              issue_pv(i, sv, true, 1);
              if (j == first_of(x, i)) umma_commit(bar_o_full0 + 8 * i);
            }
            __syncwarp();
          }
          if (leader && i == 1) umma_commit(bar_kv_empty0 + 8 * sv);
          __syncwarp();
          if (more) {
            if (i == 0) {
              sk = idx % kStages;
              if (!wait_all(bar_kv_full0 + 8 * sk, (idx / kStages) & 1)) {
                ok = false;
                break;
              }
              ++idx;
              tc_fence_after();
            }
            if (leader) {
              if (in(i, j - 1)) {
                issue_qk(i, sk);
                umma_commit(bar_s_full0 + 8 * i);
              }
              if (i == 1) {
                umma_commit(bar_kv_empty0 + 8 * sk);
                if (j - 1 == a) umma_commit(bar_q_empty);  // the item's last Q K^T
              }
            }
            __syncwarp();
          }
        }
      }
    }
    // Every MMA issued completes before tensor memory is freed.
    if (leader) umma_commit(bar_drain);
    __syncwarp();
    mbar_wait(bar_drain, 0, nullptr, p.status, kStatusTimeout, lim);
    __syncwarp();
  } else {
    setmaxnreg_inc<R::kSoftmaxRegs>();
    // ------------------------------------------------------------- softmax
    const int i = kWide ? warp / 8 : warp / 4;      // query tile
    const int half = kWide ? (warp / 4) % 2 : 0;      // wide: which keys, and which O columns to store
    const int r = threadIdx.x % 128;                  // row of the tile = tensor-memory lane
    constexpr int kCols = kWide ? D / 2 : D;
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tS = tmem + i * kBN + half * 64 + lane_off;
    const uint32_t tO = tmem + 2 * kBN + i * D + half * kCols + lane_off;
    bool ok = true;
    int g = 0;    // key tiles over all items: phases of the S barrier
    int n_o = 0;  // items with key tiles: phase of the O barrier
    auto wait_warp = [&](uint32_t bar, uint32_t parity) {
      const bool got = mbar_wait_hint(bar, parity, abort_word, p.status, kStatusTimeout, lim, kSuspendHintNs);
      return !__any_sync(0xffffffffu, !got);
    };
    ItemSlot x;
    for (int it = 0; ok && next_item(it, x, ok); ++it) {
      const int bh = x.item % (p.B * p.Hq);
      const int bt = bh / p.Hq, hq = bh % p.Hq;
      const int row = (p.blocks_per_bh - 1 - x.item / (p.B * p.Hq)) * (kQTiles * kBM) + i * kBM + r;
      const int pos = row + p.q_offset;
      float slope2 = 0.f;
      if constexpr (kBias) slope2 = __ldg(p.sm.slopes + hq) * 1.4426950408889634f;
      // Rows past Nq are computed like any other (their Q is zeros) and not
      // stored; they count as seeing everything, so that they mask nothing.
      int2 seen = make_int2(0, 0x7fffffff);
      if (row < p.Nq) {
        int t = 0;
        if (p.docs != nullptr)
          t = find_doc(p.docs + static_cast<long long>(bt) * (p.n_docs + 1), pos, x.doc0, x.doc1);
        seen = row_interval(p, bt, pos, t);
      }
      float m_ref = kWide ? p.sm.cap_ref : -INFINITY, l = 0.f;
      const int first = first_of(x, i), last = last_of(x, i);
      for (int j = last - 1; j >= first; --j, ++g) {
        if (!wait_warp(bar_s_full0 + 8 * i, g & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int k0 = j * kBN + half * 64;
        if constexpr (kWide)
          capped_keys(tS, tS, seen.x - k0, seen.y - k0, true, p.sm, l, (half ? bar_p_full0 : bar_p_part0) + 8 * i, lane);
        else
          softmax_tile<D, kCap, kBias, false>(tS, tO, seen.x - k0, seen.y - k0, static_cast<float>(pos - k0), slope2,
                                              p.sm, true, j < last - 1, m_ref, l, bar_p_part0 + 8 * i,
                                              bar_p_full0 + 8 * i, lane);
      }
      if (!ok) break;
      if (first < last) {
        if constexpr (kWide) {
          // The row's sum is both threads'.  A slot is written again two items
          // on, after a swap that the other thread enters having read it.
          const uint32_t at = base + L::kSumOff + (n_o & 1) * 2048 + i * 1024 + r * 4;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + half * 512), "f"(l) : "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_swap0 + 8 * (4 * i + warp % 4));
          if (!wait_warp(bar_swap0 + 8 * (4 * i + warp % 4), n_o & 1)) {
            ok = false;
            break;
          }
          float other;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(at + (1 - half) * 512) : "memory");
          l += other;
        }
        if (!wait_warp(bar_o_full0 + 8 * i, n_o & 1)) {
          ok = false;
          break;
        }
        ++n_o;
        tc_fence_after();
      }
      const int wrow = row - lane;  // first row of this warp
      if (wrow >= p.Nq) continue;
      const bool empty = l == 0.f;
      const float inv = empty ? 0.f : 1.f / l;
      __nv_bfloat16* o = p.o + bt * p.o_s[0] + hq * p.o_s[1] + wrow * p.o_s[2] + half * kCols;
      const uint32_t stage = base + L::kStageOff + warp * L::kStageWarpBytes;
      bool bad;
      if constexpr (kWide)
        bad = store_cols_bf16<kCols>(tO, stage, o, p.o_s[2], p.Nq - wrow, inv);
      else
        bad = store_rows<D>(tO, stage, o, p.o_s[2], p.Nq - wrow, inv);
      if (half == 0 && row < p.Nq)
        p.lse[static_cast<size_t>(bh) * p.Nq + row] =
            empty ? -INFINITY : (m_ref + lg2_approx(l)) * 0.69314718055994531f;
      const unsigned redo = __ballot_sync(0xffffffffu, bad && !empty && row < p.Nq && l <= FLT_MAX);
      if (redo != 0u) {
        const int hk = hq / p.G;
        repair_rows<D, kCols>(redo, p.q + bt * p.q_s[0] + hq * p.q_s[1] + wrow * p.q_s[2], p.q_s[2],
                              p.k + bt * p.k_s[0] + hk * p.k_s[1], p.v + bt * p.v_s[0] + hk * p.v_s[1] + half * kCols,
                              p.k_s[2], p.v_s[2], seen.x, seen.y, wrow + p.q_offset, m_ref + lg2_approx(l), slope2, p.sm,
                              kCap, kBias, o, p.o_s[2]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace mod
}  // namespace pa
