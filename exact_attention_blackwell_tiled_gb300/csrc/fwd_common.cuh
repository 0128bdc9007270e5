// fwd_common.cuh -- device helpers shared by the forward kernels: the unit
// schedule (which (head, query-tile pair) a CTA takes next), the kv-tile range
// of a query tile under masks and key counts, and bounded waits.
#pragma once

#include "fa_internal.h"
#include "ptx.cuh"
#include "var_common.cuh"

namespace fa {

// The r-th of n_units units that this CTA processes (-1 when it has no more).
// Every role of the CTA walks the same sequence.
__device__ __forceinline__ int cta_unit(const FwdArgs& a, int n_units, int r) {
  int k;
  if (a.sched == 2) {
    // boustrophedon: each round of gridDim.x units alternates direction, so
    // CTAs that got a longer unit in one round get a shorter one in the next
    k = r * (int)gridDim.x + ((r & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
  } else {
    k = blockIdx.x + r * gridDim.x;
  }
  return k < n_units ? k : -1;
}

// Unit u -> (flat batch*head index, tile pair p: query tiles 2p and 2p+1).
//   sched 0:     head-major (non-causal, and windows), so CTAs running at the
//                same time share the K/V of few heads in L2.
//   sched 2:     longest pairs of every head first (causal work grows with the
//                pair index), dealt in a snake.
//   sched 3:     split-KV; the pairs of one (head, split) are adjacent, so
//                they run together and share that split's K/V in L2.
__device__ __forceinline__ void unit_coords(const FwdArgs& a, int u, int& bh, int& pair,
                                            int& split) {
  const int np = a.n_pairs;
  split = 0;
  if (a.sched == 3) {
    const int rest = u / np;
    pair = u - rest * np;
    bh = rest / a.n_split;
    split = rest - bh * a.n_split;
    return;
  }
  if (a.sched == 2) {
    const int BH = a.B * a.Hq;
    pair = np - 1 - u / BH;
    bh = u - (u / BH) * BH;
    return;
  }
  bh = u / np;
  pair = u - bh * np;
}

// A unit of work: query head bh (flat over the batch), the pair of query tiles
// 2 * pair and 2 * pair + 1, its split of the kv tiles, and the sizes of its
// sequence.  Packed calls (kVar): units are (item, head) with the head running
// fastest, an item of the plan names a sequence (rows row0 .. row0 + Sq - 1 of
// the packed tensors) and a pair of its query tiles, and bh is the head alone.  kHeads: an
// item names one query tile, and the pair is that tile of two heads of one kv head.
struct FwdUnit {
  int bh, pair, split;
  int b, h;   // batch entry and query head
  int Sq;     // query rows of the sequence
  int row0;   // its first packed row (kVar)
};

template <bool kVar, bool kHeads = false>
__device__ __forceinline__ FwdUnit fwd_unit(const FwdArgs& a, const VarItem* items, int u) {
  FwdUnit w;
  w.row0 = 0;
  if constexpr (kVar) {
    const int per = kHeads ? a.Hq / 2 : a.Hq, item = u / per;
    const VarItem it = load_item<kHeads>(items, item);
    w.h = w.bh = (u - item * per) * (kHeads ? 2 : 1);
    w.b = it.b;
    w.pair = it.tile;
    w.split = 0;
    w.Sq = it.len;
    w.row0 = it.row0;
  } else {
    unit_coords(a, u, w.bh, w.pair, w.split);
    w.b = w.bh / a.Hq;
    w.h = w.bh - w.b * a.Hq;
    w.Sq = a.Sq;
  }
  return w;
}

// Keys of batch b that exist: seqlens_k[b] clamped to [0, Sk] (the key padding
// mask); all Sk without lengths, and always in the plain kernel.
template <bool kWin>
__device__ __forceinline__ int batch_kv_len(const FwdArgs& a, int b) {
  if (!kWin || !a.seqlens_k) return a.Sk;
  const int n = a.seqlens_k[b];
  return n < 0 ? 0 : (n < a.Sk ? n : a.Sk);
}

// The same for a unit: a packed sequence has as many keys as queries.
template <bool kWin, bool kVar>
__device__ __forceinline__ int unit_kv_len(const FwdArgs& a, const FwdUnit& w) {
  if constexpr (kVar) return w.Sq;
  return batch_kv_len<kWin>(a, w.b);
}

// kv tiles [lo, hi) that query tile qt sees under the window (wl, wr) among the
// first kv_len keys (empty when the tile lies past Sq or sees no key)
__device__ __forceinline__ void tile_kv_range(int Sq, int wl, int wr, int kv_len, int qt, int& lo,
                                              int& hi) {
  lo = hi = 0;
  if (qt * kTile >= Sq) return;
  const int last = min(Sq, (qt + 1) * kTile) - 1;  // last query row of the tile
  const int lo_key = wl >= 0 ? max(0, qt * kTile - wl) : 0;
  const int hi_key = wr >= 0 ? min(kv_len, last + wr + 1) : kv_len;
  lo = lo_key / kTile;
  hi = max(lo, (hi_key + kTile - 1) / kTile);
}

// A tile's range cut to the kv tiles of `split` (kSplit); may become empty.
template <bool kSplit>
__device__ __forceinline__ void split_kv_range(const FwdArgs& a, int Sq, int wl, int wr, int kv_len,
                                               int qt, int split, int& lo, int& hi) {
  tile_kv_range(Sq, wl, wr, kv_len, qt, lo, hi);
  if (kSplit) {
    const int s0 = split * a.split_tiles;
    lo = max(lo, s0);
    hi = max(lo, min(hi, s0 + a.split_tiles));
  }
}

// The kv tiles the two query tiles of a pair stream: lo[t], hi[t] per tile,
// and their union [jlo, jlo + nmax).  An empty tile gets lo = hi = jlo; both
// empty: nmax = 0 and the unit is skipped.
template <bool kSplit>
__device__ __forceinline__ void pair_kv_span(const FwdArgs& a, int Sq, int wl, int wr, int kv_len,
                                             int pair, int split, int lo[2], int hi[2], int& jlo,
                                             int& nmax) {
  split_kv_range<kSplit>(a, Sq, wl, wr, kv_len, 2 * pair, split, lo[0], hi[0]);
  split_kv_range<kSplit>(a, Sq, wl, wr, kv_len, 2 * pair + 1, split, lo[1], hi[1]);
  const bool e0 = hi[0] <= lo[0], e1 = hi[1] <= lo[1];
  if (e0 && e1) {
    jlo = lo[0];
    nmax = 0;
    return;
  }
  jlo = e0 ? lo[1] : (e1 ? lo[0] : min(lo[0], lo[1]));
  const int jend = e0 ? hi[1] : (e1 ? hi[0] : max(hi[0], hi[1]));
  nmax = jend - jlo;
  if (e0) lo[0] = hi[0] = jlo;
  if (e1) lo[1] = hi[1] = jlo;
}

// The same with sinks (has), as positions: kv tile 0 is position 0 for every query tile with
// rows, and where a window begins behind it (first), the windows' tiles follow from position
// 1 on, so that the tiles between the sinks and the window are left out.  Position 0 then
// has zeros for the values behind the sinks, lest a weight of zero meets an infinity there;
// if the first tile's window begins in kv tile 0 all the same (twice), that tile comes
// again at position 1, where the first query tile begins.  plo1 is the first position of
// the second one's window, phi[t] the end of tile t's.  (A packed unit has rows and sees
// itself: n is not 0.)
template <bool kHeads>
struct SinkSpan {
  int plo1, phi[2];  // phi 0: no rows (the second tile's)
  int jlo, n;
  bool has, first, twice;
  __device__ __forceinline__ int tile(int p) const { return first && p == 0 ? 0 : jlo + p - (first ? 1 : 0); }
  // Whether tile t computes at position p, its first position, and the next one.
  __device__ __forceinline__ bool active(int t, int p) const {
    if (kHeads) return p < n;
    return p < phi[t] && (t == 0 ? p > 0 || !twice : p >= plo1 || (p == 0 && has));
  }
  __device__ __forceinline__ int begin(int t) const {
    return kHeads ? 0 : t == 0 ? (twice ? 1 : 0) : has ? 0 : plo1;
  }
  __device__ __forceinline__ int next(int t, int p) const {
    return kHeads || t == 0 ? p + 1 : max(p + 1, plo1);
  }
};
template <bool kHeads>
__device__ __forceinline__ SinkSpan<kHeads> sink_kv_span(int Sq, int wl, int wr, int sinks, int pair) {
  SinkSpan<kHeads> s;
  s.has = sinks > 0;
  int lo0, hi0;
  tile_kv_range(Sq, wl, wr, Sq, kHeads ? pair : 2 * pair, lo0, hi0);
  s.jlo = lo0;
  if constexpr (kHeads) {
    s.first = s.has && lo0 > 0;
    s.twice = false;
    s.plo1 = 0;
    s.n = s.phi[0] = s.phi[1] = hi0 - lo0 + (s.first ? 1 : 0);
  } else {
    int lo1, hi1;
    tile_kv_range(Sq, wl, wr, Sq, 2 * pair + 1, lo1, hi1);  // (no rows: both are 0)
    s.first = s.has && max(lo0, lo1) > 0;
    s.twice = s.first && lo0 == 0;
    const int shift = (s.first ? 1 : 0) - lo0;
    s.phi[0] = hi0 + shift;
    s.plo1 = hi1 > lo1 ? lo1 + shift : 0;
    s.phi[1] = hi1 > lo1 ? hi1 + shift : 0;
    s.n = max(s.phi[0], s.phi[1]);
  }
  return s;
}

// Bounded wait done by every lane of a warp; the outcome is made warp-uniform so
// the warp-collective tcgen05.ld/st that follow are never reached by part of it.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const bool ok = mbar_wait(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

// Bounded wait used only while draining at exit: ignores the abort flag.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
  }
}

}  // namespace fa
