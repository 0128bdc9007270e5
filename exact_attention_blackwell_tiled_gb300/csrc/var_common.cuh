// var_common.cuh -- the plan of a packed call (sequences of different lengths
// in one [T, H, D] tensor), as the plan kernel writes it and the attention
// kernels read it.
#pragma once

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

__device__ __forceinline__ int warp_add(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Items of sequence `other` that go before item `t` of the sequence `own` with
// n_own blocks of item_rows rows; len_other / len_own in 64-row blocks.
//   forward, causal: pair t attends to 2 t + 2 kv tiles: by t, descending;
//   backward, causal: kv tile t is seen by blocks64 - 2 t query blocks;
//   otherwise: the longest sequence first, its items in order.
// Ties go to the lower sequence.  Within a sequence the backward's tiles ascend (desc: descend).
__device__ __forceinline__ int items_before(int mode, int t, int n_own, int blk_own, int n_other,
                                            int blk_other, bool lower) {
  if (mode == 0) {  // forward, causal
    const int more = max(0, n_other - 1 - t);
    return more + (lower && n_other > t ? 1 : 0);
  }
  if (mode == 1) {  // backward, causal: blk_other - 2 t' > blk_own - 2 t
    const int d = blk_other - (blk_own - 2 * t);  // 2 t' < d
    const int more = d > 0 ? min(n_other, (d + 1) / 2) : 0;
    const bool tie = d >= 0 && (d & 1) == 0 && d / 2 < n_other;
    return more + (lower && tie ? 1 : 0);
  }
  return n_other > n_own || (n_other == n_own && lower) ? n_other : 0;
}

__device__ __forceinline__ int plan_mode(const PlanArgs& p) {
  return p.causal ? (p.item_rows == 256 ? 0 : 1) : 2;
}
// Whether a sequence's items lie in the list from the last one down.
__device__ __forceinline__ bool plan_descends(const PlanArgs& p) {
  return plan_mode(p) == 0 || (plan_mode(p) == 2 && p.desc);
}

// The plan of at most 32 sequences by the `warps` warps of a block: put(place, item) for every
// item, each by one thread; returns their number, -1 where cu does not ascend in [0, T].
// Every warp reads all lengths, a lane a sequence, and places those sequences' items
// whose turn is its own.
template <typename F>
__device__ __forceinline__ int plan_in_block(const PlanArgs& p, int warp, int warps, F put) {
  const int lane = threadIdx.x & 31;
  const int shift = p.item_rows == 256 ? 8 : 7, mode = plan_mode(p);
  int lo = 0, len = 0;
  bool bad = false;
  if (lane < p.B) {
    lo = p.cu[lane];
    const int hi = p.cu[lane + 1];
    bad = lo < 0 || hi < lo || hi > p.T;
    len = hi - lo;
  }
  if (__any_sync(0xffffffffu, bad)) return -1;
  const int n = (len + p.item_rows - 1) >> shift, blk = (len + 63) >> 6;
  const int rows = (len + p.pad - 1) & -p.pad;
  int pad0 = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, pad0, o);
    if (lane >= o) pad0 += y;
  }
  pad0 -= rows;
  for (int b = warp; b < p.B; b += warps) {
    const int n_own = __shfl_sync(0xffffffffu, n, b), blk_own = __shfl_sync(0xffffffffu, blk, b);
    VarItem it{};
    it.row0 = __shfl_sync(0xffffffffu, lo, b);
    it.len = __shfl_sync(0xffffffffu, len, b);
    it.b = b;
    it.pad0 = __shfl_sync(0xffffffffu, pad0, b);
    int same = 0;  // (without a causal mask an item's own number does not count)
    if (mode == 2) same = warp_add(lane < p.B && lane != b ? items_before(2, 0, n_own, blk_own, n, blk, lane < b) : 0);
    for (int t0 = 0; t0 < n_own; t0 += 32) {
      const int t = t0 + lane;
      int before = same;
      if (mode != 2)
        for (int i = 0; i < p.B; ++i) {
          const int n_i = __shfl_sync(0xffffffffu, n, i), blk_i = __shfl_sync(0xffffffffu, blk, i);
          if (i != b) before += items_before(mode, t, n_own, blk_own, n_i, blk_i, i < b);
        }
      it.tile = t;
      if (t < n_own) put(before + (plan_descends(p) ? n_own - 1 - t : t), it);
    }
  }
  return warp_add(n);
}

// The part of an item every kernel reads, in one 16-byte load (kNarrow: all there is of it).
template <bool kNarrow = false>
__device__ __forceinline__ VarItem load_item(const VarItem* items, int i) {
  const int4 x = reinterpret_cast<const int4*>(items)[kNarrow ? i : 2 * i];
  VarItem it;
  it.row0 = x.x;
  it.len = x.y;
  it.tile = x.z;
  it.b = x.w;
  return it;
}

// The pieces' maps of N tensors on their way before the first use, a lane each.
template <int N>
__device__ __forceinline__ void prefetch_tails(const Tails<true, N>& tails, int lane) {
  if (lane < N * kTailBoxes) tma_prefetch_desc(&tails.of[lane / kTailBoxes].box[lane % kTailBoxes]);
}

// Rows row .. row + valid - 1 of head `head` of a packed tensor into a tile of kRows rows (128
// bytes each, kColBlocks blocks of 64 columns) in pieces of 64, 16, 4 and 1 rows, then
// rows T .., which do not exist and arrive as zeros.
template <int kRows, int kColBlocks>
__device__ __forceinline__ void load_pieces(uint32_t dst, uint32_t block_bytes, const TailMaps& tails,
                                            uint32_t bar, int row, int valid, int T, int head) {
  int at = 0, from = row, n = valid;
#pragma unroll 1
  for (int zeros = 0; zeros < 2; ++zeros) {
#pragma unroll 1
    for (int x = 0; x < kTailBoxes; ++x) {
      const int rows = 64 >> (2 * x);
#pragma unroll 1
      for (; n >= rows; n -= rows) {
#pragma unroll
        for (int cb = 0; cb < kColBlocks; ++cb)
          tma_load_3d(dst + cb * block_bytes + at * 128, &tails.box[x], bar, cb * 64, from, head);
        at += rows;
        if (!zeros) from += rows;
      }
    }
    from = T;
    n = kRows - at;
  }
}

// Rows row .. row + valid - 1 of head `head` of a packed tensor into a tile of kRows
// rows (128 bytes each, kColBlocks blocks of 64 columns), zeros behind them: one box
// where the tile is full, pieces of 64, 16, 4 and 1 rows where the sequence ends in
// it, at most 11 with those of rows T .., which do not exist and arrive as zeros.  So
// the products never meet another sequence's rows.  (The swizzle goes by the address
// in shared memory, so a piece lies as the full box would have put its rows.)
//
// Maps of each sequence by itself, written by the plan kernel, would need no pieces;
// but then the TMA unit reads descriptors that another kernel has just written, and a
// run of calls whose tensors lay all over the address space ended in an illegal access,
// with every other address shown in bounds.  These maps are made on the host.
template <int kRows, int kColBlocks>
__device__ __forceinline__ void load_rows(uint32_t dst, uint32_t block_bytes, const CUtensorMap* full,
                                          const TailMaps& tails, uint32_t bar, int row, int valid,
                                          int T, int head) {
  if (valid >= kRows) {
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb)
      tma_load_3d(dst + cb * block_bytes, full, bar, cb * 64, row, head);
    return;
  }
  load_pieces<kRows, kColBlocks>(dst, block_bytes, tails, bar, row, valid, T, head);
}

}  // namespace fa
