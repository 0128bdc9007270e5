// var_common.cuh -- the plan of a packed call (sequences of different lengths
// in one [T, H, D] tensor), as the plan kernel writes it and the attention
// kernels read it.
#pragma once

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

// The part of an item every kernel reads, in one 16-byte load.
__device__ __forceinline__ VarItem load_item(const VarItem* items, int i) {
  const int4 x = *reinterpret_cast<const int4*>(items + i);
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
