// cache4.cuh -- the layout of the paged 4-bit key/value cache, shared by the
// kernels that fill, read, attend to and thin it out.
//
// A head vector of D elements is held as D/32 groups of 32 codes of 4 bits, each
// with a bf16 scale and a bf16 minimum: value = min + scale * code.  A page holds
// page_size tokens (a multiple of 16) of every kv head:
//
//   cache [num_pages][Hkv][page_size / 16][block]
//   block = 16 slots: K codes 16 x D/2 bytes | K parameters 16 x D/8 bytes
//                   | V codes 16 x D/2 bytes | V parameters 16 x D/8 bytes
//
// so a sequence's keys and values of one head arrive in contiguous copies of
// 20 D bytes, and one block is what a warp of the attention kernel multiplies at
// a time.  Inside a block the order is the matrix instructions' (mma.m16n8k16,
// lanes numbered 4 i + t):
//   K row of a slot: 32-bit word t * (D/32) + g holds elements 32 g + 8 t + 0..7
//     of the vector, element j in bits 4 j .. 4 j + 3: lane t of a row's four
//     loads its words of every group in one piece.
//   V row: 16-bit half g of chunk i (D/16 bytes) holds elements 32 g + 4 i + 0..3,
//     so a lane's elements of one group are four rows of the transposed product.
//     So that the four slots a load touches at a time lie in different shared
//     memory banks, the chunks of a slot with bit 2 set are rotated by half a row
//     (D = 128), or the slots with bit 2 set swap rows in pairs (D = 64).
//   Parameters of a slot: D/32 words, the scale in the low half, the minimum in
//     the high half.
#pragma once

#include <cstdint>

namespace fa {

constexpr int kC4Block = 16;  // slots per block

template <int D>
struct C4 {
  static constexpr int kGroups = D / 32;
  static constexpr int kRow = D / 2;    // bytes of a slot's codes
  static constexpr int kPar = D / 8;    // bytes of a slot's parameters
  static constexpr int kOffKPar = kC4Block * kRow;
  static constexpr int kOffV = kOffKPar + kC4Block * kPar;
  static constexpr int kOffVPar = kOffV + kC4Block * kRow;
  static constexpr int kBytes = kOffVPar + kC4Block * kPar;  // of a block

  // byte offset in the block of 16-bit half g of chunk i of slot s's V row
  static __host__ __device__ constexpr int v_half(int s, int i, int g) {
    return D == 128 ? kOffV + s * kRow + ((i ^ (s & 4)) * 8) + g * 2
                    : kOffV + (s ^ ((s >> 2) & 1)) * kRow + i * 4 + g * 2;
  }
};

inline __host__ __device__ int c4_block_bytes(int D) { return kC4Block * (D + D / 4); }

// Sequence lengths and page ids come from device memory: what is out of range is
// cut or left out, and recorded in the cache status word.
struct C4Table {
  const int* pages;  // [B, width]
  int width;
  int num_pages;
  int shift;  // log2 of the blocks per page
  int* status;
  __host__ __device__ int blocks_per_page() const { return 1 << shift; }
  __host__ __device__ int in_page(int blk) const { return blk & ((1 << shift) - 1); }
};

inline int c4_shift(int page_size) {
  int s = 0;
  while ((kC4Block << s) < page_size) ++s;
  return s;
}

// The page of block blk of sequence b, or -1.
__device__ __forceinline__ int c4_page(const C4Table& t, int b, int blk) {
  const int e = blk >> t.shift;
  if (e >= t.width) return -1;
  const int p = __ldg(t.pages + (size_t)b * t.width + e);
  return p >= 0 && p < t.num_pages ? p : -1;
}

__device__ __forceinline__ void c4_flag(const C4Table& t) { atomicExch(t.status, 1); }

// bf16 halves of a parameter word as fp32
__device__ __forceinline__ float c4_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float c4_min(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace fa
