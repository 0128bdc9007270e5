// fa_cache4.cu -- filling, reading back and thinning out the paged 4-bit cache
// (cache4.cuh has its layout); fa_cache4_attend.cu attends to it.
//
// append: per group of 32 elements x, in fp32 with every operation rounded to
//   nearest as written, so that the codes are those of the formula:
//     mn = min x,  scale = bf16((max x - mn) / 15),
//     code = clamp(rint((x - mn) / scale), 0, 15), 0 where scale is 0.
//   mn is an element and so exact in bf16; the codes are taken with the rounded
//   scale, so its rounding (2^-9) moves the top code's value, not the others'
//   choice.  It reads 4 D bytes of a token's key and value and writes 5/4 D.  A
//   warp takes eight (token, head) pairs, whose loads it issues before it looks for
//   the places they go to.  Measured: 18304 tokens of 8 heads of 128 (98 MB) in 25
//   us, 4.0 TB/s; the SMs issue in about 65% of the cycles, most of it the exact
//   quotients of the codes, so arithmetic binds it before memory.
// read: value = min + scale * code in one fp32 FMA, rounded once to bf16.  Reads
//   5/4 D bytes of a token, writes 4 D.  Bound by memory: 352 MB in 52 us, 6.7 TB/s.
// evict: two kernels.  The first ranks one (sequence, kv head) per block: the K
//   largest weights are found digit by digit (three passes of 11, 11 and 10 bits
//   over the weights' bit patterns, which order like the values; up to 16384 of
//   them stay in registers), and a last pass in index order counts what is kept,
//   ties from the lowest index up, and writes each kept key's old place and weight.
//   The second copies the kept keys' codes to the new pages in order: 16 slots per
//   warp, in 16-byte pieces.  Measured with 16 sequences of 6000 to 8192 tokens, 8
//   heads of 128, half of them kept: ranking 14 us, a chain of block-wide steps and
//   shared atomics on 128 blocks; the copy (168 MB) 36 us, 4.6 TB/s, bound by the
//   latency of pieces picked from all over.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "cache4.cuh"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

__device__ int g_cache4_status = 0;

namespace {

// ------------------------------------------------------------------ append

struct AppendArgs {
  uint8_t* cache;
  const __nv_bfloat16 *k, *v;
  long long k_token, k_head, v_token, v_head;
  const int* cu;    // [B + 1], or null: one token per sequence
  const int* lens;  // [B] tokens held before
  const long long* slots;  // [T] (kSlots) where the tokens go, instead: -1 for nowhere
  C4Table table;
  int B, T, Hkv;
};

constexpr int kAppendWarps = 4, kAppendItems = 8;  // (token, head) pairs per warp

// Sequence that holds packed token i, or -1, by a whole warp: each step splits the
// range that cu bounds in 32.
__device__ int find_sequence(const int* cu, int B, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the sequence is among lo .. lo + n - 1, if there is one
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lo + lane * step;  // first sequence of the lane's piece
    const unsigned m = __ballot_sync(0xffffffffu, at < lo + n && cu[at] <= i);
    const int pieces = 32 - __clz(m | 1);  // cu ascends: the last piece that begins at or before i
    n = min(step, lo + n - (lo + (pieces - 1) * step));
    lo += (pieces - 1) * step;
  }
  return cu[lo] <= i && i < cu[lo + 1] ? lo : -1;
}

// RN(a / b) from y near 1 / b: the quotient of the product is off by an ulp or two,
// its remainder is exact in one FMA, and the correction leaves an error far below
// half an ulp before the last rounding (Markstein's division step).  For a code's
// quotient that is enough for the sides of a tie, d = (code + 1/2) sc: a tie comes
// out exactly, and the nearest other d, an ulp away, lies more than half an ulp of
// the quotient off it, since code + 1/2 has 5 bits and sc 8.
__device__ __forceinline__ float divide(float a, float b, float y) {
  const float q = __fmul_rn(a, y);
  return __fmaf_rn(__fmaf_rn(-q, b, a), y, q);
}

__device__ __forceinline__ float reciprocal_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Scale and codes of a lane's 16 elements f of a group whose minimum is mn and
// maximum mx; the codes come packed, element e in bits 4 (e % 8) of word e / 8.
__device__ __forceinline__ void quantise(const float (&f)[16], float mn, float mx, uint32_t* scale,
                                         uint32_t (&codes)[2]) {
  const float range = __fsub_rn(mx, mn);
  // far from the ends of fp32's range the divisions are the short ones above
  const bool plain = range >= 0x1p-80f && range <= 0x1p80f;
  const __nv_bfloat16 sc16 =
      __float2bfloat16_rn(plain ? divide(range, 15.f, 0x1.111112p-4f) : __fdiv_rn(range, 15.f));
  *scale = __bfloat16_as_ushort(sc16);
  const float sc = __bfloat162float(sc16);
  codes[0] = codes[1] = 0;
  if (plain) {
    const float y = reciprocal_approx(sc);
    // divide() on two elements to an instruction (28 -> 25 us for the tokens above);
    // adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and leaves it in
    // the low bits; the codes are at most 15 (the scale is at most 2^-9 too small),
    // so the words add up without touching each other but for a constant
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      uint32_t sum = 0, magic = 0;
#pragma unroll
      for (int e = 6; e >= 0; e -= 2) {
        const float2 y2 = make_float2(y, y), round = make_float2(12582912.f, 12582912.f);
        const float2 d = __fadd2_rn(make_float2(f[8 * z + e], f[8 * z + e + 1]), make_float2(-mn, -mn));
        const float2 q = __fmul2_rn(d, y2);
        const float2 r = __ffma2_rn(q, make_float2(-sc, -sc), d);
        const float2 m = __fadd2_rn(__ffma2_rn(r, y2, q), round);
        sum = (sum * 16u + __float_as_uint(m.y)) * 16u + __float_as_uint(m.x);
        magic = (magic * 16u + 0x4B400000u) * 16u + 0x4B400000u;
      }
      codes[z] = sum - magic;
    }
  } else if (sc > 0.f) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      codes[e / 8] |= (uint32_t)fminf(rintf(__fdiv_rn(__fsub_rn(f[e], mn), sc)), 15.f) << (4 * (e % 8));
  }
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 y = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 y = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// A lane takes 16 elements, half a group, so that 32 elements share one scale, one
// shuffle each for minimum and maximum, and four stores; D / 16 lanes hold a vector,
// and the lanes of a warp 1024 / D vectors at a time: the key and the value of
// 512 / D (token, head) items.  kSlots: the tokens' slots are given.
template <int D, bool kSlots>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendArgs a) {
  using L = C4<D>;
  constexpr int kLanes = D / 16;          // of a vector
  constexpr int kAtOnce = 16 / kLanes;    // items: 2 or 4
  constexpr int kSteps = kAppendItems / kAtOnce;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vec = lane / kLanes, l = lane % kLanes;
  const bool is_v = vec & 1;
  const int mine = vec >> 1;  // the lane's item of a step
  const int g = l >> 1, half = l & 1;
  const uint32_t total = (uint32_t)a.T * a.Hkv;  // below 2^31
  const uint32_t item0 = (blockIdx.x * kAppendWarps + warp) * kAppendItems;
  grid_dep_wait();
  grid_dep_launch();
  if (item0 >= total) return;
  // the vectors first: where they go is found while they are on their way
  uint4 x[kSteps][2];
  const uint32_t heads = a.Hkv, tok0 = item0 / heads, h0 = item0 - tok0 * heads;
  {
    const uint32_t item = item0 + mine;
    uint32_t tok = tok0, h = h0 + mine;
    for (; h >= heads; h -= heads) ++tok;
    const long long by_token = is_v ? a.v_token : a.k_token, by_head = is_v ? a.v_head : a.k_head;
    const __nv_bfloat16* base = (is_v ? a.v : a.k) + l * 16;
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      x[n][0] = x[n][1] = make_uint4(0u, 0u, 0u, 0u);
      if (item + n * kAtOnce < total) {
        const uint4* src = reinterpret_cast<const uint4*>(base + tok * by_token + h * by_head);
        x[n][0] = src[0];
        x[n][1] = src[1];
      }
      for (h += kAtOnce; h >= heads; h -= heads) ++tok;
    }
  }
  // lane n: the byte offset of item n's block, or -1, and its slot there
  long long off_n = -1;
  int slot_n = 0;
  {
    const int first = !kSlots && a.cu ? find_sequence(a.cu, a.B, (int)tok0) : (int)tok0;
    const uint32_t item = item0 + lane;
    if (lane < kAppendItems && item < total) {
      int tok = (int)tok0;
      uint32_t h = h0 + lane;
      for (; h >= heads; h -= heads) ++tok;
      int b = kSlots ? -1 : a.cu ? first : tok;
      if constexpr (kSlots) {
        const long long s = a.slots[tok], page = s >> (a.table.shift + 4);
        if (s >= 0 && page < a.table.num_pages) {
          slot_n = (int)(s % kC4Block);
          const int blk = a.table.in_page((int)((s / kC4Block) & INT_MAX));
          off_n = ((page * a.Hkv + h) * a.table.blocks_per_page() + blk) * L::kBytes;
        } else if (s >= 0) {
          c4_flag(a.table);
        }
      } else if (a.cu) {
        // later items may belong to later sequences
        if (b < 0 && tok > (int)tok0) b = 0;
        while (b >= 0 && b < a.B && tok >= a.cu[b + 1]) ++b;
        if (b >= a.B || (b >= 0 && tok < a.cu[b])) b = -1;
      }
      if (b >= 0) {
        const long long s = (long long)a.lens[b] + (a.cu ? tok - a.cu[b] : 0);
        int page = -1;
        if (s >= 0 && s < (long long)a.table.width * a.table.blocks_per_page() * kC4Block)
          page = c4_page(a.table, b, (int)(s / kC4Block));
        if (page < 0) {
          c4_flag(a.table);
        } else {
          slot_n = (int)(s % kC4Block);
          const int blk = a.table.in_page((int)(s / kC4Block));
          off_n = (((long long)page * a.Hkv + h) * a.table.blocks_per_page() + blk) * L::kBytes;
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kSteps; ++n) {
    const long long off = __shfl_sync(0xffffffffu, off_n, n * kAtOnce + mine);
    const int slot = __shfl_sync(0xffffffffu, slot_n, n * kAtOnce + mine);
    const uint32_t w[8] = {x[n][0].x, x[n][0].y, x[n][0].z, x[n][0].w,
                           x[n][1].x, x[n][1].y, x[n][1].z, x[n][1].w};
    // minimum and maximum two elements at a time, over the group's two lanes, then
    // of the two
    uint32_t lo = w[0], hi = w[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      lo = min2(lo, w[e]);
      hi = max2(hi, w[e]);
    }
    lo = min2(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    hi = max2(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
    if (off < 0) continue;
    const float mn = fminf(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u));
    const float mx = fmaxf(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      f[e] = (e & 1) ? __uint_as_float(w[e / 2] & 0xffff0000u) : __uint_as_float(w[e / 2] << 16);
    uint32_t scale, codes[2];
    quantise(f, mn, mx, &scale, codes);
    uint8_t* blk = a.cache + off;
    if (!is_v) {
      // elements 32 g + 16 half ..: words t = 2 half and 2 half + 1 of group g
      uint8_t* p = blk + slot * L::kRow + (2 * half * L::kGroups + g) * 4;
      *reinterpret_cast<uint32_t*>(p) = codes[0];
      *reinterpret_cast<uint32_t*>(p + L::kGroups * 4) = codes[1];
    } else {
      // half g of chunks i = 4 half .. 4 half + 3
      uint8_t* p = blk + L::v_half(slot, 4 * half, g);
      constexpr int kChunk = D / 16;
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)codes[0];
      *reinterpret_cast<uint16_t*>(p + kChunk) = (uint16_t)(codes[0] >> 16);
      *reinterpret_cast<uint16_t*>(p + 2 * kChunk) = (uint16_t)codes[1];
      *reinterpret_cast<uint16_t*>(p + 3 * kChunk) = (uint16_t)(codes[1] >> 16);
    }
    if (half == 0) {
      const uint32_t par = scale | (__float_as_uint(mn) & 0xffff0000u);
      *reinterpret_cast<uint32_t*>(blk + (is_v ? L::kOffVPar : L::kOffKPar) + slot * L::kPar +
                                   g * 4) = par;
    }
  }
}

// ------------------------------------------------------------------ read

struct ReadArgs {
  const uint8_t* cache;
  __nv_bfloat16 *k, *v;  // [B, Hkv, S, D]
  const int* first;      // [B] or null (0)
  const int* count;      // [B]
  C4Table table;
  int B, Hkv, S;
  int blocks;  // cache blocks that S slots can lie in
};

// The values of w's eight 4-bit fields, rounded to bf16.  A field masked into the
// mantissa of 2^23 is a number field * 2^k more; what the FMA sees is exact.
__device__ __forceinline__ uint4 eight_values(uint32_t w, float sc, float mn) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = e < 5 ? 4 * e : 4 * (e - 5);  // fields 5..7 after a shift by 20
    const uint32_t x = ((e < 5 ? w : w >> 20) & (15u << k)) | 0x4B000000u;
    const float c = __fsub_rn(__uint_as_float(x), 8388608.f);           // field * 2^k
    v[e] = __fmaf_rn(sc * __uint_as_float((127u - k) << 23), c, mn);  // sc 2^-k is exact
  }
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// One warp per cache block of 16 slots of a head, four lanes per key or value: a
// lane loads its quarter of the codes and the parameters in one piece each and
// stores 8 elements of every group, so eight loads are in flight per lane before
// the first store.
template <int D>
__global__ void __launch_bounds__(128) read_kernel(const ReadArgs a) {
  using L = C4<D>;
  constexpr int kG = L::kGroups;
  const int lane = threadIdx.x & 31;
  const uint32_t x = blockIdx.x * 4 + (threadIdx.x >> 5);  // below 2^31
  grid_dep_wait();
  grid_dep_launch();
  if (x >= (uint32_t)a.B * a.Hkv * a.blocks) return;
  const int bh = (int)(x / (uint32_t)a.blocks), j = (int)(x - (uint32_t)bh * a.blocks);
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int from = a.first ? a.first[b] : 0, count = min(a.count[b], a.S);
  const int first = max(from, 0);  // a negative one is out of range: rows of zeros
  const int blk = first / kC4Block + j;
  // output row of slot s of the block; rows outside [0, S) are not this warp's
  const long long row0 = (long long)blk * kC4Block - first;
  if (row0 >= a.S) return;
  if (count < 0 && j == 0 && lane == 0) c4_flag(a.table);
  int page = -1;
  if (max(row0, 0LL) < count) {  // (the first block begins before `first`)
    page = from >= 0 ? c4_page(a.table, b, blk) : -1;
    if (page < 0 && lane == 0) c4_flag(a.table);
  }
  const uint8_t* src = a.cache + (((long long)page * a.Hkv + h) * a.table.blocks_per_page() +
                                  a.table.in_page(blk)) * L::kBytes;
  const int t = lane & 3;
  uint32_t w[4][kG], par[4][kG];  // K of slots lane / 4 and + 8, V of the same
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int s = (lane >> 2) + 8 * (n & 1);
#pragma unroll
    for (int g = 0; g < kG; ++g) w[n][g] = par[n][g] = 0u;
    if (page < 0 || row0 + s < 0 || row0 + s >= count) continue;
    // words t * kG ..: K's lane piece; V's chunks 2 t and 2 t + 1
    const uint8_t* c = src + (n < 2 ? s * L::kRow + t * 4 * kG : L::v_half(s, 2 * t, 0));
    const uint8_t* q = src + (n < 2 ? L::kOffKPar : L::kOffVPar) + s * L::kPar;
    if constexpr (kG == 4) {
      const uint4 y = *reinterpret_cast<const uint4*>(c), z = *reinterpret_cast<const uint4*>(q);
      w[n][0] = y.x, w[n][1] = y.y, w[n][2] = y.z, w[n][3] = y.w;
      par[n][0] = z.x, par[n][1] = z.y, par[n][2] = z.z, par[n][3] = z.w;
    } else {
      const uint2 y = *reinterpret_cast<const uint2*>(c), z = *reinterpret_cast<const uint2*>(q);
      w[n][0] = y.x, w[n][1] = y.y;
      par[n][0] = z.x, par[n][1] = z.y;
    }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const long long row = row0 + (lane >> 2) + 8 * (n & 1);
    if (row < 0 || row >= a.S) continue;
    __nv_bfloat16* dst = (n < 2 ? a.k : a.v) + ((long long)bh * a.S + row) * D + 8 * t;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      // elements 32 g + 8 t + 0..7: K's word g; V's half g of two chunks
      uint32_t codes = w[n][g];
      if (n >= 2) {
        if constexpr (kG == 4)
          codes = __byte_perm(w[n][g / 2], w[n][2 + g / 2], (g & 1) ? 0x7632 : 0x5410);
        else
          codes = __byte_perm(w[n][0], w[n][1], (g & 1) ? 0x7632 : 0x5410);
      }
      const float sc = c4_scale(par[n][g]), mn = c4_min(par[n][g]);
      *reinterpret_cast<uint4*>(dst + 32 * g) = eight_values(codes, sc, mn);
    }
  }
}

// ------------------------------------------------------------------ evict

struct EvictArgs {
  uint8_t* cache;
  const float* weights;  // [B, Hkv, cap]
  float* weights_out;    // [B, Hkv, budget]
  int* src;              // [B, Hkv, budget]
  const int* lens;       // [B]
  int* lens_out;         // [B]
  C4Table in, out;
  int B, Hkv, cap, budget, recent;
};

constexpr int kRankThreads = 1024;

// Bit pattern that orders like the value (negative values reversed; -0 as +0).
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the block of one value per thread below this thread, and the total.
__device__ __forceinline__ int block_prefix(int x, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // s_warp may still be read from the call before
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int y = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_warp[lane] = y;
  }
  __syncthreads();
  *total = s_warp[31];
  return inc - x + (warp ? s_warp[warp - 1] : 0);
}

constexpr int kRankKeys = 16;  // weights a thread keeps in registers

__global__ void __launch_bounds__(kRankThreads) rank_kernel(const EvictArgs a) {
  __shared__ int s_hist[2048];
  __shared__ int s_warp[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  grid_dep_wait();
  grid_dep_launch();
  const int bh = blockIdx.x, b = bh / a.Hkv;
  const int cap = min(a.cap, (int)min((long long)a.in.width * a.in.blocks_per_page() * kC4Block,
                                      (long long)0x7fffffff));
  int n = a.lens[b];
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0) c4_flag(a.in);
    n = n < 0 ? 0 : cap;
  }
  const float* w = a.weights + (size_t)bh * a.cap;
  float* w_out = a.weights_out + (size_t)bh * a.budget;
  int* src = a.src + (size_t)bh * a.budget;
  const int kept = min(n, a.budget);
  for (int i = kept + threadIdx.x; i < a.budget; i += kRankThreads) {
    src[i] = -1;
    w_out[i] = 0.f;
  }
  if (n <= a.budget) {
    for (int i = threadIdx.x; i < n; i += kRankThreads) {
      src[i] = i;
      w_out[i] = w[i];
    }
    return;
  }
  const int early = n - a.recent;        // candidates; the rest are kept
  const int want = a.budget - a.recent;  // of them, the largest (0 <= want < early)
  // Thread t has weights t * per .. t * per + per - 1, in registers where they fit.
  const int per = (n + kRankThreads - 1) / kRankThreads;
  const bool cached = per <= kRankKeys;
  const int i0 = threadIdx.x * per;
  uint32_t key[kRankKeys];
  if (cached) {
#pragma unroll
    for (int x = 0; x < kRankKeys; ++x)
      if (x < per) key[x] = i0 + x < n ? order_key(w[i0 + x]) : 0u;
  }
  // the want-th largest key, a digit of 11, 11 and 10 bits at a time from the top
  uint32_t prefix = 0;
  int need = want;  // still to find among the keys that start with prefix
  for (int pass = 0; pass < 3 && want > 0; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
    s_hist[threadIdx.x] = s_hist[threadIdx.x + 1024] = 0;
    __syncthreads();
    auto visit = [&](int i, uint32_t k) {
      const bool on = i < early && (pass == 0 || (k >> (pass == 1 ? 21 : 10)) ==
                                                     (prefix >> (pass == 1 ? 21 : 10)));
      if (on) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1);
    };
    if (cached) {
#pragma unroll
      for (int x = 0; x < kRankKeys; ++x)
        if (x < per) visit(i0 + x, key[x]);
    } else {
      for (int i = threadIdx.x; i < per * kRankThreads; i += kRankThreads)
        visit(i, i < n ? order_key(w[i]) : 0u);
    }
    __syncthreads();
    // thread t has bins bins - 1 - 2 t and the one below, from the highest digit down
    const int top = bins - 1 - 2 * (int)threadIdx.x;
    const int c0 = top > 0 ? s_hist[top] : 0, c1 = top > 0 ? s_hist[top - 1] : 0;
    int total;
    const int above = block_prefix(c0 + c1, s_warp, &total);
    if (above < need && need <= above + c0 + c1) {
      const bool first = need <= above + c0;
      s_prefix = prefix | ((uint32_t)(first ? top : top - 1) << shift);
      s_need = need - above - (first ? 0 : c0);
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // In index order: keys above the threshold, the first `need` at it, the latest.
  // A thread counts what it keeps for certain and its ties, in one prefix sum over
  // the block; then it knows how many ties before it were taken.
  auto verdict = [&](int i, uint32_t k, bool* tie) {
    *tie = i < early && want > 0 && k == prefix;
    return i < n && (i >= early || (want > 0 && k > prefix));
  };
  auto put = [&](int at, int i, uint32_t k) {
    if (at >= a.budget) return;
    src[at] = i;
    w_out[at] = __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
  };
  if (cached) {
    int sure = 0, ties = 0;
#pragma unroll
    for (int x = 0; x < kRankKeys; ++x) {
      if (x >= per) continue;
      bool tie;
      sure += verdict(i0 + x, key[x], &tie) ? 1 : 0;
      ties += tie ? 1 : 0;
    }
    int total;
    const int before = block_prefix((ties << 16) | sure, s_warp, &total);  // at most 16384 each
    int ties_before = before >> 16, at = (before & 0xffff) + min(ties_before, need);
#pragma unroll
    for (int x = 0; x < kRankKeys; ++x) {
      if (x >= per) continue;
      bool tie;
      bool keep = verdict(i0 + x, key[x], &tie);
      if (tie) keep = ties_before++ < need;
      if (keep) put(at++, i0 + x, key[x]);
    }
    return;
  }
  int done = 0, ties = 0;
  for (int c = 0; c < n; c += kRankThreads) {
    const int i = c + threadIdx.x;
    const uint32_t k = i < n ? order_key(w[i]) : 0u;
    bool tie;
    bool keep = verdict(i, k, &tie);
    int total;
    const int before = block_prefix((tie ? 0x10000 : 0) | (keep ? 1 : 0), s_warp, &total);
    const int ties_before = ties + (before >> 16);
    const int at = done + (before & 0xffff) + min(ties_before, need) - min(ties, need);
    if (tie) keep = ties_before < need;
    if (keep) put(at, i, k);
    const int ties_after = ties + (total >> 16);
    done += (total & 0xffff) + min(ties_after, need) - min(ties, need);
    ties = ties_after;
  }
}

// One warp per block of 16 kept slots of a (sequence, kv head).
template <int D>
__global__ void __launch_bounds__(256) move_kernel(const EvictArgs a) {
  using L = C4<D>;
  constexpr int kPiece = D / 8;               // 16 or 8 bytes
  constexpr int kPieces = 10 * kC4Block;      // per block: 4 + 1 of K, 4 + 1 of V per slot
  using Piece = typename std::conditional<D == 128, uint4, uint2>::type;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int blocks = (a.budget + kC4Block - 1) / kC4Block;
  const uint32_t x = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);  // below 2^31
  if (x >= (uint32_t)a.B * a.Hkv * blocks) return;
  const int bh = (int)(x / (uint32_t)blocks), blk = (int)(x - (uint32_t)bh * blocks);
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  // lens_out may be lens itself: what is kept of what was kept is the same
  const long long in_slots = (long long)a.in.width * a.in.blocks_per_page() * kC4Block;
  const int kept = max(0, min(min(a.lens[b], a.budget), (int)min((long long)a.cap, in_slots)));
  if (h == 0 && blk == 0 && lane == 0) a.lens_out[b] = kept;
  const int slots = min(kC4Block, kept - blk * kC4Block);
  if (slots <= 0) return;
  // lane s: the byte offset of slot s's source block and its slot there
  long long from = -1;
  int from_slot = 0;
  if (lane < slots) {
    const int i = a.src[(size_t)bh * a.budget + blk * kC4Block + lane];
    const int page = i >= 0 ? c4_page(a.in, b, i / kC4Block) : -1;
    if (page >= 0) {
      from = (((long long)page * a.Hkv + h) * a.in.blocks_per_page() +
              a.in.in_page(i / kC4Block)) * L::kBytes;
      from_slot = i % kC4Block;
    } else {
      c4_flag(a.in);
    }
  }
  const int page = c4_page(a.out, b, blk);
  if (page < 0) {
    if (lane == 0) c4_flag(a.out);
    return;
  }
  uint8_t* dst = a.cache + (((long long)page * a.Hkv + h) * a.out.blocks_per_page() +
                            a.out.in_page(blk)) * L::kBytes;
  // piece p of slot s: 0..3 K codes, 4 K parameters, 5..8 V codes, 9 V parameters
  auto offset = [](int s, int p) {
    if (p < 4) return s * L::kRow + p * kPiece;
    if (p == 4) return L::kOffKPar + s * L::kPar;
    if (p < 9)
      return D == 128 ? L::kOffV + s * L::kRow + ((p - 5) ^ ((s & 4) >> 1)) * kPiece
                      : L::kOffV + (s ^ ((s >> 2) & 1)) * L::kRow + (p - 5) * kPiece;
    return L::kOffVPar + s * L::kPar;
  };
  Piece val[kPieces / 32];
#pragma unroll
  for (int n = 0; n < kPieces / 32; ++n) {
    const int e = n * 32 + lane, s = e / 10, p = e - 10 * s;
    const long long f = __shfl_sync(0xffffffffu, from, s);
    const int fs = __shfl_sync(0xffffffffu, from_slot, s);
    val[n] = Piece{};  // a token whose old page is out of range: zeros, as read gives it
    if (f >= 0) val[n] = *reinterpret_cast<const Piece*>(a.cache + f + offset(fs, p));
  }
#pragma unroll
  for (int n = 0; n < kPieces / 32; ++n) {
    const int e = n * 32 + lane, s = e / 10, p = e - 10 * s;
    if (s < slots) *reinterpret_cast<Piece*>(dst + offset(s, p)) = val[n];
  }
}

// ------------------------------------------------------------------ host

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace

int* cache4_status_word() {
  // looked up once per device: the lookup takes longer than the rest of a call
  static std::atomic<int*> known[64] = {};
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return nullptr;
  int* p = known[dev].load(std::memory_order_acquire);
  if (p) return p;
  if (cudaGetSymbolAddress(reinterpret_cast<void**>(&p), g_cache4_status) != cudaSuccess)
    return nullptr;
  known[dev].store(p, std::memory_order_release);
  return p;
}

// Shape rules of every cache call.
int check_cache4(int num_pages, int Hkv, int D, int page_size, int B, int width) {
  if (num_pages < 1 || Hkv < 1 || B < 1 || width < 1) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return FA_ERR_UNSUPPORTED;
  // a sequence's slots, and the rows over all sequences and heads, are counted in 32 bits
  if ((long long)width * page_size > (1LL << 30) || (long long)B * Hkv > (1LL << 30))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace fa

using namespace fa;

namespace {

C4Table make_table(const int* pages, int width, int num_pages, int page_size, int* status) {
  return C4Table{pages, width, num_pages, c4_shift(page_size), status};
}

int launch_append(void (*kernel)(AppendArgs), const AppendArgs& a, fa_stream_t stream) {
  const long long per = kAppendWarps * kAppendItems;
  const long long grid = ((long long)a.T * a.Hkv + per - 1) / per;
  if (launch_pdl(kernel, dim3((unsigned)grid), dim3(kAppendWarps * 32), 0,
                 static_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return FA_ERR_CUDA;
  note_launches(1);
  return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_cache4_page_bytes(int Hkv, int D, int page_size) {
  if (check_cache4(1, Hkv, D, page_size, 1, 1) != FA_OK) return 0;
  return (size_t)Hkv * (page_size / kC4Block) * c4_block_bytes(D);
}

int fa_cache4_append(void* cache, int num_pages, int page_size, const void* k, const void* v,
                     const fa_packed_stride* k_stride, const fa_packed_stride* v_stride, int B,
                     int T, int Hkv, int D, const int* cu_seqlens, const int* cache_lens,
                     const int* page_table, int table_width, fa_stream_t stream) {
  reset_launches();
  int rc = check_cache4(num_pages, Hkv, D, page_size, B, table_width);
  if (rc) return rc;
  if (T < 0 || (!cu_seqlens && T != B) || (long long)T * Hkv >= (1LL << 31) - 64) return FA_ERR_INVALID_ARG;
  const fa_packed_stride plain = {(int64_t)Hkv * D, D};
  const fa_packed_stride ks = k_stride ? *k_stride : plain, vs = v_stride ? *v_stride : plain;
  for (int64_t s : {ks.token, ks.head, vs.token, vs.head}) {
    if (s < 0) return FA_ERR_INVALID_ARG;
    if (s & 7) return FA_ERR_MISALIGNED;
  }
  if (T == 0) return FA_OK;
  if (!cache || !k || !v || !cache_lens || !page_table) return FA_ERR_INVALID_ARG;
  if (misaligned(cache, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(cu_seqlens, 4) ||
      misaligned(cache_lens, 4) || misaligned(page_table, 4))
    return FA_ERR_MISALIGNED;
  if ((rc = check_device())) return rc;
  int* status = cache4_status_word();
  if (!status) return FA_ERR_CUDA;
  AppendArgs a{static_cast<uint8_t*>(cache), static_cast<const __nv_bfloat16*>(k),
               static_cast<const __nv_bfloat16*>(v), ks.token, ks.head, vs.token, vs.head,
               cu_seqlens, cache_lens, nullptr,
               make_table(page_table, table_width, num_pages, page_size, status), B, T, Hkv};
  return launch_append(D == 128 ? append_kernel<128, false> : append_kernel<64, false>, a, stream);
}

int fa_cache4_append_slots(void* cache, int num_pages, int page_size, const void* k, const void* v,
                           const fa_packed_stride* k_stride, const fa_packed_stride* v_stride, int T,
                           int Hkv, int D, const int64_t* slots, fa_stream_t stream) {
  reset_launches();
  int rc = check_cache4(num_pages, Hkv, D, page_size, 1, 1);
  if (rc) return rc;
  if (T < 0 || (long long)T * Hkv >= (1LL << 31) - 64) return FA_ERR_INVALID_ARG;
  const fa_packed_stride plain = {(int64_t)Hkv * D, D};
  const fa_packed_stride ks = k_stride ? *k_stride : plain, vs = v_stride ? *v_stride : plain;
  for (int64_t s : {ks.token, ks.head, vs.token, vs.head}) {
    if (s < 0) return FA_ERR_INVALID_ARG;
    if (s & 7) return FA_ERR_MISALIGNED;
  }
  if (T == 0) return FA_OK;
  if (!cache || !k || !v || !slots) return FA_ERR_INVALID_ARG;
  if (misaligned(cache, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 8))
    return FA_ERR_MISALIGNED;
  if ((rc = check_device())) return rc;
  int* status = cache4_status_word();
  if (!status) return FA_ERR_CUDA;
  AppendArgs a{static_cast<uint8_t*>(cache), static_cast<const __nv_bfloat16*>(k),
               static_cast<const __nv_bfloat16*>(v), ks.token, ks.head, vs.token, vs.head,
               nullptr, nullptr, reinterpret_cast<const long long*>(slots),
               make_table(nullptr, 0, num_pages, page_size, status), 1, T, Hkv};
  return launch_append(D == 128 ? append_kernel<128, true> : append_kernel<64, true>, a, stream);
}

int fa_cache4_read(const void* cache, int num_pages, int page_size, void* k, void* v, int B, int Hkv,
                   int S, int D, const int* first, const int* count, const int* page_table,
                   int table_width, fa_stream_t stream) {
  reset_launches();
  int rc = check_cache4(num_pages, Hkv, D, page_size, B, table_width);
  if (rc) return rc;
  if (S < 0) return FA_ERR_INVALID_ARG;
  if (S == 0) return FA_OK;
  if (!cache || !k || !v || !count || !page_table) return FA_ERR_INVALID_ARG;
  if (misaligned(cache, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(first, 4) ||
      misaligned(count, 4) || misaligned(page_table, 4))
    return FA_ERR_MISALIGNED;
  if ((rc = check_device())) return rc;
  int* status = cache4_status_word();
  if (!status) return FA_ERR_CUDA;
  // S slots from any first one
  const int blocks = (int)(((long long)S + (first ? kC4Block - 1 : 0) + kC4Block - 1) / kC4Block);
  const long long grid = ((long long)B * Hkv * blocks + 3) / 4;
  if (grid >= (1LL << 29)) return FA_ERR_INVALID_ARG;
  ReadArgs a{static_cast<const uint8_t*>(cache), static_cast<__nv_bfloat16*>(k),
             static_cast<__nv_bfloat16*>(v), first, count,
             make_table(page_table, table_width, num_pages, page_size, status), B, Hkv, S,
             blocks};
  const auto kernel = D == 128 ? read_kernel<128> : read_kernel<64>;
  if (launch_pdl(kernel, dim3((unsigned)grid), dim3(128), 0, static_cast<cudaStream_t>(stream), a) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  note_launches(1);
  return FA_OK;
}

int fa_cache4_evict(void* cache, int num_pages, int page_size, const float* weights, int cap,
                    const int* cache_lens, const int* page_table, int table_width, int B, int Hkv,
                    int D, int budget, int recent, const int* out_page_table, int out_table_width,
                    int* src, float* weights_out, int* lens_out, fa_stream_t stream) {
  reset_launches();
  int rc = check_cache4(num_pages, Hkv, D, page_size, B, table_width);
  if (rc) return rc;
  if (out_table_width < 1 || cap < 1 || budget < 1 || recent < 0 || recent > budget ||
      (long long)out_table_width * page_size < budget)
    return FA_ERR_INVALID_ARG;
  if (!cache || !weights || !cache_lens || !page_table || !out_page_table || !src || !weights_out ||
      !lens_out)
    return FA_ERR_INVALID_ARG;
  if (misaligned(cache, 16) || misaligned(weights, 4) || misaligned(cache_lens, 4) ||
      misaligned(page_table, 4) || misaligned(out_page_table, 4) || misaligned(src, 4) ||
      misaligned(weights_out, 4) || misaligned(lens_out, 4))
    return FA_ERR_MISALIGNED;
  const long long blocks = (long long)B * Hkv * ((budget + kC4Block - 1) / kC4Block);
  if (blocks >= (1LL << 31) - 64) return FA_ERR_INVALID_ARG;
  if ((rc = check_device())) return rc;
  int* status = cache4_status_word();
  if (!status) return FA_ERR_CUDA;
  EvictArgs a{static_cast<uint8_t*>(cache), weights, weights_out, src, cache_lens, lens_out,
              make_table(page_table, table_width, num_pages, page_size, status),
              make_table(out_page_table, out_table_width, num_pages, page_size, status),
              B, Hkv, cap, budget, recent};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pdl(rank_kernel, dim3(B * Hkv), dim3(kRankThreads), 0, st, a) != cudaSuccess)
    return FA_ERR_CUDA;
  const auto kernel = D == 128 ? move_kernel<128> : move_kernel<64>;
  if (launch_pdl(kernel, dim3((unsigned)((blocks + 7) / 8)), dim3(256), 0, st, a) != cudaSuccess)
    return FA_ERR_CUDA;
  note_launches(2);
  return FA_OK;
}

int fa_cache4_status(fa_stream_t stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_cache4_status, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_cache4_status, &zero, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return v;
}

}  // extern "C"
