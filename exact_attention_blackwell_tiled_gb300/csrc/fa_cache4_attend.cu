// fa_cache4_attend.cu -- one query token per sequence attends to its 4-bit cache
// (cache4.cuh), with the keys' softmax weights added to a running sum on request.
//
//   s_j = scale q . k_j,  k_j = m_j + c_j z_j  per group of 32 elements (minimum m,
//   scale c, codes z), so  q . k_j = sum_g c_jg (q_g . z_jg) + m_jg sum(q_g):
// the codes, small integers, go to the matrix instruction exactly, as does the
// bf16 query, and the scales are applied to its fp32 result.  Codes become bf16
// numbers by placing their bits in the mantissa of 16.0 or 128.0 (one and-or,
// and a shift for three of four); with z' = z + off the score is
//   sum_g c_jg (q_g . z'_jg) + sum_g [c_jg, m_jg] . [-sum(off q_g), sum(q_g)]
// whose second part is one more small product: a lane's stored parameter word is
// its A fragment as it stands, and the sums, split into three bf16 parts each (24
// bits), are the B fragments, made once per row.  For the values
//   O = sum_j p_j (m_j + 8 c_j) + sum_j (p_j c_j) (z_j - 8)
// the first sum stays in fp32 and p_j c_j is rounded to bf16 for the second, the
// only rounding before O's own.  (z - 8, not z' with a correction at the end:
// over a long cache the offset's accumulation error would outgrow O.)
//
// Bound by memory: a key and its value are 5/2 D bytes of codes and parameters,
// read once for all query heads of the kv head (up to 8 NT of them, the columns of
// the products); the arithmetic to unpack them is about 20 warp instructions per
// key, 0.7 of what the SM can issue in the time the bytes take.
//
// Every warp works by itself: the 16-slot blocks of all (sequence, kv head) rows
// lie in one list, and each warp takes an equal contiguous share of it, streams it
// through a ring of its own in shared memory (bulk copies that its lane 0 issues,
// an mbarrier per stage) and keeps maximum, sum and O of the row at hand in
// registers.  So sequences of any lengths load the SMs evenly with no barrier
// between warps.  A row that lies inside one share is finished there; a row cut
// by shares leaves parts (fp32 O, maximum, sum), at most two per warp, which a
// second kernel joins; it also writes the rows of empty sequences.  A third, when
// weights are asked for, turns the stored scores into them, now that the sums are
// known.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "cache4.cuh"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kWarps = 4;      // per block; they share nothing but the launch
constexpr int kJoinThreads = 256;
constexpr int kWeightKeys = 1024;  // keys of a (sequence, kv head) per step of the weight pass

struct AttendArgs {
  const __nv_bfloat16* q;
  long long q_batch, q_head;
  const uint8_t* cache;
  __nv_bfloat16* o;
  float* lse;
  const int* lens;
  C4Table table;
  int B, Hq, Hkv, group;
  int tiles;  // query-head tiles of 8 NT per kv head
  int cap;    // slots a sequence may have
  float scale_log2;
  int n_warps;
  float* part_o;    // [n_warps, 2, 8 NT, D]
  float2* part_ml;  // [n_warps, 2, 8 NT]: maximum (log2 units) and sum
  float* scores;    // [B, Hkv, cap, group] in log2 units, or null
  float* lse2;      // [B, Hq] log2 of the sums, for the weights
  const float* w_in;
  float* w_out;  // [B, Hkv, w_stride]
  int w_stride;
};

// Fewest 16-slot blocks worth a warp of its own: with fewer, the parts to join
// cost more than the work split off.
constexpr int kMinBlocks = 4;

// A warp's ring of blocks in shared memory, filled kFill at a time: 10 KB, so that
// 16 warps keep up to 160 KB on their way to an SM (the bytes that cover the
// memory's latency at its full rate are about 45 KB).
template <int D>
struct Ring {
  static constexpr int kCount = D == 128 ? 4 : 8;
  static constexpr int kFill = kCount / 2;
  static constexpr int kBytes = kCount * C4<D>::kBytes;
};

__device__ __forceinline__ int seq_len(const AttendArgs& a, int b) {
  const int n = a.lens[b];
  return n < 0 ? 0 : (n < a.cap ? n : a.cap);
}

__device__ __forceinline__ int seq_blocks(const AttendArgs& a, int b) {
  return (seq_len(a, b) + kC4Block - 1) / kC4Block;
}

// Blocks of the whole list, by a whole warp: rows (b, kv head, tile) in order,
// row by row.
__device__ long long list_blocks(const AttendArgs& a) {
  long long n = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) n += seq_blocks(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * a.Hkv * a.tiles;
}

// The sequence whose entries hold position x, and its first position; a sequence
// has `unit(b)` x mult entries.  By a whole warp; x lies inside the list.
template <typename Unit>
__device__ int locate(const AttendArgs& a, long long x, int mult, Unit unit, long long* base) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const long long n = b0 + lane < a.B ? (long long)unit(b0 + lane) * mult : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x < before + inc);
    if (hit) {
      const int l = __ffs(hit) - 1;
      *base = before + __shfl_sync(0xffffffffu, inc - n, l);
      return b0 + l;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  *base = before;
  return a.B;
}

// Shares: warp w of W takes list positions w N / W .. (w + 1) N / W - 1.
__device__ __forceinline__ int share_count(const AttendArgs& a, long long N) {
  const long long most = (N + kMinBlocks - 1) / kMinBlocks;
  return (int)(most < a.n_warps ? most : a.n_warps);
}
__device__ __forceinline__ long long share_begin(long long N, int W, int w) { return w * N / W; }
__device__ __forceinline__ int share_of(long long N, int W, long long x) {
  return (int)(((x + 1) * W - 1) / N);
}

// A place in the warp's share: row (b, hk, tile) = (b, row / tiles, row % tiles),
// next block blk of it, and where the share or the row ends.
struct Cursor {
  int b, row, blk, end, nb;
  long long left;  // blocks of the share from blk on
};

__device__ __forceinline__ void cursor_row(Cursor& c) {
  const long long e = c.blk + c.left;
  c.end = (int)(e < c.nb ? e : c.nb);
}

// Past n blocks; at a row's end on to the next row that has blocks.
__device__ __forceinline__ void cursor_advance(const AttendArgs& a, Cursor& c, int n) {
  c.blk += n;
  c.left -= n;
  if (c.left <= 0 || c.blk < c.end) return;
  c.blk = 0;
  if (++c.row == a.Hkv * a.tiles) {
    c.row = 0;
    do {
      ++c.b;
    } while (c.b < a.B && (c.nb = seq_blocks(a, c.b)) == 0);
    if (c.b >= a.B) {  // not reached: the share ends inside the list
      c.left = 0;
      return;
    }
  }
  cursor_row(c);
}

// ------------------------------------------------------------------ fragments

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// ... with K = 8 and the accumulator starting at c.
__device__ __forceinline__ void mma1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// mma16816 on a zero accumulator.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 4-bit field R of the low and of the high half of w as bf16 numbers field + kOff<R>.
template <int R>
constexpr float kOff = R == 0 ? 128.f : 16.f;
template <int R>
__device__ __forceinline__ uint32_t offset_code(uint32_t w) {
  if constexpr (R == 0) return (w & 0x000f000fu) | 0x43004300u;
  else return ((w >> (4 * R - 3)) & 0x00780078u) | 0x41804180u;
}

// ... as field - 8 (exact).
template <int R>
__device__ __forceinline__ uint32_t minus8(uint32_t w) {
  const uint32_t x = offset_code<R>(w);
  const __nv_bfloat16 k = __ushort_as_bfloat16(R == 0 ? 0x4308 : 0x41C0);  // 136, 24
  const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), __nv_bfloat162(k, k));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// x as three bf16 parts (their sum is x to 24 bits).
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&p)[3]) {
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    p[e] = __float2bfloat16_rn(x);
    x -= __bfloat162float(p[e]);
  }
}

__device__ __forceinline__ uint32_t pair16(__nv_bfloat16 lo, __nv_bfloat16 hi) {
  return (uint32_t)__bfloat16_as_ushort(lo) | ((uint32_t)__bfloat16_as_ushort(hi) << 16);
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&r)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    r[0] = x.x, r[1] = x.y;
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

__device__ __forceinline__ void copy_block(uint32_t dst, const void* src, uint32_t bytes,
                                           uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// ------------------------------------------------------------------ main kernel

// Registers of a row in progress.  Lane 4 i + t holds query columns 2 t and
// 2 t + 1 of every 8-column tile.
template <int D, int NT>
struct RowState {
  static constexpr int kG = D / 32;
  float acc[2 * kG][NT][4];  // O^T: tile 2 g + x, rows i and i + 8 are elements 32 g + 4 i + 2 x, + 1
  float mid[kG][NT][2];      // this lane's sum of p (m + 8 c)
  float m[NT][2], l[NT][2];  // maximum (log2 units; the same in the lanes of one t), lane's sum
};

// A row's log-sum-exp from its maximum and sum.
__device__ __forceinline__ void write_lse(const AttendArgs& a, size_t row, float m, float l) {
  const float z = l > 0.f ? m + __log2f(l) : -INFINITY;
  a.lse[row] = z * 0.69314718055994531f;
  if (a.scores) a.lse2[row] = z;
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 2) attend_kernel(const AttendArgs a) {
  using L = C4<D>;
  using R = Ring<D>;
  constexpr int kG = L::kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ alignas(8) uint64_t s_bar[kWarps][R::kCount];
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, t = lane & 3;
  const uint8_t* ring = smem + warp * R::kBytes;
  const uint32_t bars = smem_u32(&s_bar[warp][0]);
  if (threadIdx.x == 0) s_abort = 0;
  if (lane < R::kCount) mbar_init(bars + 8 * lane, 1);
  fence_mbarrier_init();
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const long long N = list_blocks(a);
  if (N == 0) return;
  const int W = share_count(a, N);
  const int w = blockIdx.x + warp * gridDim.x;  // neighbouring shares on different SMs
  if (w >= W) return;
  const long long begin = share_begin(N, W, w), end = share_begin(N, W, w + 1);

  Cursor head;  // of the copies; the products follow behind it
  {
    long long base;
    head.b = locate(a, begin, a.Hkv * a.tiles, [&](int b) { return seq_blocks(a, b); }, &base);
    head.nb = seq_blocks(a, head.b);
    const long long r = begin - base;
    head.row = (int)(r / head.nb);
    head.blk = (int)(r - (long long)head.row * head.nb);
    head.left = end - begin;
    cursor_row(head);
  }
  Cursor cur = head;
  int win_b = -1, win = 0, win_page = -1;  // page of block win + lane of sequence win_b
  uint32_t issued = 0, n = 0;              // blocks copied (or on their way) and consumed
  uint32_t have_bits = 0;                  // bit (block number & 31): its page was in range
  const int page_mask = a.table.blocks_per_page - 1;
  // Copies the next blocks of the head's row, at most kFill: a lane each.
  auto fill = [&]() {
    if (head.left <= 0) return;
    const int count = min(R::kFill, head.end - head.blk);
    if (head.b != win_b || head.blk < win || head.blk + count > win + 32) {
      win_b = head.b;
      win = head.blk;
      win_page = win + lane < head.nb ? c4_page(a.table, win_b, win + lane) : -1;
    }
    const int page = __shfl_sync(0xffffffffu, win_page, (head.blk + lane - win) & 31);
    const uint32_t good = __ballot_sync(0xffffffffu, lane < count && page >= 0);
    if (lane < count) {
      const int s = (issued + lane) % R::kCount;
      const uint32_t bar = bars + 8 * s;
      mbar_arrive_expect_tx(bar, page >= 0 ? L::kBytes : 0);
      if (page >= 0)
        copy_block(smem_u32(ring) + s * L::kBytes,
                   a.cache + (((long long)page * a.Hkv + head.row / a.tiles) *
                                  a.table.blocks_per_page + ((head.blk + lane) & page_mask)) * L::kBytes,
                   L::kBytes, bar);
      else
        c4_flag(a.table);
    }
    const uint32_t mask = (1u << count) - 1;
    have_bits = (have_bits & ~__funnelshift_l(mask, mask, issued & 31)) |
                __funnelshift_l(good, good, issued & 31);
    issued += count;
    cursor_advance(a, head, count);
  };
  for (int s = 0; s < R::kCount / R::kFill; ++s) fill();

  const int slot_i = i ^ ((i >> 1) & 1);  // slot of product row i; row i + 8 is slot_i + 8
  // this lane's value slots: product rows 2 t and 2 t + 1 (and those + 8)
  const int va = (2 * t) ^ (t & 1), vb = (2 * t + 1) ^ (t & 1);
  while (cur.left > 0) {
    // ---- a row: its queries
    const int row_b = cur.b, hk = cur.row / a.tiles, tile = cur.row - hk * a.tiles;
    const int blk0 = cur.blk, blk1 = cur.end, nb = cur.nb;
    const int len = seq_len(a, row_b);
    const int heads = min(8 * NT, a.group - tile * 8 * NT);  // real query columns
    uint32_t qf[kG][NT][4];  // B fragments: steps 2 g (0, 1) and 2 g + 1 (2, 3)
    uint32_t qp[NT][3];      // B fragments of the parameter product
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = nt * 8 + i;
      const __nv_bfloat16* src =
          a.q + row_b * a.q_batch + (long long)(hk * a.group + tile * 8 * NT + col) * a.q_head + 8 * t;
      float sum_t = 0.f, off_t = 0.f;  // of this lane's group in the parameter product
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (col < heads) x = *reinterpret_cast<const uint4*>(src + 32 * g);
        // elements 0..7 in pairs x.x = (0,1) .. x.w = (6,7)
        qf[g][nt][0] = __byte_perm(x.x, x.z, 0x5410);  // (0, 4): fields 0
        qf[g][nt][1] = __byte_perm(x.x, x.z, 0x7632);  // (1, 5): fields 1
        qf[g][nt][2] = __byte_perm(x.y, x.w, 0x5410);  // (2, 6): fields 2
        qf[g][nt][3] = __byte_perm(x.y, x.w, 0x7632);  // (3, 7): fields 3
        float sum = 0.f, first = 0.f;
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = __uint_as_float(xs[e] << 16), hi = __uint_as_float(xs[e] & 0xffff0000u);
          if ((e & 1) == 0) first += lo;  // elements 0 and 4
          sum += lo + hi;
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
          first += __shfl_xor_sync(0xffffffffu, first, o);
        }
        if (g == (t & (kG - 1))) {
          sum_t = sum;
          off_t = kOff<1> * sum + (kOff<0> - kOff<1>) * first;
        }
      }
      __nv_bfloat16 sp[3], op[3];
      split3(sum_t, sp);
      split3(-off_t, op);
      // k index 2 t is the scale, 2 t + 1 the minimum, of group t (D = 128), with
      // parts 0 and 1, then 2; at D = 64 lanes t >= 2 take part 2 of group t - 2
      if constexpr (D == 128) {
        qp[nt][0] = pair16(op[0], sp[0]);
        qp[nt][1] = pair16(op[1], sp[1]);
        qp[nt][2] = pair16(op[2], sp[2]);
      } else {
        qp[nt][0] = t < 2 ? pair16(op[0], sp[0]) : pair16(op[2], sp[2]);
        qp[nt][1] = t < 2 ? pair16(op[1], sp[1]) : 0u;
        qp[nt][2] = 0u;
      }
    }
    RowState<D, NT> r;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2 * kG; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) r.acc[x][nt][e] = 0.f;
#pragma unroll
      for (int g = 0; g < kG; ++g) r.mid[g][nt][0] = r.mid[g][nt][1] = 0.f;
      r.m[nt][0] = r.m[nt][1] = -INFINITY;
      r.l[nt][0] = r.l[nt][1] = 0.f;
    }
    float* score = nullptr;  // of this lane's first column and row i's key
    if (a.scores)
      score = a.scores + (((size_t)row_b * a.Hkv + hk) * a.cap + blk0 * kC4Block + slot_i) * a.group +
              tile * 8 * NT + 2 * t;
    // ---- its blocks
#pragma unroll 1
    for (int at = blk0; at < blk1; ++at) {
      const bool ok = mbar_wait(bars + 8 * (n % R::kCount), (n / R::kCount) & 1, &s_abort);
      if (!__all_sync(0xffffffffu, ok)) {
        // give up, once the copies under way have landed (or that wait runs out too)
        if (lane == 0) {
          atomicExch(a.table.status, (int)FA_ERR_TIMEOUT);
          for (uint32_t f = n; f < issued; ++f) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bars + 8 * (f % R::kCount), (f / R::kCount) & 1))
              if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
          }
        }
        __syncwarp();
        return;
      }
      const uint8_t* blk = ring + (n % R::kCount) * L::kBytes;
      // scores of 16 keys: [0, 1] row i, [2, 3] row i + 8
      float sc[NT][4];
      {
        uint32_t k0[kG], k1[kG], p0[kG], p1[kG];
        const uint8_t* par = blk + L::kOffKPar + slot_i * L::kPar;
        lds(k0, blk + slot_i * L::kRow + t * 4 * kG);
        lds(k1, blk + (slot_i + 8) * L::kRow + t * 4 * kG);
        lds(p0, par);
        lds(p1, par + 8 * L::kPar);
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(par + (t & (kG - 1)) * 4);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(par + 8 * L::kPar + (t & (kG - 1)) * 4);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816_first(sc[nt], w0, w1, w0, w1, qp[nt][0], qp[nt][1]);
          if constexpr (D == 128) mma1688(sc[nt], w0, w1, qp[nt][2]);
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const uint32_t a00 = offset_code<0>(k0[g]), a01 = offset_code<1>(k0[g]),
                         a02 = offset_code<2>(k0[g]), a03 = offset_code<3>(k0[g]);
          const uint32_t a10 = offset_code<0>(k1[g]), a11 = offset_code<1>(k1[g]),
                         a12 = offset_code<2>(k1[g]), a13 = offset_code<3>(k1[g]);
          const float c0 = c4_scale(p0[g]), c1 = c4_scale(p1[g]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4];
            mma16816_first(d, a00, a10, a01, a11, qf[g][nt][0], qf[g][nt][1]);
            mma16816(d, a02, a12, a03, a13, qf[g][nt][2], qf[g][nt][3]);
            sc[nt][0] = fmaf(c0, d[0], sc[nt][0]);
            sc[nt][1] = fmaf(c0, d[1], sc[nt][1]);
            sc[nt][2] = fmaf(c1, d[2], sc[nt][2]);
            sc[nt][3] = fmaf(c1, d[3], sc[nt][3]);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] *= a.scale_log2;
      // a block with slots behind the last key, or whose page is out of range
      const int left = len - at * kC4Block - slot_i;  // row i has a key iff left > 0
      const bool have = (have_bits >> (n & 31)) & 1;
      const bool full = have && (at + 1) * kC4Block <= len;
      const bool live0 = have && left > 0, live1 = have && left > 8;
      if (!full) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = (e < 2 ? live0 : live1) ? sc[nt][e] : -INFINITY;
      }
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // a stale maximum stands until a score passes it by 8 (weights up to 2^8)
        grow |= fmaxf(sc[nt][0], sc[nt][2]) > r.m[nt][0] + 8.f;
        grow |= fmaxf(sc[nt][1], sc[nt][3]) > r.m[nt][1] + 8.f;
      }
      if (a.scores) {
        float* next = score + 8 * a.group;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int col = nt * 8 + 2 * t;
          if ((a.group & 1) == 0) {
            if (col < heads) {
              if (left > 0) *reinterpret_cast<float2*>(score + nt * 8) = make_float2(sc[nt][0], sc[nt][1]);
              if (left > 8) *reinterpret_cast<float2*>(next + nt * 8) = make_float2(sc[nt][2], sc[nt][3]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (col + c < heads) {
                if (left > 0) score[nt * 8 + c] = sc[nt][c];
                if (left > 8) next[nt * 8 + c] = sc[nt][2 + c];
              }
          }
        }
        score += 16 * a.group;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(sc[nt][c], sc[nt][2 + c]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (mx > r.m[nt][c]) {
              const float f = ex2_mufu(r.m[nt][c] - mx);  // 0 from -inf
              r.m[nt][c] = mx;
              r.l[nt][c] *= f;
#pragma unroll
              for (int x2 = 0; x2 < 2 * kG; ++x2) {
                r.acc[x2][nt][c] *= f;
                r.acc[x2][nt][2 + c] *= f;
              }
#pragma unroll
              for (int g = 0; g < kG; ++g) r.mid[g][nt][c] *= f;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float n0 = r.m[nt][0] == -INFINITY ? 0.f : r.m[nt][0];
        const float n1 = r.m[nt][1] == -INFINITY ? 0.f : r.m[nt][1];
        sc[nt][0] = ex2_mufu(sc[nt][0] - n0);
        sc[nt][1] = ex2_mufu(sc[nt][1] - n1);
        sc[nt][2] = ex2_mufu(sc[nt][2] - n0);
        sc[nt][3] = ex2_mufu(sc[nt][3] - n1);
        r.l[nt][0] += sc[nt][0] + sc[nt][2];
        r.l[nt][1] += sc[nt][1] + sc[nt][3];
      }
      uint32_t v[4][(kG + 1) / 2], p0[kG], p1[kG];
      lds(v[0], blk + L::v_half(va, i, 0));
      lds(v[1], blk + L::v_half(vb, i, 0));
      lds(v[2], blk + L::v_half(va + 8, i, 0));
      lds(v[3], blk + L::v_half(vb + 8, i, 0));
      lds(p0, blk + L::kOffVPar + slot_i * L::kPar);
      lds(p1, blk + L::kOffVPar + (slot_i + 8) * L::kPar);
      if (!full) {
        // a slot without a key holds anything: its parameters count as zero
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          p0[g] = live0 ? p0[g] : 0u;
          p1[g] = live1 ? p1[g] : 0u;
        }
      }
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const float c0 = c4_scale(p0[g]), m0 = fmaf(8.f, c0, c4_min(p0[g]));
        const float c1 = c4_scale(p1[g]), m1 = fmaf(8.f, c1, c4_min(p1[g]));
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          r.mid[g][nt][0] = fmaf(sc[nt][0], m0, fmaf(sc[nt][2], m1, r.mid[g][nt][0]));
          r.mid[g][nt][1] = fmaf(sc[nt][1], m0, fmaf(sc[nt][3], m1, r.mid[g][nt][1]));
          b0[nt] = transpose8x8(pack_bf16x2(sc[nt][0] * c0, sc[nt][1] * c0));
          b1[nt] = transpose8x8(pack_bf16x2(sc[nt][2] * c1, sc[nt][3] * c1));
        }
        constexpr uint32_t kLow = 0x5410, kHigh = 0x7632;
        const uint32_t y0 = __byte_perm(v[0][g / 2], v[1][g / 2], (g & 1) ? kHigh : kLow);
        const uint32_t y1 = __byte_perm(v[2][g / 2], v[3][g / 2], (g & 1) ? kHigh : kLow);
        const uint32_t e0 = minus8<0>(y0), e1 = minus8<1>(y0), e2 = minus8<2>(y0), e3 = minus8<3>(y0);
        const uint32_t f0 = minus8<0>(y1), f1 = minus8<1>(y1), f2 = minus8<2>(y1), f3 = minus8<3>(y1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(r.acc[2 * g][nt], e0, e1, f0, f1, b0[nt], b1[nt]);
          mma16816(r.acc[2 * g + 1][nt], e2, e3, f2, f3, b0[nt], b1[nt]);
        }
      }
      ++n;
      if (issued - n <= R::kCount - R::kFill) {
        __syncwarp();  // every lane has read the blocks whose places are filled again
        fill();
      }
    }
    cursor_advance(a, cur, blk1 - blk0);
    // ---- the row's result, or this share's part of it
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          r.l[nt][c] += __shfl_xor_sync(0xffffffffu, r.l[nt][c], o);
#pragma unroll
          for (int g = 0; g < kG; ++g)
            r.mid[g][nt][c] += __shfl_xor_sync(0xffffffffu, r.mid[g][nt][c], o);
        }
      }
    const bool whole = blk0 == 0 && blk1 == nb;
    const size_t part = ((size_t)w * 2 + (blk0 == 0 ? 1 : 0)) * (8 * NT);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = nt * 8 + 2 * t + c;
        if (col >= heads) continue;
        const float l = r.l[nt][c], m = r.m[nt][c];
        const float inv = whole ? (l > 0.f ? 1.0f / l : 0.f) : 1.f;
        const size_t out = (size_t)row_b * a.Hq + hk * a.group + tile * 8 * NT + col;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const float mid = r.mid[g][nt][c];
          const float x0 = (r.acc[2 * g][nt][c] + mid) * inv;
          const float x1 = (r.acc[2 * g][nt][2 + c] + mid) * inv;
          const float x2 = (r.acc[2 * g + 1][nt][c] + mid) * inv;
          const float x3 = (r.acc[2 * g + 1][nt][2 + c] + mid) * inv;
          if (whole)
            *reinterpret_cast<uint2*>(a.o + out * D + 32 * g + 4 * i) =
                make_uint2(pack_bf16x2(x0, x1), pack_bf16x2(x2, x3));
          else
            *reinterpret_cast<float4*>(a.part_o + (part + col) * D + 32 * g + 4 * i) =
                make_float4(x0, x1, x2, x3);
        }
        if (i == 0) {
          if (whole)
            write_lse(a, out, m, l);
          else
            a.part_ml[part + col] = make_float2(m, l);
        }
      }
  }
}

// ------------------------------------------------------------------ join and weights

// Where row (b, hk, tile)'s blocks lie in the list, and the shares that hold them.
struct RowSpan {
  int w0, w1;  // first and last share; w0 == w1: the row was finished by it
  int nb;
};

__device__ RowSpan row_span(const AttendArgs& a, long long N, int b, int row) {
  RowSpan s{0, 0, seq_blocks(a, b)};
  if (s.nb == 0) return s;
  long long before = 0;
  for (int x = threadIdx.x & 31; x < b; x += 32) before += seq_blocks(a, x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const long long first = before * a.Hkv * a.tiles + (long long)row * s.nb;
  const int W = share_count(a, N);
  s.w0 = share_of(N, W, first);
  s.w1 = share_of(N, W, first + s.nb - 1);
  return s;
}

// Index of column col of the part that share w of the row holds.
template <int NT>
__device__ __forceinline__ size_t part_index(const RowSpan& s, int w, int col) {
  return ((size_t)w * 2 + (w == s.w0 ? 1 : 0)) * (8 * NT) + col;
}

// Maximum and sum over a cut row's parts, by a whole warp.
template <int NT>
__device__ float2 join_ml(const AttendArgs& a, const RowSpan& s, int col) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
  for (int w = s.w0 + lane; w <= s.w1; w += 32) {
    const float2 x = a.part_ml[part_index<NT>(s, w, col)];
    if (x.y > 0.f) {
      const float mm = fmaxf(m, x.x);
      l = l * ex2_mufu(m - mm) + x.y * ex2_mufu(x.x - mm);
      m = mm;
    }
  }
  float mx = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  l = l > 0.f ? l * ex2_mufu(m - mx) : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  return make_float2(mx, l);
}

// One block per (sequence, query head) whose row was cut by shares, or is empty.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttendArgs a) {
  constexpr int kV = D / 32, kW = kJoinThreads / 32;
  __shared__ float s_o[kW][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The lengths were complete before the attention kernel let this one start, so
  // they are read, and the row's parts found, while it still runs.
  const long long N = list_blocks(a);
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x - b * a.Hq;
  const int hk = hq / a.group, in_group = hq - hk * a.group;
  const int tile = in_group / (8 * NT), col = in_group - tile * 8 * NT;
  const RowSpan s = row_span(a, N, b, hk * a.tiles + tile);
  grid_dep_wait();
  grid_dep_launch();
  if (hq == 0 && threadIdx.x == 0 && a.lens[b] != seq_len(a, b)) c4_flag(a.table);
  __nv_bfloat16* o = a.o + (size_t)blockIdx.x * D;
  if (s.nb == 0) {  // an empty sequence
    if (threadIdx.x < D / 2) reinterpret_cast<uint32_t*>(o)[threadIdx.x] = 0u;
    if (threadIdx.x == 0) write_lse(a, blockIdx.x, 0.f, 0.f);
    return;
  }
  if (s.w0 == s.w1) return;
  const float2 ml = join_ml<NT>(a, s, col);
  float acc[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int w = s.w0 + warp; w <= s.w1; w += kW) {
    const size_t p = part_index<NT>(s, w, col);
    const float2 x = a.part_ml[p];
    const float f = x.y > 0.f ? ex2_mufu(x.x - ml.x) : 0.f;
    const float* src = a.part_o + p * D + lane * kV;
    float v[kV];
    if constexpr (kV == 4) {
      const float4 y = *reinterpret_cast<const float4*>(src);
      v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(src);
      v[0] = y.x, v[1] = y.y;
    }
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = fmaf(f, v[e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < kV; ++e) s_o[warp][lane * kV + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D / 2) {
    const float inv = ml.y > 0.f ? 1.0f / ml.y : 0.f;
    float x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int y = 0; y < kW; ++y) {
      x0 += s_o[y][2 * threadIdx.x];
      x1 += s_o[y][2 * threadIdx.x + 1];
    }
    reinterpret_cast<uint32_t*>(o)[threadIdx.x] = pack_bf16x2(x0 * inv, x1 * inv);
  }
  if (threadIdx.x == 0) write_lse(a, blockIdx.x, ml.x, ml.y);
}

// w_out = w_in + sum over the group of 2^(score - log2 sum), for kWeightKeys keys of
// a (sequence, kv head) per block.
__global__ void __launch_bounds__(256) weight_kernel(const AttendArgs a) {
  __shared__ float s_lse2[128];
  const int b = blockIdx.z, hk = blockIdx.y, len = seq_len(a, b);
  const int j0 = blockIdx.x * kWeightKeys;
  constexpr int kPer = kWeightKeys / 256;
  const size_t row = (size_t)b * a.Hkv + hk;
  float w[kPer];
  if (j0 < len && a.w_in) {
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int j = j0 + x * 256 + threadIdx.x;
      w[x] = j < len ? a.w_in[row * a.w_stride + j] : 0.f;
    }
  } else {
#pragma unroll
    for (int x = 0; x < kPer; ++x) w[x] = 0.f;
  }
  grid_dep_wait();
  grid_dep_launch();
  if (j0 >= len) return;
  if (threadIdx.x < a.group) s_lse2[threadIdx.x] = a.lse2[(size_t)b * a.Hq + hk * a.group + threadIdx.x];
  __syncthreads();
  const bool empty = s_lse2[0] == -INFINITY;  // every page out of range
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int j = j0 + x * 256 + threadIdx.x;
    if (j >= len) break;
    const float* src = a.scores + (row * a.cap + j) * a.group;
    float sum = 0.f;
    if ((a.group & 3) == 0) {
      for (int h = 0; h < a.group; h += 4) {
        const float4 s = *reinterpret_cast<const float4*>(src + h);
        sum += (ex2_mufu(s.x - s_lse2[h]) + ex2_mufu(s.y - s_lse2[h + 1])) +
               (ex2_mufu(s.z - s_lse2[h + 2]) + ex2_mufu(s.w - s_lse2[h + 3]));
      }
    } else {
      for (int h = 0; h < a.group; ++h) sum += ex2_mufu(src[h] - s_lse2[h]);
    }
    a.w_out[row * a.w_stride + j] = w[x] + (empty ? 0.f : sum);
  }
}

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Query heads of a kv head: one 8-column tile, or two at a time.
int tile_count(int group, int* nt) {
  *nt = group <= 8 ? 1 : 2;
  return (group + 8 * *nt - 1) / (8 * *nt);
}

// Shares: every warp that is resident at once.
int share_limit(int sms, int nt) { return sms * (nt == 1 ? 4 : 2) * kWarps; }

struct AttendLayout {
  size_t off_ml, off_lse2, off_scores, total;
};

AttendLayout attend_layout(int B, int Hq, int Hkv, int D, int cap, int sms) {
  int nt;
  tile_count(Hq / Hkv, &nt);
  const size_t rows = (size_t)share_limit(sms, nt) * 2 * 8 * nt;
  AttendLayout L;
  L.off_ml = rows * D * sizeof(float);
  L.off_lse2 = (L.off_ml + rows * sizeof(float2) + 255) & ~(size_t)255;
  L.off_scores = (L.off_lse2 + (cap > 0 ? (size_t)B * Hq * sizeof(float) : 0) + 255) & ~(size_t)255;
  L.total = L.off_scores + (size_t)B * Hq * cap * sizeof(float);
  return L;
}

template <int D, int NT>
int launch_attend(const AttendArgs& a, cudaStream_t stream) {
  constexpr int kSmem = kWarps * Ring<D>::kBytes;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  static bool attr_done[64] = {};
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(attend_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem) != cudaSuccess)
      return FA_ERR_CUDA;
    attr_done[dev] = true;
  }
  record_timing(false, stream);
  if (launch_pdl(attend_kernel<D, NT>, dim3(a.n_warps / kWarps), dim3(kWarps * 32), kSmem, stream,
                 a) != cudaSuccess)
    return FA_ERR_CUDA;
  record_timing(true, stream);
  if (launch_pdl(join_kernel<D, NT>, dim3(a.B * a.Hq), dim3(kJoinThreads), 0, stream, a) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  int launches = 2;
  if (a.scores) {
    const dim3 grid((a.cap + kWeightKeys - 1) / kWeightKeys, a.Hkv, a.B);
    if (launch_pdl(weight_kernel, grid, dim3(256), 0, stream, a) != cudaSuccess) return FA_ERR_CUDA;
    ++launches;
  }
  note_launches(launches);
  return FA_OK;
}

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_cache4_attend_workspace_bytes(int B, int Hq, int Hkv, int D, int weight_slots) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (D != 64 && D != 128) || weight_slots < 0)
    return 0;
  int dev;
  DeviceInfo info;
  const int sms = current_device(&dev, &info) ? info.sm_count : 0;
  if (sms < 1) return 0;
  return attend_layout(B, Hq, Hkv, D, weight_slots, sms).total;
}

int fa_cache4_attend(const void* q, int64_t q_batch_stride, int64_t q_head_stride, const void* cache,
                     int num_pages, int page_size, void* o, float* lse, int B, int Hq, int Hkv,
                     int D, const int* cache_lens, const int* page_table, int table_width,
                     float scale, const float* weights_in, float* weights_out, int weight_slots,
                     void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  reset_launches();
  int rc = check_cache4(num_pages, Hkv, D, page_size, B, table_width);
  if (rc) return rc;
  if (Hq < 1 || Hq % Hkv != 0 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (Hq / Hkv > 128) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Hq > (1LL << 30)) return FA_ERR_INVALID_ARG;
  if (weights_out && (B > 65535 || Hkv > 65535)) return FA_ERR_UNSUPPORTED;  // its launch grid
  if (q_batch_stride < 0 || q_head_stride < 0) return FA_ERR_INVALID_ARG;
  if ((q_batch_stride & 7) || (q_head_stride & 7)) return FA_ERR_MISALIGNED;
  if (!q || !cache || !o || !lse || !cache_lens || !page_table) return FA_ERR_INVALID_ARG;
  if ((weights_out && weight_slots < 1) || (weights_in && !weights_out)) return FA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(cache, 16) || misaligned(o, 16) || misaligned(lse, 4) ||
      misaligned(cache_lens, 4) || misaligned(page_table, 4) || misaligned(weights_in, 4) ||
      misaligned(weights_out, 4))
    return FA_ERR_MISALIGNED;
  if (!workspace || misaligned(workspace, 256)) return FA_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  const int slots = table_width * page_size;
  AttendArgs a{};
  a.cap = weights_out ? (weight_slots < slots ? weight_slots : slots) : slots;
  const AttendLayout L = attend_layout(B, Hq, Hkv, D, weights_out ? a.cap : 0, info.sm_count);
  if (workspace_bytes < L.total) return FA_ERR_WORKSPACE;
  int* status = cache4_status_word();
  if (!status) return FA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int nt;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_batch = q_batch_stride;
  a.q_head = q_head_stride;
  a.cache = static_cast<const uint8_t*>(cache);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.lens = cache_lens;
  a.table = C4Table{page_table, table_width, num_pages, page_size / kC4Block, status};
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.tiles = tile_count(a.group, &nt);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.n_warps = share_limit(info.sm_count, nt);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + L.off_ml);
  a.lse2 = reinterpret_cast<float*>(ws + L.off_lse2);
  a.scores = weights_out ? reinterpret_cast<float*>(ws + L.off_scores) : nullptr;
  a.w_in = weights_in;
  a.w_out = weights_out;
  a.w_stride = weight_slots;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D == 128)
    return nt == 1 ? launch_attend<128, 1>(a, st)
                   : launch_attend<128, 2>(a, st);
  return nt == 1 ? launch_attend<64, 1>(a, st)
                 : launch_attend<64, 2>(a, st);
}

}  // extern "C"
