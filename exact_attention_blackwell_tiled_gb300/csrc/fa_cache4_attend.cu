// fa_cache4_attend.cu -- one query token per sequence attends to its 4-bit cache
// (cache4.cuh), with the keys' softmax weights added to a running sum on request.
//
//   s_j = scale q . k_j,  k_j = m_j + c_j z_j  per group of 32 elements (minimum m,
//   scale c, codes z), so  q . k_j = sum_g c_jg (q_g . z_jg) + m_jg sum(q_g):
// the codes, small integers, go to the matrix instruction exactly, as does the
// bf16 query, and the scales are applied to its fp32 result.  A 4-bit code masked
// out of its word in place is already a bf16 number: z in bits 0..3 of a half is
// z 2^-133 and in bits 4..7 16 z 2^-133 (subnormal, or of the smallest exponent,
// where bf16 is linear), which the matrix unit multiplies exactly.  So two codes
// cost one mask, and every other pair a shift; 2^64 times the query (2^60 where
// the code has the factor 16), and exponentials 2^64 times too large, bring the
// products back into fp32's normal range.  The second sum, over the minima, is one
// more small product: a lane's stored parameter word is its A fragment as it
// stands, and sum(q_g), split into three bf16 parts (24 bits), the B fragment, made
// once per row.  For the values
//   O = sum_j p_j (m_j + 8 c_j) + sum_j (p_j c_j) (z_j - 8)
// the first sum stays in fp32 and p_j c_j is rounded to bf16 for the second, the
// only rounding before O's own.  (z - 8, not z: the rounding then counts for the
// value's distance from the middle of its group only.)
//
// A key and its value are 5/4 D bytes of codes and parameters, read once for all
// query heads of the kv head (up to 8 NT of them, the columns of the products), and
// cost about 24 warp instructions to unpack, multiply and weigh at D = 128.
// Measured with 64 sequences of 512 to 8192 tokens, 32 query and 8 kv heads of 128
// (265 MB): 60 us, 4.4 TB/s, the SMs issuing in 57% of the cycles; the copies alone
// take 50 us.  So memory and issue bound it together: with 12 warps per SM (registers)
// a warp's chains of dependent steps are not wholly covered by the others.  Storing
// the scores for the weights adds 7 us, the second kernel 5 to 9 (17 with weights,
// cold).
//
// Every warp works by itself: the 16-slot blocks of all (sequence, kv head) rows
// lie in one list, and each warp takes an equal contiguous share of it, streams it
// through a ring of its own in shared memory (bulk copies that its lane 0 issues,
// an mbarrier per stage) and keeps maximum, sum and O of the row at hand in
// registers.  So sequences of any lengths load the SMs evenly with no barrier
// between warps.  A row that lies inside one share is finished there; a row cut
// by shares leaves parts (fp32 O, maximum, sum), at most two per warp, and the
// numbers of its first and last share, by which a second kernel finds and joins them
// (finding them from the lengths again took 8 us more); it also writes the rows of
// empty sequences and, when weights are asked for, turns the stored scores into them,
// now that the sums are known.
// Short caches in few rows, where that second launch is most of the time, take a
// block per row instead and join in shared memory.
//
// Under a window with sinks (kWin) a row's list is the sinks' blocks and the window's; the
// others are neither read nor counted, and their running weights only copied.  64 sequences of
// 512 to 16,384 tokens, a window of 4,096, 4 sinks, with weights (236 MB): 66 us and 15 to
// 20 for the second kernel, 80 together; one sequence of 5,000 tokens, a window of 512: 6.3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "cache4.cuh"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kWarps = 4;      // per block; they share nothing but the launch
// One block per row (kOwn): caches of up to 64 blocks of 16 slots, so that a warp has
// at most 8, and at most two rows per SM, eight where two blocks of it fit an SM
// (D = 64, 8 columns).  Measured, us of a step without / with weights, one block per
// row against shares, 32 query and 8 kv heads:
//   D = 128, 1 x 300 tokens 5.1 / 6.6 against 10.0 / 10.6;  38 x 300 (two rows per
//   SM): 10.5 / 13.8 against 13.7 / 16.0;  38 x 1000: 16.5 / 22.7 against 18.3 / 22.1;
//   64 x 300: 19.5 / 25.3 against 17.5 / 19.1;
//   D = 64, 38 x 300: 5.1 / 6.8 against 11.7 / 13.8;  152 x 300 (eight rows per SM):
//   18.3 / 25.0 against 20.1 / 23.4;  152 x 1000: 34.7 / 47.4 against 35.8 / 43.4;
//   228 x 300: 27.4 / 37.7 against 29.1 / 34.2;  400 x 300: 49.0 / 65.7 against 42.1 / 51.7.
// The rule goes by the step without weights: with them it loses 2 to 9% at the most
// rows it takes.  It sees the table's width, not the lengths (which are on the device):
// short caches in a table of more than 1024 slots take shares.  Other groups than four
// query heads were not measured.
constexpr int kOwnWarps = 8, kOwnBlocks = 64;
template <int D, int NT>
constexpr int kOwnRowsPerSm = D == 64 && NT == 1 ? 8 : 2;
constexpr int kWeightKeys = 1024;  // keys of a (sequence, kv head) per unit of the weight pass

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
  int* span;        // [B Hkv tiles, 2]: first and last share of a row that is not empty
  float* scores;    // [B, Hkv, cap, group] in log2 units, or null
  float* lse2;      // [B, Hq] log2 of the sums of the rows that no share cut, or unused
  const float* w_in;
  float* w_out;  // [B, Hkv, w_stride]
  int w_stride;
  int wl, sinks;  // the window (kWin): the last wl + 1 tokens and the first `sinks`
};

// Fewest 16-slot blocks worth a warp of its own: with fewer, the parts to join
// cost more than the work split off.
constexpr int kMinBlocks = 4;

// Resident blocks of attend_kernel with shares, by the registers a row takes (D = 64,
// 8 columns: four of 126 registers, 2 x 32768 tokens of 16 heads 27.2 us; three 28.3,
// five of 96 30.4.  D = 128: four, of 128 registers, measured 6% slower than three).
__host__ __device__ constexpr int blocks_per_sm(int D, int nt) {
  return nt == 2 ? 2 : (D == 64 ? 4 : 3);
}

// A warp's ring in shared memory: two stages of 5 KB, so that an SM's 12 warps have
// 60 to 120 KB on their way (the bytes that cover the memory's latency at its full
// rate are about 45 KB); a third stage measured the same or 3% slower.
template <int D>
struct Ring {
  static constexpr int kStages = 2;
  static constexpr int kBlocks = D == 128 ? 2 : 4;  // of a stage
  static constexpr int kBytes = kBlocks * C4<D>::kBytes;
};

__device__ __forceinline__ int seq_len(const AttendArgs& a, int b) {
  const int n = a.lens[b];
  return n < 0 ? 0 : (n < a.cap ? n : a.cap);
}

// The blocks that a sequence's query sees, numbered 0 .. nb - 1: the first `front` ones,
// which hold sinks, and those from block front + gap on.  Without a window: all.
template <bool kWin>
struct View {
  int len, nb;
  int lo, front, gap, sinks;  // (kWin) keys from lo on and below `sinks` are visible
  __device__ __forceinline__ int block(int i) const { return !kWin || i < front ? i : i + gap; }
  __device__ __forceinline__ bool key(int j) const { return j < len && (!kWin || j >= lo || j < sinks); }
  // (kWin) blocks [in0, in1) lie behind one another and all their keys are visible
  __device__ __forceinline__ int in0() const { return front + (lo % kC4Block ? 1 : 0); }
  __device__ __forceinline__ int in1() const { return len / kC4Block - gap; }
};
template <bool kWin>
__device__ __forceinline__ View<kWin> seq_view(const AttendArgs& a, int b) {
  View<kWin> v;
  v.len = seq_len(a, b);
  const int all = (v.len + kC4Block - 1) / kC4Block;
  v.nb = all;
  if constexpr (kWin) {
    v.sinks = a.sinks;
    v.lo = max(0, v.len - 1 - a.wl);
    const int first = v.lo / kC4Block;
    v.front = min((a.sinks + kC4Block - 1) / kC4Block, first);
    v.gap = first - v.front;
    v.nb = all - v.gap;
  }
  return v;
}

template <bool kWin>
__device__ __forceinline__ int seq_blocks(const AttendArgs& a, int b) {
  return seq_view<kWin>(a, b).nb;
}

// Prefix sums of the sequences' blocks by a whole warp: lane l holds sequences
// l * per .. and the blocks before them, so that one round of loads serves both
// the total and the search for a position.
struct List {
  int per;           // sequences per lane
  long long before;  // blocks of the sequences of lower lanes
  long long own;     // blocks of this lane's
  long long total;
};

template <bool kWin>
__device__ __forceinline__ List read_list(const AttendArgs& a) {
  const int lane = threadIdx.x & 31;
  List s;
  s.per = (a.B + 31) >> 5;
  s.own = 0;
  const int b0 = lane * s.per, b1 = min(a.B, b0 + s.per);
#pragma unroll 4
  for (int b = b0; b < b1; ++b) s.own += seq_blocks<kWin>(a, b);
  long long inc = s.own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  s.before = inc - s.own;
  s.total = __shfl_sync(0xffffffffu, inc, 31);
  return s;
}

// The sequence that holds block x of the list (x < total), and its first block.
template <bool kWin>
__device__ __forceinline__ int locate(const AttendArgs& a, const List& s, long long x,
                                      long long* base) {
  const int lane = threadIdx.x & 31;
  const unsigned hit = __ballot_sync(0xffffffffu, x >= s.before && x < s.before + s.own);
  const int l = __ffs(hit) - 1;
  long long at = s.before;
  int b = lane * s.per;
  if (lane == l)
    for (int n; x >= at + (n = seq_blocks<kWin>(a, b)); ++b) at += n;
  *base = __shfl_sync(0xffffffffu, at, l);
  return __shfl_sync(0xffffffffu, b, l);
}

// Shares: warp w of W takes list positions w N / W .. (w + 1) N / W - 1.
__device__ __forceinline__ int share_count(const AttendArgs& a, long long N) {
  const long long most = (N + kMinBlocks - 1) / kMinBlocks;
  return (int)(most < a.n_warps ? most : a.n_warps);
}
__device__ __forceinline__ long long share_begin(long long N, int W, int w) { return w * N / W; }

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

// 4-bit field R (0..3) of the low and of the high half of w as bf16 numbers: times
// 2^-133 for the even fields, 16 * 2^-133 for the odd ones.
template <int R>
__device__ __forceinline__ uint32_t code(uint32_t w) {
  return (R < 2 ? w : w >> 8) & ((R & 1) ? 0x00f000f0u : 0x000f000fu);
}

// ... the field minus 8 (exact).
template <int R>
__device__ __forceinline__ uint32_t minus8(uint32_t w) {
  const uint32_t x = code<R>(w), k = (R & 1) ? 0x00800080u : 0x00080008u;
  const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                   *reinterpret_cast<const __nv_bfloat162*>(&k));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Two bf16 numbers times a power of two.
__device__ __forceinline__ uint32_t times(uint32_t w, float f) {
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(f));
  return *reinterpret_cast<const uint32_t*>(&y);
}

constexpr float kTop = 64.f;         // exponentials are 2^(s - m + kTop)
constexpr float kScoreUp = 0x1p69f;  // products of queries and codes carry 2^(64 - 133)

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

// The codes pass through L2 as lines to be evicted first: they are read once in a
// call, while the scores and parts are read again by the second kernel (77.3 us
// against 74.0 for the 64 sequences above with weights).
__device__ __forceinline__ void copy_block(uint32_t dst, const void* src, uint32_t bytes,
                                           uint32_t bar) {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// ------------------------------------------------------------------ main kernel

// Registers of a row in progress.  Lane 4 i + t holds query columns 2 t and
// 2 t + 1 of every 8-column tile.
template <int D, int NT>
struct RowState {
  static constexpr int kG = D / 32;
  float acc[2 * kG][NT][4];  // O^T: tile 2 g + x, rows i and i + 8 are elements 32 g + 4 i + 2 x, + 1
  // (times 2^-69, 2^-65 for the odd elements)
  float mid[kG][NT][2];      // this lane's sum of p (m + 8 c), times 2^64
  float m[NT][2], l[NT][2];  // maximum (log2 units; the same in the lanes of one t), lane's sum
                             // times 2^64
};

// A row's log-sum-exp from its maximum and sum.
__device__ __forceinline__ void write_lse(const AttendArgs& a, size_t row, float m, float l) {
  const float z = l > 0.f ? m + __log2f(l) : -INFINITY;
  a.lse[row] = z * 0.69314718055994531f;
  if (a.scores) a.lse2[row] = z;
}

// kOwn: short caches and few rows.  A block of 8 warps takes one row, its warps equal
// parts of it, and joins them in shared memory, weights included: one launch.
// Otherwise every warp takes a share of the list.  kWin: a window with sinks; blocks count
// as View numbers them, and only those are looked up and read.
template <int D, int NT, bool kOwn, bool kWin>
__global__ void __launch_bounds__((kOwn ? kOwnWarps : kWarps) * 32, kOwn ? 1 : blocks_per_sm(D, NT))
    attend_kernel(const AttendArgs a) {
  using L = C4<D>;
  using R = Ring<D>;
  constexpr int kG = L::kGroups, kW = kOwn ? kOwnWarps : kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ alignas(8) uint64_t s_bar[kW][R::kStages];
  __shared__ float2 s_ml[kOwn ? kW : 1][8 * NT];  // maximum and sum of a warp's part
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, t = lane & 3;
  const uint8_t* ring = smem + warp * R::kStages * R::kBytes;
  const uint32_t bars = smem_u32(&s_bar[warp][0]);
  if (threadIdx.x == 0) s_abort = 0;
  if (lane < R::kStages) mbar_init(bars + 8 * lane, 1);
  fence_mbarrier_init();
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  // rows (b, kv head, tile) in order: a sequence has rows_per rows of its blocks
  const int rows_per = a.Hkv * a.tiles;
  int row_b, row, blk0, left;  // left: blocks still to do
  View<kWin> view;
  int w = 0;
  if constexpr (kOwn) {
    row_b = blockIdx.x / rows_per;
    row = blockIdx.x - row_b * rows_per;
    view = seq_view<kWin>(a, row_b);
    const int nb = view.nb;
    const int per = (nb + 2 * kW - 1) / (2 * kW) * 2;  // pairs of blocks
    blk0 = min(nb, warp * per);
    left = min(per, nb - blk0);
    if (lane < 8 * NT) s_ml[warp][lane] = make_float2(-INFINITY, 0.f);
    if (row == 0 && threadIdx.x == 0 && a.lens[row_b] != view.len) c4_flag(a.table);
  } else {
    const List list = read_list<kWin>(a);
    const long long N = list.total * rows_per;
    if (N == 0) return;
    const int W = share_count(a, N);
    w = blockIdx.x + warp * gridDim.x;  // neighbouring shares on different SMs
    if (w >= W) return;
    const long long begin = share_begin(N, W, w);
    left = (int)(share_begin(N, W, w + 1) - begin);
    long long base;
    row_b = locate<kWin>(a, list, begin / rows_per, &base);
    view = seq_view<kWin>(a, row_b);
    // where in the sequence's rows the share begins
    row = (int)((begin - base * rows_per) / view.nb);
    blk0 = (int)(begin - base * rows_per - (long long)row * view.nb);
  }

  const float score_up = a.scale_log2 * kScoreUp;
  const int slot_i = i ^ ((i >> 1) & 1);  // slot of product row i; row i + 8 is slot_i + 8
  // this lane's value slots: product rows 2 t and 2 t + 1 (and those + 8)
  const int va = (2 * t) ^ (t & 1), vb = (2 * t + 1) ^ (t & 1);
  int st = 0;          // the stage consumed next, and its barrier's phase
  uint32_t phase = 0;
  while (left > 0) {
    const int nb = view.nb, len = view.len;
    const int blk1 = min(nb, blk0 + left);
    const int hk = row / a.tiles, tile = row - hk * a.tiles;
    // ---- copies: lane x takes block x of a stage; its page is looked up a stage ahead
    const uint8_t* head_base = a.cache + (size_t)hk * a.table.blocks_per_page() * L::kBytes;
    const size_t page_bytes = (size_t)a.Hkv * a.table.blocks_per_page() * L::kBytes;
    int next = blk0 + lane;  // block of the lane's next copy
    auto look_up = [&]() { return lane < R::kBlocks && next < blk1 ? c4_page(a.table, row_b, view.block(next)) : 0; };
    int page = look_up();
    uint32_t bad = 0;  // bit kBlocks * stage + x: that block's page is out of range
    auto fill = [&](int st, int first) {  // blocks first .. of the row into stage st
      if (first >= blk1) return;
      const bool mine = lane < R::kBlocks && next < blk1;
      const uint32_t miss = __ballot_sync(0xffffffffu, mine && page < 0);
      const int count = min(R::kBlocks, blk1 - first) - __popc(miss);
      if (lane == 0) mbar_arrive_expect_tx(bars + 8 * st, count * L::kBytes);
      if (mine && page >= 0)
        copy_block(smem_u32(ring) + st * R::kBytes + lane * L::kBytes,
                   head_base + page * page_bytes +
                       a.table.in_page(view.block(next)) * L::kBytes,
                   L::kBytes, bars + 8 * st);
      bad = (bad & ~(((1u << R::kBlocks) - 1) << (st * R::kBlocks))) | (miss << (st * R::kBlocks));
      if (miss && lane == 0) c4_flag(a.table);
      next += R::kBlocks;
      page = look_up();
    };
#pragma unroll
    for (int f = 0; f < R::kStages; ++f)
      fill(st + f < R::kStages ? st + f : st + f - R::kStages, blk0 + f * R::kBlocks);
    // ---- a row: its queries
    const int heads = min(8 * NT, a.group - tile * 8 * NT);  // real query columns
    uint32_t qf[kG][NT][4];  // B fragments: steps 2 g (0, 1) and 2 g + 1 (2, 3)
    uint32_t qp[NT][3];      // B fragments of the parameter product
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = nt * 8 + i;
      const __nv_bfloat16* src =
          a.q + row_b * a.q_batch + (long long)(hk * a.group + tile * 8 * NT + col) * a.q_head + 8 * t;
      float sum_t = 0.f;  // of this lane's group in the parameter product
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (col < heads) x = *reinterpret_cast<const uint4*>(src + 32 * g);
        // elements 0..7 in pairs x.x = (0,1) .. x.w = (6,7)
        qf[g][nt][0] = times(__byte_perm(x.x, x.z, 0x5410), 0x1p64f);  // (0, 4): fields 0
        qf[g][nt][1] = times(__byte_perm(x.x, x.z, 0x7632), 0x1p60f);  // (1, 5): fields 1
        qf[g][nt][2] = times(__byte_perm(x.y, x.w, 0x5410), 0x1p64f);  // (2, 6): fields 2
        qf[g][nt][3] = times(__byte_perm(x.y, x.w, 0x7632), 0x1p60f);  // (3, 7): fields 3
        float sum = 0.f;
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum += __uint_as_float(xs[e] << 16) + __uint_as_float(xs[e] & 0xffff0000u);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (g == (t & (kG - 1))) sum_t = sum;
      }
      __nv_bfloat16 part[3];
      split3(sum_t * (1.f / kScoreUp), part);
      // k index 2 t is the scale (times zero), 2 t + 1 the minimum, of group t
      // (D = 128), with parts 0 and 1, then 2; at D = 64 lanes t >= 2 take part 2 of
      // group t - 2
      const __nv_bfloat16 zero = __ushort_as_bfloat16(0);
      qp[nt][0] = pair16(zero, D == 128 || t < 2 ? part[0] : part[2]);
      qp[nt][1] = pair16(zero, D == 128 || t < 2 ? part[1] : zero);
      qp[nt][2] = pair16(zero, part[2]);
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
      score = a.scores +
              (((size_t)row_b * a.Hkv + hk) * a.cap + (kWin ? 0 : blk0) * kC4Block + slot_i) * a.group +
              tile * 8 * NT + 2 * t;
    const int in0 = kWin ? view.in0() : 0, in1 = kWin ? min(view.in1(), blk1) : 0;
    // ---- its blocks, two at a time: their chains of dependent steps interleave
#pragma unroll 1
    for (int at = blk0; at < blk1; at += 2) {
      const int x = (at - blk0) & (R::kBlocks - 1);
      if (x == 0) {
        const bool ok = mbar_wait(bars + 8 * st, phase, &s_abort);
        if (!__all_sync(0xffffffffu, ok)) {
          // give up, once the copies under way have landed (or that wait runs out too)
          if (lane == 0) {
            atomicExch(a.table.status, (int)FA_ERR_TIMEOUT);
            for (int f = 0; f < R::kStages && at + f * R::kBlocks < blk1; ++f) {
              const int y = st + f < R::kStages ? st + f : st + f - R::kStages;
              const uint64_t t0 = global_timer_ns();
              while (!mbar_try_wait(bars + 8 * y, phase ^ (y < st ? 1u : 0u)))
                if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
            }
          }
          __syncwarp();
          if constexpr (!kOwn) return;
          left = 0;  // (the other warps of the block are not left waiting)
          break;
        }
      }
      // the second block may lie behind the row's last: what its place in the ring
      // holds then counts for nothing, like a slot behind the last key
      const uint8_t* blk = ring + st * R::kBytes + x * L::kBytes;
      // scores of 2 x 16 keys: [0, 1] row i, [2, 3] row i + 8
      float sc[2][NT][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t k0[kG], k1[kG], p0[kG], p1[kG];
        const uint8_t* kb = blk + y * L::kBytes;
        const uint8_t* par = kb + L::kOffKPar + slot_i * L::kPar;
        lds(k0, kb + slot_i * L::kRow + t * 4 * kG);
        lds(k1, kb + (slot_i + 8) * L::kRow + t * 4 * kG);
        lds(p0, par);
        lds(p1, par + 8 * L::kPar);
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(par + (t & (kG - 1)) * 4);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(par + 8 * L::kPar + (t & (kG - 1)) * 4);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816_first(sc[y][nt], w0, w1, w0, w1, qp[nt][0], qp[nt][1]);
          if constexpr (D == 128) mma1688(sc[y][nt], w0, w1, qp[nt][2]);
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const uint32_t a00 = code<0>(k0[g]), a01 = code<1>(k0[g]),
                         a02 = code<2>(k0[g]), a03 = code<3>(k0[g]);
          const uint32_t a10 = code<0>(k1[g]), a11 = code<1>(k1[g]),
                         a12 = code<2>(k1[g]), a13 = code<3>(k1[g]);
          const float c0 = c4_scale(p0[g]), c1 = c4_scale(p1[g]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4];
            mma16816_first(d, a00, a10, a01, a11, qf[g][nt][0], qf[g][nt][1]);
            mma16816(d, a02, a12, a03, a13, qf[g][nt][2], qf[g][nt][3]);
            sc[y][nt][0] = fmaf(c0, d[0], sc[y][nt][0]);
            sc[y][nt][1] = fmaf(c0, d[1], sc[y][nt][1]);
            sc[y][nt][2] = fmaf(c1, d[2], sc[y][nt][2]);
            sc[y][nt][3] = fmaf(c1, d[3], sc[y][nt][3]);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[y][nt][e] *= score_up;
      // slots behind the last key, and blocks whose page is out of range
      const uint32_t miss = (bad >> (st * R::kBlocks + x)) & 3u;
      const int ends = min(len, blk1 * kC4Block) - at * kC4Block;  // the share's keys from here on
      const bool full = miss == 0 && (kWin ? at >= in0 && at + 2 <= in1 : ends >= 2 * kC4Block);
      bool live[2][2] = {{true, true}, {true, true}};
      if constexpr (kWin) {
        if (!full) {
          asm volatile("" ::: "memory");  // a branch
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z)
              live[y][z] = !((miss >> y) & 1) && at + y < blk1 &&
                           view.key(view.block(at + y) * kC4Block + slot_i + 8 * z);
        }
      } else {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z)
            live[y][z] = !((miss >> y) & 1) && y * kC4Block + slot_i + 8 * z < ends;
      }
      if (!full) {
        asm volatile("" ::: "memory");  // a branch, not selects in every iteration
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[y][nt][e] = live[y][e >> 1] ? sc[y][nt][e] : -INFINITY;
      }
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // a stale maximum stands until a score passes it by 8 (weights up to 2^8)
        grow |= fmaxf(fmaxf(sc[0][nt][0], sc[0][nt][2]), fmaxf(sc[1][nt][0], sc[1][nt][2])) >
                r.m[nt][0] + 8.f;
        grow |= fmaxf(fmaxf(sc[0][nt][1], sc[0][nt][3]), fmaxf(sc[1][nt][1], sc[1][nt][3])) >
                r.m[nt][1] + 8.f;
      }
      if (a.scores) {
        const int mine = ends - slot_i;  // keys of the share from row i on
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if constexpr (kWin) {
              // keys out of sight have no score, in these blocks and in others
              if (!full && !(at + y < blk1 && view.key(view.block(at + y) * kC4Block + slot_i + 8 * z))) continue;
            } else {
              if (mine <= y * kC4Block + 8 * z) continue;
            }
            float* dst = score + (kWin ? (size_t)view.block(at + y) * kC4Block + 8 * z
                                       : (size_t)(y * kC4Block + 8 * z)) * a.group;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int col = nt * 8 + 2 * t;
              if ((a.group & 1) == 0) {
                if (col < heads)
                  *reinterpret_cast<float2*>(dst + nt * 8) =
                      make_float2(sc[y][nt][2 * z], sc[y][nt][2 * z + 1]);
              } else {
                if (col < heads) dst[nt * 8] = sc[y][nt][2 * z];
                if (col + 1 < heads) dst[nt * 8 + 1] = sc[y][nt][2 * z + 1];
              }
            }
          }
        if (!kWin) score += 2 * kC4Block * a.group;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(fmaxf(sc[0][nt][c], sc[0][nt][2 + c]), fmaxf(sc[1][nt][c], sc[1][nt][2 + c]));
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
        const float n0 = r.m[nt][0] == -INFINITY ? 0.f : r.m[nt][0] - kTop;
        const float n1 = r.m[nt][1] == -INFINITY ? 0.f : r.m[nt][1] - kTop;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          sc[y][nt][0] = ex2_mufu(sc[y][nt][0] - n0);
          sc[y][nt][1] = ex2_mufu(sc[y][nt][1] - n1);
          sc[y][nt][2] = ex2_mufu(sc[y][nt][2] - n0);
          sc[y][nt][3] = ex2_mufu(sc[y][nt][3] - n1);
          r.l[nt][0] += sc[y][nt][0] + sc[y][nt][2];
          r.l[nt][1] += sc[y][nt][1] + sc[y][nt][3];
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint8_t* vb_ = blk + y * L::kBytes;
        uint32_t v[4][(kG + 1) / 2], p0[kG], p1[kG];
        lds(v[0], vb_ + L::v_half(va, i, 0));
        lds(v[1], vb_ + L::v_half(vb, i, 0));
        lds(v[2], vb_ + L::v_half(va + 8, i, 0));
        lds(v[3], vb_ + L::v_half(vb + 8, i, 0));
        lds(p0, vb_ + L::kOffVPar + slot_i * L::kPar);
        lds(p1, vb_ + L::kOffVPar + (slot_i + 8) * L::kPar);
        if (!full) {
          // a slot without a key holds anything: its parameters count as zero
          asm volatile("" ::: "memory");
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            p0[g] = live[y][0] ? p0[g] : 0u;
            p1[g] = live[y][1] ? p1[g] : 0u;
          }
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const float c0 = c4_scale(p0[g]), m0 = fmaf(8.f, c0, c4_min(p0[g]));
          const float c1 = c4_scale(p1[g]), m1 = fmaf(8.f, c1, c4_min(p1[g]));
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float(&p)[4] = sc[y][nt];
            r.mid[g][nt][0] = fmaf(p[0], m0, fmaf(p[2], m1, r.mid[g][nt][0]));
            r.mid[g][nt][1] = fmaf(p[1], m0, fmaf(p[3], m1, r.mid[g][nt][1]));
            b0[nt] = transpose8x8(pack_bf16x2(p[0] * c0, p[1] * c0));
            b1[nt] = transpose8x8(pack_bf16x2(p[2] * c1, p[3] * c1));
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
      }
      if (x == R::kBlocks - 2 || at + 2 >= blk1) {
        __syncwarp();  // every lane has read the stage that is filled again
        fill(st, at - x + R::kStages * R::kBlocks);
        if (++st == R::kStages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
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
    const bool whole = !kOwn && blk0 == 0 && blk1 == nb;
    if (!kOwn && lane == 0) {
      int* span = a.span + 2 * ((size_t)row_b * rows_per + row);
      if (blk0 == 0) span[0] = w;
      if (blk1 == nb) span[1] = w;
    }
    const size_t part = ((size_t)w * 2 + (blk0 == 0 ? 1 : 0)) * (8 * NT);
    float* mine = kOwn ? reinterpret_cast<float*>(smem + warp * R::kStages * R::kBytes)
                       : a.part_o + part * D;  // the warp's own ring, which it has read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = nt * 8 + 2 * t + c;
        if (col >= heads) continue;
        const float l = r.l[nt][c] * 0x1p-64f, m = r.m[nt][c];
        const float inv = whole ? (l > 0.f ? 1.0f / l : 0.f) : 1.f;
        const size_t out = (size_t)row_b * a.Hq + hk * a.group + tile * 8 * NT + col;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const float mid = r.mid[g][nt][c] * 0x1p-64f;
          const float x0 = fmaf(r.acc[2 * g][nt][c], 0x1p69f, mid) * inv;
          const float x1 = fmaf(r.acc[2 * g][nt][2 + c], 0x1p65f, mid) * inv;
          const float x2 = fmaf(r.acc[2 * g + 1][nt][c], 0x1p69f, mid) * inv;
          const float x3 = fmaf(r.acc[2 * g + 1][nt][2 + c], 0x1p65f, mid) * inv;
          if (whole)
            *reinterpret_cast<uint2*>(a.o + out * D + 32 * g + 4 * i) =
                make_uint2(pack_bf16x2(x0, x1), pack_bf16x2(x2, x3));
          else
            *reinterpret_cast<float4*>(mine + col * D + 32 * g + 4 * i) = make_float4(x0, x1, x2, x3);
        }
        if (i == 0) {
          if (whole)
            write_lse(a, out, m, l);
          else if (kOwn)
            s_ml[warp][col] = make_float2(m, l);
          else
            a.part_ml[part + col] = make_float2(m, l);
        }
      }
    // ---- on to the next row of the share
    if (kOwn) break;
    left -= blk1 - blk0;
    blk0 = 0;
    if (left > 0 && ++row == rows_per) {
      row = 0;
      do {
        view = seq_view<kWin>(a, ++row_b);  // the share ends inside the list
      } while (view.len == 0);
    }
  }
  if constexpr (kOwn) {
    // ---- the row from its warps' parts (a warp without blocks has sum 0)
    __syncthreads();
    const int hk = row / a.tiles, tile = row - hk * a.tiles;
    const int heads = min(8 * NT, a.group - tile * 8 * NT);
    const size_t out0 = (size_t)row_b * a.Hq + hk * a.group + tile * 8 * NT;
    for (int x = threadIdx.x; x < heads * (D / 4); x += kW * 32) {
      const int col = x / (D / 4), d = (x - col * (D / 4)) * 4;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int y = 0; y < kW; ++y) m = fmaxf(m, s_ml[y][col].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < kW; ++y) {
        const float2 ml = s_ml[y][col];
        if (!(ml.y > 0.f)) continue;
        const float f = ex2_mufu(ml.x - m);
        const float4 v = *reinterpret_cast<const float4*>(smem + y * R::kStages * R::kBytes +
                                                          (col * D + d) * 4);
        l = fmaf(f, ml.y, l);
        o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
      }
      const float inv = l > 0.f ? 1.0f / l : 0.f;
      *reinterpret_cast<uint2*>(a.o + (out0 + col) * D + d) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (d == 0) write_lse(a, out0 + col, m, l);
    }
    if (a.scores) {
      // the weights of the row's keys: the scores and sums are the block's own
      __syncthreads();
      const size_t bh = (size_t)row_b * a.Hkv + hk;
      for (int j = threadIdx.x; j < view.len; j += kW * 32) {
        const float* src = a.scores + (bh * a.cap + j) * a.group;
        float sum = 0.f;
        const int heads_seen = view.key(j) ? a.group : 0;
        for (int h = 0; h < heads_seen; ++h) {
          const float z = a.lse2[out0 + h];
          sum += z == -INFINITY ? 0.f : ex2_mufu(src[h] - z);
        }
        const size_t at = bh * a.w_stride + j;
        a.w_out[at] = a.w_in ? a.w_in[at] + sum : sum;
      }
    }
  }
}

// ------------------------------------------------------------------ join and weights

// The shares that hold a row's blocks; w0 == w1: the row was finished by that one.
struct RowSpan {
  int w0, w1;
};

__device__ __forceinline__ RowSpan row_span(const AttendArgs& a, int b, int row) {
  const int2 s = *reinterpret_cast<const int2*>(a.span + 2 * ((size_t)b * a.Hkv * a.tiles + row));
  // (a share that gave up wrote nothing)
  const int w0 = min(max(s.x, 0), a.n_warps - 1);
  return {w0, min(max(s.y, w0), a.n_warps - 1)};
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

// w_out = w_in + sum over the group of 2^(score - log2 sum), for kWeightKeys keys of
// a (sequence, kv head).  The scores are on their way while the sums of rows that
// shares cut are joined, a warp per query head.  Keys out of sight (kWin) have no score and
// add nothing.
template <int NT, int kW, bool kWin>
__device__ __forceinline__ void weigh(const AttendArgs& a, int unit, float* s_lse2) {
  constexpr int kPer = kWeightKeys / (kW * 32);
  const int units = (a.cap + kWeightKeys - 1) / kWeightKeys;
  const int bh = unit / units, first = (unit - bh * units) * kWeightKeys;
  const int b = bh / a.Hkv, hk = bh - b * a.Hkv, j0 = first + threadIdx.x;
  const View<kWin> view = seq_view<kWin>(a, b);
  const int len = view.len;
  if (first >= len) return;
  if (kWin && first >= view.sinks && first + kWeightKeys <= view.lo) {
    // out of sight as a whole: nothing to add
    if (a.w_in == a.w_out) return;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {  // (its keys are below lo, and so below len)
      const size_t at = (size_t)bh * a.w_stride + j0 + x * kW * 32;
      a.w_out[at] = a.w_in ? a.w_in[at] : 0.f;
    }
    return;
  }
  const float* src = a.scores + ((size_t)bh * a.cap + j0) * a.group;
  const size_t step = (size_t)kW * 32 * a.group, at = (size_t)bh * a.w_stride + j0;
  const bool four = (a.group & 3) == 0;
  float4 s[kPer];  // the first four (or one) of each key
  float w[kPer];
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    s[x] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    w[x] = 0.f;
    if (j0 + x * kW * 32 >= len) continue;
    if (a.w_in) w[x] = a.w_in[at + x * kW * 32];
    if (kWin && !view.key(j0 + x * kW * 32)) continue;
    if (four) s[x] = *reinterpret_cast<const float4*>(src + x * step);
    else s[x].x = src[x * step];
  }
  for (int h = threadIdx.x >> 5; h < a.group; h += kW) {
    const int tile = h / (8 * NT), col = h - tile * 8 * NT;
    const RowSpan sp = row_span(a, b, hk * a.tiles + tile);
    float z;
    if (sp.w0 == sp.w1) {
      z = a.lse2[(size_t)b * a.Hq + hk * a.group + h];
    } else {
      const float2 ml = join_ml<NT>(a, sp, col);
      z = ml.y > 0.f ? ml.x + __log2f(ml.y) : -INFINITY;
    }
    if ((threadIdx.x & 31) == 0) s_lse2[h] = z;
  }
  __syncthreads();
  const bool empty = s_lse2[0] == -INFINITY;  // every page out of range
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    if (j0 + x * kW * 32 >= len) break;
    float sum = 0.f;
    if (kWin && !view.key(j0 + x * kW * 32)) {
      // (nothing)
    } else if (four) {
      float4 y = s[x];
      for (int h = 0;;) {
        sum += (ex2_mufu(y.x - s_lse2[h]) + ex2_mufu(y.y - s_lse2[h + 1])) +
               (ex2_mufu(y.z - s_lse2[h + 2]) + ex2_mufu(y.w - s_lse2[h + 3]));
        if ((h += 4) >= a.group) break;
        y = *reinterpret_cast<const float4*>(src + x * step + h);
      }
    } else {
      sum = ex2_mufu(s[x].x - s_lse2[0]);
      for (int h = 1; h < a.group; ++h) sum += ex2_mufu(src[x * step + h] - s_lse2[h]);
    }
    a.w_out[at + x * kW * 32] = w[x] + (empty ? 0.f : sum);
  }
}

// The first blocks: a unit of weights each, where weights are asked for.  The others:
// one (sequence, query head) each, whose row was cut by shares or is empty.  kW
// warps: four where there are rows enough to fill the GPU, eight where few rows were
// cut into many parts; with weights or without, so that O has the same bits.  A block
// is a chain of dependent loads, so what counts is how many are resident: 32 warps
// per SM with 64 registers a thread, for 20 with 95 (1 us less).
template <int D, int NT, int kW, bool kWin>
__global__ void __launch_bounds__(kW * 32, 32 / kW) join_kernel(const AttendArgs a, int units) {
  constexpr int kV = D / 32;
  __shared__ float s_o[kW][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if ((int)blockIdx.x < units) {
    __shared__ float s_lse2[128];
    weigh<NT, kW, kWin>(a, blockIdx.x, s_lse2);
    return;
  }
  const int out = blockIdx.x - units;  // (sequence, query head)
  const int b = out / a.Hq, hq = out - b * a.Hq;
  const int hk = hq / a.group, in_group = hq - hk * a.group;
  const int tile = in_group / (8 * NT), col = in_group - tile * 8 * NT;
  const int len = seq_len(a, b);
  const RowSpan s = row_span(a, b, hk * a.tiles + tile);
  if (hq == 0 && threadIdx.x == 0 && a.lens[b] != len) c4_flag(a.table);
  __nv_bfloat16* o = a.o + (size_t)out * D;
  if (len == 0) {  // an empty sequence
    for (int x = threadIdx.x; x < D / 2; x += kW * 32) reinterpret_cast<uint32_t*>(o)[x] = 0u;
    if (threadIdx.x == 0) a.lse[out] = -INFINITY;
    return;
  }
  if (s.w0 == s.w1) return;
  const float2 ml = join_ml<NT>(a, s, col);
  float acc[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) acc[e] = 0.f;
#pragma unroll 8
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
  if (threadIdx.x < D / 2) {  // at most 64 threads
    const float inv = ml.y > 0.f ? 1.0f / ml.y : 0.f;
    float x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int y = 0; y < kW; ++y) {
      x0 += s_o[y][2 * threadIdx.x];
      x1 += s_o[y][2 * threadIdx.x + 1];
    }
    reinterpret_cast<uint32_t*>(o)[threadIdx.x] = pack_bf16x2(x0 * inv, x1 * inv);
  }
  if (threadIdx.x == 0)
    a.lse[out] = ml.y > 0.f ? (ml.x + __log2f(ml.y)) * 0.69314718055994531f : -INFINITY;
}

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Query heads of a kv head: one 8-column tile, or two at a time.
int tile_count(int group, int* nt) {
  *nt = group <= 8 ? 1 : 2;
  return (group + 8 * *nt - 1) / (8 * *nt);
}

// Shares: every warp that is resident at once.
int share_limit(int sms, int D, int nt) { return sms * blocks_per_sm(D, nt) * kWarps; }

struct AttendLayout {
  size_t off_ml, off_span, off_lse2, off_scores, total;
};

AttendLayout attend_layout(int B, int Hq, int Hkv, int D, int cap, int sms) {
  int nt;
  const int tiles = tile_count(Hq / Hkv, &nt);
  const size_t rows = (size_t)share_limit(sms, D, nt) * 2 * 8 * nt;
  AttendLayout L;
  L.off_ml = rows * D * sizeof(float);
  L.off_span = L.off_ml + rows * sizeof(float2);
  L.off_lse2 = (L.off_span + (size_t)B * Hkv * tiles * 2 * sizeof(int) + 255) & ~(size_t)255;
  L.off_scores = (L.off_lse2 + (cap > 0 ? (size_t)B * Hq * sizeof(float) : 0) + 255) & ~(size_t)255;
  L.total = L.off_scores + (size_t)B * Hq * cap * sizeof(float);
  return L;
}

// slots: those that a sequence's query can see, by the table and the window
template <int D, int NT, bool kWin>
int launch_attend(const AttendArgs& a, int slots, int sms, cudaStream_t stream) {
  constexpr int kSmem = kWarps * Ring<D>::kStages * Ring<D>::kBytes;
  constexpr int kOwnSmem = kOwnWarps * Ring<D>::kStages * Ring<D>::kBytes;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  static bool attr_done[64] = {};
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(attend_kernel<D, NT, false, kWin>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(attend_kernel<D, NT, true, kWin>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kOwnSmem) != cudaSuccess)
      return FA_ERR_CUDA;
    attr_done[dev] = true;
  }
  // One launch with a block per row, by the table's slots: the lengths are on the device
  const long long own_rows = (long long)a.B * a.Hkv;
  if (slots <= kOwnBlocks * kC4Block && a.tiles == 1 &&
      own_rows <= (long long)kOwnRowsPerSm<D, NT> * sms) {
    record_timing(false, stream);
    if (launch_pdl(attend_kernel<D, NT, true, kWin>, dim3((unsigned)own_rows), dim3(kOwnWarps * 32),
                   kOwnSmem, stream, a) != cudaSuccess)
      return FA_ERR_CUDA;
    record_timing(true, stream);
    note_launches(1);
    return FA_OK;
  }
  record_timing(false, stream);
  if (launch_pdl(attend_kernel<D, NT, false, kWin>, dim3(a.n_warps / kWarps), dim3(kWarps * 32), kSmem,
                 stream, a) != cudaSuccess)
    return FA_ERR_CUDA;
  record_timing(true, stream);
  const int rows = a.B * a.Hq;
  const int units = a.scores ? a.B * a.Hkv * ((a.cap + kWeightKeys - 1) / kWeightKeys) : 0;
  const int warps = rows >= 1024 ? 4 : 8;
  const auto join = warps == 4 ? join_kernel<D, NT, 4, kWin> : join_kernel<D, NT, 8, kWin>;
  if (launch_pdl(join, dim3((unsigned)units + (unsigned)rows), dim3(warps * 32), 0, stream, a, units) != cudaSuccess)
    return FA_ERR_CUDA;
  note_launches(2);
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
  return fa_cache4_attend_sink(q, q_batch_stride, q_head_stride, cache, num_pages, page_size, o, lse, B,
                               Hq, Hkv, D, cache_lens, page_table, table_width, -1, 0, scale, weights_in,
                               weights_out, weight_slots, workspace, workspace_bytes, stream);
}

int fa_cache4_attend_sink(const void* q, int64_t q_batch_stride, int64_t q_head_stride,
                          const void* cache, int num_pages, int page_size, void* o, float* lse, int B,
                          int Hq, int Hkv, int D, const int* cache_lens, const int* page_table,
                          int table_width, int window_left, int sinks, float scale,
                          const float* weights_in, float* weights_out, int weight_slots,
                          void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  reset_launches();
  int rc = check_cache4(num_pages, Hkv, D, page_size, B, table_width);
  if (rc) return rc;
  if (Hq < 1 || Hq % Hkv != 0 || !std::isfinite(scale) || sinks < 0) return FA_ERR_INVALID_ARG;
  if (Hq / Hkv > 128) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Hq > (1LL << 30)) return FA_ERR_INVALID_ARG;
  if (weights_out && (long long)B * Hkv * (weight_slots / kWeightKeys + 1) > (1LL << 30))
    return FA_ERR_INVALID_ARG;
  const int slots = table_width * page_size;
  // the list of blocks over all rows, and a warp's share of it, are counted in 64 and
  // 32 bits
  if ((long long)B * Hq * (slots / kC4Block + 1LL) >= (1LL << 40)) return FA_ERR_INVALID_ARG;
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
  a.table = C4Table{page_table, table_width, num_pages, c4_shift(page_size), status};
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.tiles = tile_count(a.group, &nt);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.n_warps = share_limit(info.sm_count, D, nt);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + L.off_ml);
  a.span = reinterpret_cast<int*>(ws + L.off_span);
  a.lse2 = reinterpret_cast<float*>(ws + L.off_lse2);
  a.scores = weights_out ? reinterpret_cast<float*>(ws + L.off_scores) : nullptr;
  a.w_in = weights_in;
  a.w_out = weights_out;
  a.w_stride = weight_slots;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // a window that hides a key of some length the table allows
  if (window_left >= 0 && window_left < slots - 1 && sinks < slots - 1 - window_left) {
    a.wl = window_left;
    a.sinks = sinks;
    // wl + 1 keys lie in at most (wl + 15) / 16 + 1 blocks
    const long long seen =
        ((sinks + kC4Block - 1LL) / kC4Block + (window_left + kC4Block - 1LL) / kC4Block + 1) * kC4Block;
    const int most = (int)(seen < slots ? seen : slots);
    if (D == 128)
      return nt == 1 ? launch_attend<128, 1, true>(a, most, info.sm_count, st)
                     : launch_attend<128, 2, true>(a, most, info.sm_count, st);
    return nt == 1 ? launch_attend<64, 1, true>(a, most, info.sm_count, st)
                   : launch_attend<64, 2, true>(a, most, info.sm_count, st);
  }
  if (D == 128)
    return nt == 1 ? launch_attend<128, 1, false>(a, slots, info.sm_count, st)
                   : launch_attend<128, 2, false>(a, slots, info.sm_count, st);
  return nt == 1 ? launch_attend<64, 1, false>(a, slots, info.sm_count, st)
                 : launch_attend<64, 2, false>(a, slots, info.sm_count, st);
}

}  // extern "C"
