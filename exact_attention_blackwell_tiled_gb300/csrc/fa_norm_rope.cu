// fa_norm_rope.cu -- RMS norms of every query and key head and the rotation of both by
// position, in one pass, and its backward pass.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps),  n_d = x_d r w_d,
//   pairs (a, b) of the first `rot` elements at position p, angle index i:
//     y_a = n_a cos_pi - n_b sin_pi,  y_b = n_b cos_pi + n_a sin_pi,  else y_d = n_d
//   backward, g the rotation of dy by the negative angle, h = g w:
//     dw_d = sum over rows g_d x_d r,   dx = r (h - x r^2 mean_d(h x))
// in fp32 throughout; y and dx are rounded once, to bf16.
//
// Memory bounds it: 4 D bytes per head forward, 6 D backward, against some 12 and 30
// operations an element.  A lane holds 16 elements of a row, so that a pair's two lie in
// one lane: halves paired (a, a + rot / 2): 8 elements of each half, two 16-byte pieces;
// neighbours paired: 16 in a row.  A row is then D / 16 lanes, and a warp's step 4 or 8 rows:
// heads of one token.  A warp walks whole tokens, so that their angles are loaded, and
// multiplied by the weights, once for all their heads (once a step: 73 us instead of 64 for
// the prompt below); where tokens are few their steps are dealt to several warps.  The
// grid stays, and each warp keeps the rows of its next 8 (backward 4) steps on their way to
// shared memory, 64 KB a block, 128 KB an SM.  dw: sums per lane over all rows that it meets, then over
// the lanes and warps of a block in shared memory; a second kernel adds the blocks', always
// in the same order.
//
// Measured, 40 heads of 128 (32 of q, 8 of k): 16,384 tokens, 344 MB: 62 us, 5.6 TB/s, issue
// slots 48% full.  32 heads of 128, 16,384 tokens: forward 43 us (6.2 TB/s), backward 68 (5.9)
// and 4 to 6 for the sums.  64 tokens of 40 heads: 2.6 us, a launch and a chain of latencies.
// Slower: a block per unit of 8 heads (86 us for the first), its rows ahead in registers
// (73), angles in the ring as well (80), 8 elements a lane (70).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kBlocks = 2;                // per SM
constexpr int kDepth = 8, kGradDepth = 4;  // steps whose rows are on their way, of a warp

struct Rows {
  const __nv_bfloat16* x;
  long long token, head;  // elements apart
};
struct RowsOut {
  __nv_bfloat16* x;
  long long token, head;
};

// How the rows are dealt to warps: a unit is a token's steps of kRows heads, q's before k's, or
// one of `split` parts of them.
struct Plan {
  int steps[2], split, per;  // steps of q and of k; parts of a token, their steps
  uint32_t units;            // below 2^31
};

struct NormRopeArgs {
  Plan plan;
  Rows in[2], dy[2];  // q, k; the gradients of the results
  RowsOut out[2];     // the results, or the inputs' gradients
  const void* w[2];
  int w_bf16;
  const float *cos, *sin;  // [P, rot / 2]
  const int* pos;          // [T]
  int T, H[2], P, rot;
  int zero;  // rows of no sequence get zeros
  float eps;
  int* status;
  float* part;   // [blocks, D] sums of dw, the first blocks_q of them q's
  float* dw[2];  // [D]
  int blocks, blocks_q;
};

// Eight bf16 numbers as pairs of fp32.
__device__ __forceinline__ void widen(const uint4& x, float2 (&f)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
}
__device__ __forceinline__ uint4 narrow(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                    pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ void load8(const float* p, float2 (&f)[4]) {
  const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
  f[0] = make_float2(x.x, x.y), f[1] = make_float2(x.z, x.w);
  f[2] = make_float2(y.x, y.y), f[3] = make_float2(y.z, y.w);
}
__device__ __forceinline__ float2 swapped(float2 x) { return make_float2(x.y, x.x); }
__device__ __forceinline__ float2 negated(float2 x) { return make_float2(-x.x, -x.y); }

// What a lane holds of a row: elements a0 .. a0 + 7 and b0 .. b0 + 7.
template <int D, bool kPairs>
struct Lane {
  static constexpr int kPerRow = D / 16;      // lanes
  static constexpr int kRows = 32 / kPerRow;  // rows of a warp's step
  int l, sub, a0, b0;
  bool turns;  // the lane's elements are rotated
  __device__ __forceinline__ Lane(int rot) {
    const int lane = threadIdx.x & 31;
    l = lane % kPerRow;
    sub = lane / kPerRow;
    turns = 16 * l < rot;
    a0 = kPairs || !turns ? 16 * l : 8 * l;
    b0 = kPairs || !turns ? 16 * l + 8 : 8 * l + rot / 2;
  }
};

// The rotation's factors for what a lane holds, at position p: an element times `own`, plus
// its pair's other element (halves: the one of the other eight; neighbours: the one
// beside it) times `other`.  (Elements that are not rotated have no other one: a product of
// zero and an infinity there would be NaN.)
template <int D, bool kPairs>
__device__ __forceinline__ void load_factors(const NormRopeArgs& a, const Lane<D, kPairs>& L, int p,
                                             float2 (&own_a)[4], float2 (&own_b)[4],
                                             float2 (&other_a)[4], float2 (&other_b)[4]) {
  float2 c[4], s[4];  // of the lane's eight pairs
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = make_float2(1.f, 1.f), s[e] = make_float2(0.f, 0.f);
  if (L.turns) {
    const size_t at = (size_t)p * (a.rot / 2) + 8 * L.l;
    load8(a.cos + at, c);
    load8(a.sin + at, s);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (kPairs) {
      // pairs 0 .. 3 are a's, 4 .. 7 b's
      const float2 ca = c[e / 2], cb = c[2 + e / 2], sa = s[e / 2], sb = s[2 + e / 2];
      const float x = (e & 1) ? ca.y : ca.x, y = (e & 1) ? cb.y : cb.x;
      const float u = (e & 1) ? sa.y : sa.x, v = (e & 1) ? sb.y : sb.x;
      own_a[e] = make_float2(x, x), own_b[e] = make_float2(y, y);
      other_a[e] = make_float2(-u, u), other_b[e] = make_float2(-v, v);
    } else {
      own_a[e] = own_b[e] = c[e];
      other_a[e] = negated(s[e]), other_b[e] = s[e];
    }
  }
}

// The pair's other elements of a and of b.
template <bool kPairs>
__device__ __forceinline__ float2 other(const float2& own, const float2& across) {
  return kPairs ? swapped(own) : across;
}

// A warp's work: units of a token's steps, kRows heads each, q's before k's.  Rows of the
// next steps are on their way to shared memory meanwhile, in a ring of a thread's own
// 16-byte slots: no other thread reads them, so its own wait is all that orders them.
template <int D>
struct Cursor {
  static constexpr int kRows = 32 / (D / 16);
  uint32_t u;
  int token, i, end;  // step i of [.., end) of the token; q's come first
  __device__ __forceinline__ bool more(const Plan& p) const { return u < p.units; }
  __device__ __forceinline__ void place(const Plan& p) {
    token = p.split == 1 ? (int)u : (int)(u / (uint32_t)p.split);
    i = (int)(u - (uint32_t)token * p.split) * p.per;
    end = min(i + p.per, p.steps[0] + p.steps[1]);
  }
  // Whether the next step is of another unit.
  __device__ __forceinline__ bool next(const Plan& p, uint32_t by) {
    if (++i < end) return false;
    u += by;
    place(p);
    return true;
  }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void end_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The lane's place in row (token, first head of a step + sub).
template <typename R>
__device__ __forceinline__ auto row_of(const R& x, int token, int h) {
  return x.x + (token * x.token + h * x.head);
}

// A token's position; -1 where it is of no sequence, or has no angles.
__device__ __forceinline__ int position(const NormRopeArgs& a, int token) {
  const int p = a.pos[token];
  if (p >= a.P && (threadIdx.x & 31) == 0) atomicExch(a.status, (int)FA_ERR_INVALID_ARG);
  return p < a.P ? p : -1;
}

// Both weight vectors as fp32 in shared memory.
template <int D>
__device__ __forceinline__ void load_weights(const NormRopeArgs& a, float (&s_w)[2][D]) {
  if (threadIdx.x < 2 * D) {
    const int kind = threadIdx.x / D, d = threadIdx.x % D;
    s_w[kind][d] = a.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w[kind])[d])
                            : static_cast<const float*>(a.w[kind])[d];
  }
}

template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_rope_kernel(const NormRopeArgs a) {
  using L = Lane<D, kPairs>;
  extern __shared__ uint4 s_rows[];  // [kDepth][2][kThreads]
  __shared__ __align__(16) float s_w[2][D];
  const L lane(a.rot);
  const uint32_t mine = smem_u32(s_rows + threadIdx.x);
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t by = kWarps * gridDim.x;
  const Plan& plan = a.plan;
  Cursor<D> at, ahead;
  at.u = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  at.place(plan);
  ahead = at;
  uint32_t slot = 0, fill = 0;  // of the ring
  auto copy = [&]() {           // step `ahead`
    if (ahead.more(plan)) {
      const int kind = ahead.i >= plan.steps[0] ? 1 : 0;
      const int h = (ahead.i - (kind ? plan.steps[0] : 0)) * L::kRows + lane.sub;
      const bool on = h < a.H[kind];
      const __nv_bfloat16* row = row_of(a.in[kind], ahead.token, on ? h : 0);
      const uint32_t dst = mine + fill * (2 * kThreads * 16);
      copy16(dst, row + lane.a0, on);
      copy16(dst + kThreads * 16, row + lane.b0, on);
      fill = (fill + 1) & (kDepth - 1);
      ahead.next(plan, by);
    }
    end_copies();
  };
#pragma unroll 1
  for (int n = 0; n < kDepth; ++n) copy();
  load_weights<D>(a, s_w);
  __syncthreads();
  int p = at.more(plan) ? position(a, at.token) : -1;
#pragma unroll 1
  while (at.more(plan)) {
    const int token = at.token, end = at.end;
    // the next unit's position, and its angles on their way to L2
    int p_next = -1;
    if (at.u + by < plan.units) {
      Cursor<D> then = at;
      then.u += by;
      then.place(plan);
      p_next = position(a, then.token);
      if (p_next >= 0 && lane.sub == 0 && lane.turns) {
        const size_t to = (size_t)p_next * (a.rot / 2) + 8 * lane.l;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.cos + to));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.sin + to));
      }
    }
    float2 own_a[4], own_b[4], other_a[4], other_b[4];
#pragma unroll 1
    while (at.i < end) {
      const int kind = at.i >= plan.steps[0] ? 1 : 0;
      {
        // the rotation's factors times the weights
        float2 wa[4], wb[4];
        load_factors<D, kPairs>(a, lane, p < 0 ? 0 : p, own_a, own_b, other_a, other_b);
        load8(&s_w[kind][lane.a0], wa);
        load8(&s_w[kind][lane.b0], wb);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          own_a[e] = __fmul2_rn(own_a[e], wa[e]);
          own_b[e] = __fmul2_rn(own_b[e], wb[e]);
          other_a[e] = __fmul2_rn(other_a[e], other<kPairs>(wa[e], wb[e]));
          other_b[e] = __fmul2_rn(other_b[e], other<kPairs>(wb[e], wa[e]));
        }
      }
      const int stop = kind ? end : min(end, plan.steps[0]);
      int h = (at.i - (kind ? plan.steps[0] : 0)) * L::kRows + lane.sub;
      const RowsOut& out = a.out[kind];
      __nv_bfloat16* row = row_of(out, token, h);
      const long long step = L::kRows * out.head;
      const int H = p >= 0 || a.zero ? a.H[kind] : 0;
#pragma unroll 1
      for (; at.i < stop; ++at.i, h += L::kRows, row += step) {
        wait_copies<kDepth - 1>();
        float2 xa[4], xb[4], sum = make_float2(0.f, 0.f), more = sum;
        const uint4* src = s_rows + slot * (2 * kThreads) + threadIdx.x;
        widen(src[0], xa);
        widen(src[kThreads], xb);
        slot = (slot + 1) & (kDepth - 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum = __ffma2_rn(xa[e], xa[e], sum);
          more = __ffma2_rn(xb[e], xb[e], more);
        }
        float ss = (sum.x + sum.y) + (more.x + more.y);
#pragma unroll
        for (int o = L::kPerRow / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        copy();
        const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        const float2 r2 = make_float2(r, r);
        float2 ya[4], yb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 za = __fmul2_rn(xa[e], own_a[e]), zb = __fmul2_rn(xb[e], own_b[e]);
          if (lane.turns) {
            za = __ffma2_rn(other<kPairs>(xa[e], xb[e]), other_a[e], za);
            zb = __ffma2_rn(other<kPairs>(xb[e], xa[e]), other_b[e], zb);
          }
          ya[e] = __fmul2_rn(za, r2);
          yb[e] = __fmul2_rn(zb, r2);
        }
        if (h < H) {
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(row + lane.a0) = p < 0 ? zero : narrow(ya);
          *reinterpret_cast<uint4*>(row + lane.b0) = p < 0 ? zero : narrow(yb);
        }
      }
    }
    at.u += by;
    at.place(plan);
    p = p_next;
  }
}

// The same walk, by blocks of their own for q and for k (one after the other in every block,
// the second would wait for its first rows again).  A warp sums dw over its rows, and the
// sums of its lanes, then of the block's warps, meet in shared memory.  kAll: all of a row is
// rotated, in halves (asked per lane, that takes registers that are not there: 70 -> 71 us for
// 16,384 tokens of 32 heads of 128).
template <int D, bool kPairs, bool kAll>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_rope_grad_kernel(const NormRopeArgs a) {
  using L = Lane<D, kPairs>;
  extern __shared__ uint4 s_rows[];  // [kGradDepth][x, dy][2][kThreads]
  __shared__ __align__(16) float s_w[2][D], s_dw[kWarps][D];
  const L lane(a.rot);
  const uint32_t mine = smem_u32(s_rows + threadIdx.x);
  const int warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int kind = (int)blockIdx.x >= a.blocks_q ? 1 : 0;
  const uint32_t blocks = kind ? gridDim.x - a.blocks_q : a.blocks_q;
  const uint32_t by = kWarps * blocks;
  Plan plan = a.plan;
  plan.steps[0] = a.plan.steps[kind];
  plan.steps[1] = 0;
  plan.per = (plan.steps[0] + plan.split - 1) / plan.split;
  Cursor<D> at, ahead;
  at.u = warp * blocks + blockIdx.x - (kind ? a.blocks_q : 0);
  at.place(plan);
  ahead = at;
  // (a part of a token may have no steps: then it is passed over)
  uint32_t slot = 0, fill = 0;
  auto copy = [&]() {
    while (ahead.more(plan) && ahead.i >= ahead.end) {
      ahead.u += by;
      ahead.place(plan);
    }
    if (ahead.more(plan)) {
      const int h = ahead.i * L::kRows + lane.sub;
      const bool on = h < a.H[kind];
      const __nv_bfloat16* x = row_of(a.in[kind], ahead.token, on ? h : 0);
      const __nv_bfloat16* g = row_of(a.dy[kind], ahead.token, on ? h : 0);
      const uint32_t dst = mine + fill * (4 * kThreads * 16);
      copy16(dst, x + lane.a0, on);
      copy16(dst + kThreads * 16, x + lane.b0, on);
      copy16(dst + 2 * kThreads * 16, g + lane.a0, on);
      copy16(dst + 3 * kThreads * 16, g + lane.b0, on);
      fill = (fill + 1) & (kGradDepth - 1);
      ++ahead.i;
    }
    end_copies();
  };
#pragma unroll 1
  for (int n = 0; n < kGradDepth; ++n) copy();
  load_weights<D>(a, s_w);
  __syncthreads();
  float2 wa[4], wb[4], da[4], db[4];
  load8(&s_w[kind][lane.a0], wa);
  load8(&s_w[kind][lane.b0], wb);
#pragma unroll
  for (int e = 0; e < 4; ++e) da[e] = db[e] = make_float2(0.f, 0.f);
  int p = at.more(plan) ? position(a, at.token) : -1;
#pragma unroll 1
  while (at.more(plan)) {
    const int token = at.token;
    int p_next = -1;
    if (at.u + by < plan.units) {
      Cursor<D> then = at;
      then.u += by;
      then.place(plan);
      p_next = position(a, then.token);
      if (p_next >= 0 && lane.sub == 0 && lane.turns) {
        const size_t to = (size_t)p_next * (a.rot / 2) + 8 * lane.l;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.cos + to));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.sin + to));
      }
    }
    // the transposed rotation: the same factors, the other one's sign turned
    float2 own_a[4], own_b[4], other_a[4], other_b[4];
    load_factors<D, kPairs>(a, lane, p < 0 ? 0 : p, own_a, own_b, other_a, other_b);
    int h = at.i * L::kRows + lane.sub;
    const RowsOut& out = a.out[kind];
    __nv_bfloat16* row = row_of(out, token, h);
    const long long step = L::kRows * out.head;
    const int H = a.H[kind];
#pragma unroll 1
    for (; at.i < at.end; ++at.i, h += L::kRows, row += step) {
      wait_copies<kGradDepth - 1>();
      float2 xa[4], xb[4], ga[4], gb[4];
      const uint4* src = s_rows + slot * (4 * kThreads) + threadIdx.x;
      {
        float2 ya[4], yb[4];
        widen(src[2 * kThreads], ya);
        widen(src[3 * kThreads], yb);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ga[e] = __fmul2_rn(ya[e], own_a[e]);
          gb[e] = __fmul2_rn(yb[e], own_b[e]);
          if (kAll || lane.turns) {
            ga[e] = __ffma2_rn(other<kPairs>(ya[e], yb[e]), kPairs ? swapped(other_a[e]) : other_b[e], ga[e]);
            gb[e] = __ffma2_rn(other<kPairs>(yb[e], ya[e]), kPairs ? swapped(other_b[e]) : other_a[e], gb[e]);
          }
        }
      }
      widen(src[0], xa);
      widen(src[kThreads], xb);
      slot = (slot + 1) & (kGradDepth - 1);
      // sums of x^2 and of h x, h = g w; g x
      float2 sx = make_float2(0.f, 0.f), sy = sx, sh = sx, sg = sx, ta[4], tb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sx = __ffma2_rn(xa[e], xa[e], sx);
        sy = __ffma2_rn(xb[e], xb[e], sy);
        ta[e] = __fmul2_rn(ga[e], xa[e]);
        tb[e] = __fmul2_rn(gb[e], xb[e]);
        sh = __ffma2_rn(ta[e], wa[e], sh);
        sg = __ffma2_rn(tb[e], wb[e], sg);
      }
      float ss = (sx.x + sx.y) + (sy.x + sy.y), hx = (sh.x + sh.y) + (sg.x + sg.y);
#pragma unroll
      for (int o = L::kPerRow / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        hx += __shfl_xor_sync(0xffffffffu, hx, o);
      }
      copy();
      const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
      if (h < H) {
        if (p >= 0) {
          const float m = -(hx * r * (1.f / D)) * (r * r);  // (r^3 may leave fp32's range)
          const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            da[e] = __ffma2_rn(ta[e], r2, da[e]);
            db[e] = __ffma2_rn(tb[e], r2, db[e]);
            ga[e] = __ffma2_rn(__fmul2_rn(ga[e], wa[e]), r2, __fmul2_rn(xa[e], m2));
            gb[e] = __ffma2_rn(__fmul2_rn(gb[e], wb[e]), r2, __fmul2_rn(xb[e], m2));
          }
          *reinterpret_cast<uint4*>(row + lane.a0) = narrow(ga);
          *reinterpret_cast<uint4*>(row + lane.b0) = narrow(gb);
        } else if (a.zero) {
          *reinterpret_cast<uint4*>(row + lane.a0) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(row + lane.b0) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    at.u += by;
    at.place(plan);
    p = p_next;
  }
#pragma unroll
  for (int o = L::kPerRow; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      da[e].x += __shfl_xor_sync(0xffffffffu, da[e].x, o);
      da[e].y += __shfl_xor_sync(0xffffffffu, da[e].y, o);
      db[e].x += __shfl_xor_sync(0xffffffffu, db[e].x, o);
      db[e].y += __shfl_xor_sync(0xffffffffu, db[e].y, o);
    }
  if (lane.sub == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *reinterpret_cast<float2*>(&s_dw[warp][lane.a0 + 2 * e]) = da[e];
      *reinterpret_cast<float2*>(&s_dw[warp][lane.b0 + 2 * e]) = db[e];
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_dw[w][threadIdx.x];
    a.part[(size_t)blockIdx.x * D + threadIdx.x] = sum;
  }
}

// dw from the blocks' sums: 32 of q's or k's D columns a block, 32 warps over the rows.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_sum_kernel(const NormRopeArgs a) {
  __shared__ float s_sum[32][33];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kind = blockIdx.x * 32 / D, col = blockIdx.x * 32 % D + lane;
  const int b0 = kind ? a.blocks_q : 0, b1 = kind ? a.blocks : a.blocks_q;
  float sum = 0.f;
#pragma unroll 10
  for (int b = b0 + warp; b < b1; b += 32) sum += a.part[(size_t)b * D + col];
  s_sum[warp][lane] = sum;
  __syncthreads();
  // column `warp` of the block's, its 32 partial sums a lane each
  float x = s_sum[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0) {
    a.dw[kind][blockIdx.x * 32 % D + warp] = x;
  }
}

// cos and sin of p base^(-2 i / rot), the angle in 64 bits: at p = 131071 fp32 would hold
// it to 2^-7 only.
__global__ void __launch_bounds__(256) rope_table_kernel(float* cos_, float* sin_, long long n, int half,
                                                         double log_base) {
  grid_dep_wait();
  grid_dep_launch();
  for (long long x = (long long)blockIdx.x * 256 + threadIdx.x; x < n; x += (long long)gridDim.x * 256) {
    const long long p = x / half;
    const int i = (int)(x - p * half);
    double s, c;
    sincos((double)p * exp(-log_base * i / half), &s, &c);
    cos_[x] = (float)c;
    sin_[x] = (float)s;
  }
}

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

int check_shape(int T, int Hq, int Hkv, int D, int P, int rot, float eps) {
  if (T < 0 || Hq < 1 || Hkv < 1 || P < 1 || !std::isfinite(eps) || eps < 0.f) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (rot < 16 || rot > D || rot % 16) return FA_ERR_INVALID_ARG;
  // (units, and those a warp looks ahead, are counted in 32 bits: T where it is large)
  if (T > (1 << 30) || Hq > (1 << 20) || Hkv > (1 << 20)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Rows and heads apart by non-negative multiples of 8 elements; outputs by D at least.
int strides(const fa_packed_stride* s, int H, int D, bool written, long long* token, long long* head) {
  *token = s ? (long long)s->token : (long long)H * D;
  *head = s ? (long long)s->head : (long long)D;
  const long long least = written ? D : 0;
  if (*token < least || *head < least || *token > (1LL << 36) || *head > (1LL << 36))
    return FA_ERR_INVALID_ARG;
  return (*token & 7) || (*head & 7) ? FA_ERR_MISALIGNED : FA_OK;
}

// Splits tokens where they are fewer than the warps of the grid, into parts of two steps at
// least; returns the grid: a warp of every SM before a second one of any.
int set_plan(NormRopeArgs* a, int D, int sms, bool backward) {
  const int rows = 32 / (D / 16);
  Plan& p = a->plan;
  for (int i = 0; i < 2; ++i) p.steps[i] = (a->H[i] + rows - 1) / rows;
  const int steps = backward ? (p.steps[0] > p.steps[1] ? p.steps[0] : p.steps[1]) : p.steps[0] + p.steps[1];
  const long long warps = (long long)sms * kBlocks * kWarps;
  long long split = a->T > 0 ? warps / a->T : 1;
  if (split > steps / 2) split = steps / 2;
  p.split = split < 1 ? 1 : (int)split;
  p.per = (steps + p.split - 1) / p.split;
  if (!backward) p.split = (steps + p.per - 1) / p.per;  // (no part without steps)
  p.units = (uint32_t)((long long)a->T * p.split);
  const long long grid = p.units < 1 ? 1 : p.units, most = (long long)sms * kBlocks;
  if (!backward) return (int)(grid < most ? grid : most);
  // q's and k's blocks by their steps, and one for a token's angles
  const long long q = p.steps[0] + 1, all = q + p.steps[1] + 1;
  a->blocks = (int)(2 * grid < most ? 2 * grid : most);
  long long share = (a->blocks * q + all / 2) / all;
  if (share < 1) share = 1;
  if (share > a->blocks - 1) share = a->blocks - 1;
  a->blocks_q = (int)share;
  return a->blocks;
}

// Shared memory of the rings.
constexpr int kSmem = kDepth * 2 * kThreads * 16, kGradSmem = kGradDepth * 4 * kThreads * 16;

int launch(void (*kernel)(NormRopeArgs), long long grid, int threads, int smem, cudaStream_t stream,
           const NormRopeArgs& a) {
  if (launch_pdl(kernel, dim3((unsigned)grid), dim3(threads), smem, stream, a) != cudaSuccess) return FA_ERR_CUDA;
  note_launches(1);
  return FA_OK;
}

// The kernels' shared memory, once per device.
int allow_smem(int dev) {
  static bool done[64] = {};
  if (done[dev]) return FA_OK;
  const auto set = [](void (*kernel)(NormRopeArgs), int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  if (!set(norm_rope_kernel<64, false>, kSmem) ||
      !set(norm_rope_kernel<64, true>, kSmem) ||
      !set(norm_rope_kernel<128, false>, kSmem) ||
      !set(norm_rope_kernel<128, true>, kSmem) ||
      !set(norm_rope_grad_kernel<64, false, false>, kGradSmem) ||
      !set(norm_rope_grad_kernel<64, false, true>, kGradSmem) ||
      !set(norm_rope_grad_kernel<64, true, false>, kGradSmem) ||
      !set(norm_rope_grad_kernel<128, false, false>, kGradSmem) ||
      !set(norm_rope_grad_kernel<128, false, true>, kGradSmem) ||
      !set(norm_rope_grad_kernel<128, true, false>, kGradSmem))
    return FA_ERR_CUDA;
  done[dev] = true;
  return FA_OK;
}

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" {

int fa_rope_table(float* cos, float* sin, int64_t positions, int rot, double base, fa_stream_t stream) {
  reset_launches();
  if (positions < 1 || positions > INT32_MAX || rot < 16 || rot > 128 || rot % 16 || !std::isfinite(base) ||
      base <= 0.0)
    return FA_ERR_INVALID_ARG;
  if (!cos || !sin) return FA_ERR_INVALID_ARG;
  if (misaligned(cos, 16) || misaligned(sin, 16)) return FA_ERR_MISALIGNED;
  int rc = check_device();
  if (rc) return rc;
  const long long n = positions * (rot / 2), blocks = (n + 255) / 256;
  if (launch_pdl(rope_table_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0,
                 static_cast<cudaStream_t>(stream), cos, sin, n, rot / 2, std::log(base)) != cudaSuccess)
    return FA_ERR_CUDA;
  note_launches(1);
  return FA_OK;
}

int fa_norm_rope_fwd(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                     const void* k_weight, int weight_bf16, const float* cos, const float* sin,
                     const int* positions, int T, int Hq, int Hkv, int D, int table_rows, int rot,
                     int interleaved, float eps, const fa_packed_stride* q_stride,
                     const fa_packed_stride* k_stride, const fa_packed_stride* q_out_stride,
                     const fa_packed_stride* k_out_stride, int zero_skipped, fa_stream_t stream) {
  reset_launches();
  int rc = check_shape(T, Hq, Hkv, D, table_rows, rot, eps);
  if (rc) return rc;
  NormRopeArgs a{};
  if ((rc = strides(q_stride, Hq, D, false, &a.in[0].token, &a.in[0].head)) ||
      (rc = strides(k_stride, Hkv, D, false, &a.in[1].token, &a.in[1].head)) ||
      (rc = strides(q_out_stride, Hq, D, true, &a.out[0].token, &a.out[0].head)) ||
      (rc = strides(k_out_stride, Hkv, D, true, &a.out[1].token, &a.out[1].head)))
    return rc;
  if (T == 0) return FA_OK;
  for (const void* p : {q, k, (const void*)q_out, (const void*)k_out, q_weight, k_weight, (const void*)cos,
                        (const void*)sin}) {
    if (!p) return FA_ERR_INVALID_ARG;
    if (misaligned(p, 16)) return FA_ERR_MISALIGNED;
  }
  if (!positions) return FA_ERR_INVALID_ARG;
  if (misaligned(positions, 4)) return FA_ERR_MISALIGNED;
  if ((rc = check_device())) return rc;
  a.in[0].x = static_cast<const __nv_bfloat16*>(q);
  a.in[1].x = static_cast<const __nv_bfloat16*>(k);
  a.out[0].x = static_cast<__nv_bfloat16*>(q_out);
  a.out[1].x = static_cast<__nv_bfloat16*>(k_out);
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.w_bf16 = weight_bf16 ? 1 : 0;
  a.cos = cos;
  a.sin = sin;
  a.pos = positions;
  a.T = T;
  a.H[0] = Hq;
  a.H[1] = Hkv;
  a.P = table_rows;
  a.rot = rot;
  a.zero = zero_skipped ? 1 : 0;
  a.eps = eps;
  a.status = fwd_status_word();
  int dev;
  DeviceInfo info;
  if (!a.status || !current_device(&dev, &info) || allow_smem(dev) != FA_OK) return FA_ERR_CUDA;
  const auto kernel = D == 128 ? (interleaved ? norm_rope_kernel<128, true> : norm_rope_kernel<128, false>)
                               : (interleaved ? norm_rope_kernel<64, true> : norm_rope_kernel<64, false>);
  return launch(kernel, set_plan(&a, D, info.sm_count, false), kThreads, kSmem,
                static_cast<cudaStream_t>(stream), a);
}

size_t fa_norm_rope_workspace_bytes(int T, int Hq, int Hkv, int D) {
  if (check_shape(T, Hq, Hkv, D, 1, 16, 0.f) != FA_OK) return 0;
  int dev;
  DeviceInfo info;
  const int sms = current_device(&dev, &info) ? info.sm_count : 0;
  if (sms < 1) return 0;
  NormRopeArgs a{};
  a.T = T, a.H[0] = Hq, a.H[1] = Hkv;
  return (size_t)set_plan(&a, D, sms, true) * D * sizeof(float);
}

int fa_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq,
                     void* dk, float* dq_weight, float* dk_weight, const void* q_weight,
                     const void* k_weight, int weight_bf16, const float* cos, const float* sin,
                     const int* positions, int T, int Hq, int Hkv, int D, int table_rows, int rot,
                     int interleaved, float eps, const fa_packed_stride* q_stride,
                     const fa_packed_stride* k_stride, const fa_packed_stride* dq_out_stride,
                     const fa_packed_stride* dk_out_stride, const fa_packed_stride* dq_stride,
                     const fa_packed_stride* dk_stride, int zero_skipped, void* workspace,
                     size_t workspace_bytes, fa_stream_t stream) {
  reset_launches();
  int rc = check_shape(T, Hq, Hkv, D, table_rows, rot, eps);
  if (rc) return rc;
  NormRopeArgs a{};
  if ((rc = strides(q_stride, Hq, D, false, &a.in[0].token, &a.in[0].head)) ||
      (rc = strides(k_stride, Hkv, D, false, &a.in[1].token, &a.in[1].head)) ||
      (rc = strides(dq_out_stride, Hq, D, false, &a.dy[0].token, &a.dy[0].head)) ||
      (rc = strides(dk_out_stride, Hkv, D, false, &a.dy[1].token, &a.dy[1].head)) ||
      (rc = strides(dq_stride, Hq, D, true, &a.out[0].token, &a.out[0].head)) ||
      (rc = strides(dk_stride, Hkv, D, true, &a.out[1].token, &a.out[1].head)))
    return rc;
  if (!dq_weight || !dk_weight || !q_weight || !k_weight) return FA_ERR_INVALID_ARG;
  if (T > 0 && (!q || !k || !dq_out || !dk_out || !dq || !dk || !cos || !sin || !positions))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {q, k, dq_out, dk_out, (const void*)dq, (const void*)dk, q_weight, k_weight,
                        (const void*)cos, (const void*)sin})
    if (misaligned(p, 16)) return FA_ERR_MISALIGNED;
  if (misaligned(dq_weight, 4) || misaligned(dk_weight, 4) || misaligned(positions, 4)) return FA_ERR_MISALIGNED;
  if (!workspace || misaligned(workspace, 16)) return FA_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  a.T = T;
  a.H[0] = Hq;
  a.H[1] = Hkv;
  set_plan(&a, D, info.sm_count, true);
  if (workspace_bytes < (size_t)a.blocks * D * sizeof(float)) return FA_ERR_WORKSPACE;
  a.in[0].x = static_cast<const __nv_bfloat16*>(q);
  a.in[1].x = static_cast<const __nv_bfloat16*>(k);
  a.dy[0].x = static_cast<const __nv_bfloat16*>(dq_out);
  a.dy[1].x = static_cast<const __nv_bfloat16*>(dk_out);
  a.out[0].x = static_cast<__nv_bfloat16*>(dq);
  a.out[1].x = static_cast<__nv_bfloat16*>(dk);
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.w_bf16 = weight_bf16 ? 1 : 0;
  a.cos = cos;
  a.sin = sin;
  a.pos = positions;
  a.T = T;
  a.H[0] = Hq;
  a.H[1] = Hkv;
  a.P = table_rows;
  a.rot = rot;
  a.zero = zero_skipped ? 1 : 0;
  a.eps = eps;
  a.part = static_cast<float*>(workspace);
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  a.status = fwd_status_word();
  if (!a.status) return FA_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto kernel = D == 128 ? (interleaved  ? norm_rope_grad_kernel<128, true, false>
                                  : rot == D ? norm_rope_grad_kernel<128, false, true>
                                             : norm_rope_grad_kernel<128, false, false>)
                               : (interleaved  ? norm_rope_grad_kernel<64, true, false>
                                  : rot == D ? norm_rope_grad_kernel<64, false, true>
                                             : norm_rope_grad_kernel<64, false, false>);
  if (allow_smem(dev) != FA_OK) return FA_ERR_CUDA;
  if ((rc = launch(kernel, a.blocks, kThreads, kGradSmem, st, a))) return rc;
  return D == 128 ? launch(norm_rope_sum_kernel<128>, 2 * 128 / 32, 1024, 0, st, a)
                  : launch(norm_rope_sum_kernel<64>, 2 * 64 / 32, 1024, 0, st, a);
}

}  // extern "C"
