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
// neighbours paired: 16 in a row.  A row is then D / 16 lanes, a warp holds 8 or 4 rows, and
// takes 8 heads of one token, so that cosines, sines and weights are loaded once for
// them.  dw: sums per lane over all rows that it meets, then over the lanes and warps of
// a block in shared memory; a second kernel adds the blocks', always in the same order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kWarps = 8;
constexpr int kBlocks = 3, kGradBlocks = 2;  // per SM, forward and backward
constexpr int kDepth = 4, kGradDepth = 3;     // steps whose rows are on their way, of a warp
constexpr int kHeads = 8;  // heads of a unit where tokens are few

struct Rows {
  const __nv_bfloat16* x;
  long long token, head;  // elements apart
};
struct RowsOut {
  __nv_bfloat16* x;
  long long token, head;
};

struct NormRopeArgs {
  Rows in[2], dy[2];  // q, k; the gradients of the results
  RowsOut out[2];     // the results, or the inputs' gradients
  const void* w[2];
  int w_bf16;
  const float *cos, *sin;  // [P, rot / 2]
  const int* pos;          // [T]
  int T, H[2], P, rot;
  int heads;  // of a unit
  int zero;  // rows of no sequence get zeros
  float eps;
  int* status;
  float* part;    // [blocks, 2, D] sums of dw
  float* dw[2];   // [D]
  int blocks;
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

// What a lane holds of a row: elements a0 .. a0 + 7 and b0 .. b0 + 7.
template <int D, bool kPairs>
struct Lane {
  static constexpr int kPerRow = D / 16;       // lanes
  static constexpr int kRows = 32 / kPerRow;   // rows of a warp
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

// 8 numbers at p, fp32 or bf16.
__device__ __forceinline__ void load_weights(const void* w, int bf16, int at, float2 (&f)[4]) {
  if (bf16) {
    widen(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at), f);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 x = p[0], y = p[1];
    f[0] = make_float2(x.x, x.y), f[1] = make_float2(x.z, x.w);
    f[2] = make_float2(y.x, y.y), f[3] = make_float2(y.z, y.w);
  }
}

// The lane's cosines and sines at position p: of its 8 pairs.
template <int D, bool kPairs>
__device__ __forceinline__ void load_angles(const NormRopeArgs& a, const Lane<D, kPairs>& L, int p,
                                            float2 (&c)[4], float2 (&s)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = make_float2(1.f, 1.f), s[e] = make_float2(0.f, 0.f);
  if (!L.turns) return;
  const size_t at = (size_t)p * (a.rot / 2) + 8 * L.l;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const float4 x = *reinterpret_cast<const float4*>(a.cos + at + 4 * y);
    const float4 z = *reinterpret_cast<const float4*>(a.sin + at + 4 * y);
    c[2 * y] = make_float2(x.x, x.y), c[2 * y + 1] = make_float2(x.z, x.w);
    s[2 * y] = make_float2(z.x, z.y), s[2 * y + 1] = make_float2(z.z, z.w);
  }
}

// Rotates the lane's 8 pairs by the angle (kBack: its negative).  Halves: (a, b) element by
// element.  Neighbours: pair e of a's four uses angle e, of b's 4 + e.
template <bool kPairs, bool kBack>
__device__ __forceinline__ void turn(float2 (&a)[4], float2 (&b)[4], const float2 (&c)[4],
                                     const float2 (&s)[4]) {
  if constexpr (kPairs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ca = (e & 1) ? c[e / 2].y : c[e / 2].x, sa = (e & 1) ? s[e / 2].y : s[e / 2].x;
      const float cb = (e & 1) ? c[2 + e / 2].y : c[2 + e / 2].x;
      const float sb = (e & 1) ? s[2 + e / 2].y : s[2 + e / 2].x;
      const float2 x = a[e], y = b[e];
      const float ta = kBack ? -sa : sa, tb = kBack ? -sb : sb;
      a[e] = make_float2(fmaf(x.x, ca, -x.y * ta), fmaf(x.y, ca, x.x * ta));
      b[e] = make_float2(fmaf(y.x, cb, -y.y * tb), fmaf(y.y, cb, y.x * tb));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = kBack ? make_float2(-s[e].x, -s[e].y) : s[e];
      const float2 n = make_float2(-t.x, -t.y);
      const float2 x = a[e], y = b[e];
      a[e] = __ffma2_rn(x, c[e], __fmul2_rn(y, n));
      b[e] = __ffma2_rn(y, c[e], __fmul2_rn(x, t));
    }
  }
}

// Token of a unit's rows: -1 where it is of no sequence, or its position has no angles.
__device__ __forceinline__ int position(const NormRopeArgs& a, int token) {
  const int p = __ldg(a.pos + token);
  if (p >= a.P && (threadIdx.x & 31) == 0) atomicExch(a.status, (int)FA_ERR_INVALID_ARG);
  return p < a.P ? p : -1;
}

// A step is kRows heads of one token; a warp takes its units' steps one after the other,
// the next one's rows on their way while it turns the present one's.  A unit is a token and
// `heads` of its heads.
template <int D, bool kPairs>
struct Walk {
  using L = Lane<D, kPairs>;
  int token, h, end;  // the step's heads: h .. min(end, h + kRows) - 1
  uint32_t u, stride, units;  // units are below 2^31
  int per_token, heads, H;
  __device__ __forceinline__ void start(const NormRopeArgs& a, int kind, uint32_t first, uint32_t by) {
    H = a.H[kind];
    heads = a.heads;
    per_token = (H + heads - 1) / heads;
    units = (uint32_t)a.T * per_token;
    u = first;
    stride = by;
    place();
  }
  __device__ __forceinline__ void place() {
    token = (int)(u / (uint32_t)per_token);
    h = (int)(u - (uint32_t)token * per_token) * heads;
    end = min(H, h + heads);
  }
  __device__ __forceinline__ bool more() const { return u < units; }
  __device__ __forceinline__ void next() {
    h += L::kRows;
    if (h >= end) {
      u += stride;
      place();
    }
  }
};

// A lane's two pieces of its row of a step, on their way to shared memory: slots of its own,
// which no other lane reads, so that its own wait is all that orders them.  Zeros where
// the step has no row for it.
__device__ __forceinline__ void copy16(uint32_t dst, const __nv_bfloat16* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
template <int D, bool kPairs>
__device__ __forceinline__ void copy_row(uint32_t dst, const Rows& x, const Walk<D, kPairs>& w,
                                         const Lane<D, kPairs>& lane) {
  const int h = w.h + lane.sub;
  const bool on = w.more() && h < w.end;
  const __nv_bfloat16* row = x.x + (on ? w.token * x.token + h * x.head : 0);
  copy16(dst, row + lane.a0, on);
  copy16(dst + kWarps * 32 * 16, row + lane.b0, on);
}
__device__ __forceinline__ void end_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All groups but the latest n have arrived.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) norm_rope_kernel(const NormRopeArgs a) {
  using L = Lane<D, kPairs>;
  extern __shared__ uint4 s_rows[];  // [kDepth][2][threads]
  constexpr uint32_t kStep = 2 * kWarps * 32 * 16;  // bytes
  const uint32_t mine = smem_u32(s_rows + threadIdx.x);
  const L lane(a.rot);
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t first = (threadIdx.x >> 5) * gridDim.x + blockIdx.x, by = kWarps * gridDim.x;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    Walk<D, kPairs> w;
    // (the other kind's units begin where these end, so that few units spread over all warps)
    const uint32_t shift = kind ? (uint32_t)a.T * ((a.H[0] + a.heads - 1) / a.heads) % by : 0u;
    w.start(a, kind, first >= shift ? first - shift : first - shift + by, by);
    if (!w.more()) continue;
    const RowsOut& out = a.out[kind];
    float2 c[4], s[4], wa[4], wb[4];
    Walk<D, kPairs> ahead = w;
#pragma unroll
    for (int n = 0; n < kDepth; ++n) {
      copy_row<D, kPairs>(mine + n * kStep, a.in[kind], ahead, lane);
      end_copies();
      ahead.next();
    }
    load_weights(a.w[kind], a.w_bf16, lane.a0, wa);
    load_weights(a.w[kind], a.w_bf16, lane.b0, wb);
    int token = -1, p = -1;
#pragma unroll 1
    while (w.more()) {
#pragma unroll
      for (int n = 0; n < kDepth; ++n) {
        if (!w.more()) break;
        if (w.token != token) {
          token = w.token;
          p = position(a, token);
          load_angles<D, kPairs>(a, lane, p < 0 ? 0 : p, c, s);
        }
        float2 fa_[4], fb[4], sum = make_float2(0.f, 0.f);
        wait_copies<kDepth - 1>();
        const uint4* at = s_rows + n * (kStep / 16) + threadIdx.x;
        widen(at[0], fa_);
        widen(at[kWarps * 32], fb);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum = __ffma2_rn(fa_[e], fa_[e], sum);
          sum = __ffma2_rn(fb[e], fb[e], sum);
        }
        float ss = sum.x + sum.y;
#pragma unroll
        for (int o = L::kPerRow / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          fa_[e] = __fmul2_rn(__fmul2_rn(fa_[e], r2), wa[e]);
          fb[e] = __fmul2_rn(__fmul2_rn(fb[e], r2), wb[e]);
        }
        if (lane.turns) turn<kPairs, false>(fa_, fb, c, s);
        copy_row<D, kPairs>(mine + n * kStep, a.in[kind], ahead, lane);
        end_copies();
        ahead.next();
        const int h = w.h + lane.sub;
        if (h < w.end && (p >= 0 || a.zero)) {
          __nv_bfloat16* row = out.x + w.token * out.token + h * out.head;
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(row + lane.a0) = p < 0 ? zero : narrow(fa_);
          *reinterpret_cast<uint4*>(row + lane.b0) = p < 0 ? zero : narrow(fb);
        }
        w.next();
      }
    }
    wait_copies<0>();  // (the next kind's take the same slots)
  }
}

// The warps walk q's units, then k's, and sum dw as they go.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32, kGradBlocks) norm_rope_grad_kernel(const NormRopeArgs a) {
  using L = Lane<D, kPairs>;
  extern __shared__ uint4 s_rows[];  // [kGradDepth][x, dy][2][threads]
  constexpr uint32_t kStep = 4 * kWarps * 32 * 16;  // bytes
  const uint32_t mine = smem_u32(s_rows + threadIdx.x);
  __shared__ float s_dw[kWarps][D];
  const L lane(a.rot);
  const int warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const RowsOut& out = a.out[kind];
    Walk<D, kPairs> w;
    w.start(a, kind, warp * gridDim.x + blockIdx.x, kWarps * gridDim.x);
    float2 wa[4], wb[4], da[4], db[4], c[4], s[4];
    Walk<D, kPairs> ahead = w;
#pragma unroll
    for (int n = 0; n < kGradDepth; ++n) {
      copy_row<D, kPairs>(mine + n * kStep, a.in[kind], ahead, lane);
      copy_row<D, kPairs>(mine + n * kStep + kStep / 2, a.dy[kind], ahead, lane);
      end_copies();
      ahead.next();
    }
    load_weights(a.w[kind], a.w_bf16, lane.a0, wa);
    load_weights(a.w[kind], a.w_bf16, lane.b0, wb);
#pragma unroll
    for (int e = 0; e < 4; ++e) da[e] = db[e] = make_float2(0.f, 0.f);
    int token = -1, p = -1;
#pragma unroll 1
    while (w.more()) {
#pragma unroll
      for (int n = 0; n < kGradDepth; ++n) {
        if (!w.more()) break;
        if (w.token != token) {
          token = w.token;
          p = position(a, token);
          load_angles<D, kPairs>(a, lane, p < 0 ? 0 : p, c, s);
        }
        float2 fa_[4], fb[4], ha[4], hb[4];
        wait_copies<kGradDepth - 1>();
        const uint4* at = s_rows + n * (kStep / 16) + threadIdx.x;
        widen(at[0], fa_);
        widen(at[kWarps * 32], fb);
        widen(at[2 * kWarps * 32], ha);
        widen(at[3 * kWarps * 32], hb);
        if (lane.turns) turn<kPairs, true>(ha, hb, c, s);
        // sums of x^2 and of h x, h = g w
        float2 sx = make_float2(0.f, 0.f), sh = make_float2(0.f, 0.f);
        float2 ta[4], tb[4];  // g x
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sx = __ffma2_rn(fa_[e], fa_[e], sx);
          sx = __ffma2_rn(fb[e], fb[e], sx);
          ta[e] = __fmul2_rn(ha[e], fa_[e]);
          tb[e] = __fmul2_rn(hb[e], fb[e]);
          sh = __ffma2_rn(ta[e], wa[e], sh);
          sh = __ffma2_rn(tb[e], wb[e], sh);
        }
        float ss = sx.x + sx.y, hx = sh.x + sh.y;
#pragma unroll
        for (int o = L::kPerRow / 2; o > 0; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          hx += __shfl_xor_sync(0xffffffffu, hx, o);
        }
        const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        copy_row<D, kPairs>(mine + n * kStep, a.in[kind], ahead, lane);
        copy_row<D, kPairs>(mine + n * kStep + kStep / 2, a.dy[kind], ahead, lane);
        end_copies();
        ahead.next();
        const int h = w.h + lane.sub;
        __nv_bfloat16* row = out.x + w.token * out.token + h * out.head;
        if (p >= 0 && h < w.end) {
          const float m = -(hx * r * (1.f / D)) * (r * r);  // (r^3 may leave fp32's range)
          const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            da[e] = __ffma2_rn(ta[e], r2, da[e]);
            db[e] = __ffma2_rn(tb[e], r2, db[e]);
            ha[e] = __ffma2_rn(__fmul2_rn(ha[e], wa[e]), r2, __fmul2_rn(fa_[e], m2));
            hb[e] = __ffma2_rn(__fmul2_rn(hb[e], wb[e]), r2, __fmul2_rn(fb[e], m2));
          }
          *reinterpret_cast<uint4*>(row + lane.a0) = narrow(ha);
          *reinterpret_cast<uint4*>(row + lane.b0) = narrow(hb);
        } else if (a.zero && h < w.end) {
          *reinterpret_cast<uint4*>(row + lane.a0) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(row + lane.b0) = make_uint4(0u, 0u, 0u, 0u);
        }
        w.next();
      }
    }
    wait_copies<0>();
    // the warp's sums over its rows, then the block's over its warps
#pragma unroll
    for (int o = L::kPerRow; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        da[e].x += __shfl_xor_sync(0xffffffffu, da[e].x, o);
        da[e].y += __shfl_xor_sync(0xffffffffu, da[e].y, o);
        db[e].x += __shfl_xor_sync(0xffffffffu, db[e].x, o);
        db[e].y += __shfl_xor_sync(0xffffffffu, db[e].y, o);
      }
    __syncthreads();
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
      for (int w2 = 0; w2 < kWarps; ++w2) sum += s_dw[w2][threadIdx.x];
      a.part[((size_t)blockIdx.x * 2 + kind) * D + threadIdx.x] = sum;
    }
  }
}

// dw from the blocks' sums: 32 of the 2 D columns a block, 32 warps over the rows.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_sum_kernel(const NormRopeArgs a) {
  __shared__ float s_sum[32][33];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float sum = 0.f;
#pragma unroll 4
  for (int b = warp; b < a.blocks; b += 32) sum += a.part[(size_t)b * 2 * D + col];
  s_sum[warp][lane] = sum;
  __syncthreads();
  // column `warp` of the block's, its 32 partial sums a lane each
  float x = s_sum[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0) {
    const int at = blockIdx.x * 32 + warp;
    a.dw[at / D][at % D] = x;
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
  // units of eight heads, and warps of blocks, are counted in 32 bits
  if ((long long)T * (Hq / kHeads + Hkv / kHeads + 2) >= (1LL << 31) || Hq > (1 << 20) || Hkv > (1 << 20))
    return FA_ERR_INVALID_ARG;
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

// A unit's heads: few where that gives no warp more than kFew units, else a token's, so
// that its angles are loaded once.  Returns the grid, at most `most` blocks.
constexpr int kFew = 4;
int set_units(NormRopeArgs* a, long long most) {
  const int H = a->H[0] > a->H[1] ? a->H[0] : a->H[1];
  const auto count = [&](int heads) {
    return (long long)a->T * ((a->H[0] + heads - 1) / heads + (a->H[1] + heads - 1) / heads);
  };
  a->heads = count(kHeads) <= kFew * most * kWarps ? kHeads : (H + 7) / 8 * 8;
  const long long blocks = (count(a->heads) + kWarps - 1) / kWarps;
  return (int)(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

int grad_blocks(int sms, int T, int Hq, int Hkv) {
  NormRopeArgs a{};
  a.T = T, a.H[0] = Hq, a.H[1] = Hkv;
  return set_units(&a, (long long)sms * kGradBlocks);
}

int launch(void (*kernel)(NormRopeArgs), long long grid, int threads, int smem, cudaStream_t stream,
           const NormRopeArgs& a) {
  if (launch_pdl(kernel, dim3((unsigned)grid), dim3(threads), smem, stream, a) != cudaSuccess) return FA_ERR_CUDA;
  note_launches(1);
  return FA_OK;
}

// Shared memory of the kernels' rows on their way.
constexpr int kSmem = kDepth * 2 * kWarps * 32 * 16, kGradSmem = kGradDepth * 4 * kWarps * 32 * 16;

// The kernels' shared memory, once per device: 0 forward, 1 backward.
int allow_smem(int dev) {
  static bool done[64] = {};
  if (done[dev]) return FA_OK;
  const auto set = [](void (*kernel)(NormRopeArgs), int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  if (!set(norm_rope_kernel<64, false>, kSmem) || !set(norm_rope_kernel<64, true>, kSmem) ||
      !set(norm_rope_kernel<128, false>, kSmem) || !set(norm_rope_kernel<128, true>, kSmem) ||
      !set(norm_rope_grad_kernel<64, false>, kGradSmem) || !set(norm_rope_grad_kernel<64, true>, kGradSmem) ||
      !set(norm_rope_grad_kernel<128, false>, kGradSmem) || !set(norm_rope_grad_kernel<128, true>, kGradSmem))
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
  return launch(kernel, set_units(&a, (long long)info.sm_count * kBlocks), kWarps * 32, kSmem,
                static_cast<cudaStream_t>(stream), a);
}

size_t fa_norm_rope_workspace_bytes(int T, int Hq, int Hkv, int D) {
  if (check_shape(T, Hq, Hkv, D, 1, 16, 0.f) != FA_OK) return 0;
  int dev;
  DeviceInfo info;
  const int sms = current_device(&dev, &info) ? info.sm_count : 0;
  return sms < 1 ? 0 : (size_t)grad_blocks(sms, T, Hq, Hkv) * 2 * D * sizeof(float);
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
  a.blocks = set_units(&a, (long long)info.sm_count * kGradBlocks);
  if (workspace_bytes < (size_t)a.blocks * 2 * D * sizeof(float)) return FA_ERR_WORKSPACE;
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
  const auto kernel =
      D == 128 ? (interleaved ? norm_rope_grad_kernel<128, true> : norm_rope_grad_kernel<128, false>)
               : (interleaved ? norm_rope_grad_kernel<64, true> : norm_rope_grad_kernel<64, false>);
  if (allow_smem(dev) != FA_OK) return FA_ERR_CUDA;
  if ((rc = launch(kernel, a.blocks, kWarps * 32, kGradSmem, st, a))) return rc;
  return D == 128 ? launch(norm_rope_sum_kernel<128>, 2 * 128 / 32, 1024, 0, st, a)
                  : launch(norm_rope_sum_kernel<64>, 2 * 64 / 32, 1024, 0, st, a);
}

}  // extern "C"
