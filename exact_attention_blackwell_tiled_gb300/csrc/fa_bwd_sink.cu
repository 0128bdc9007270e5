// fa_bwd_sink.cu -- backward over the pairs of a query and a sink behind its window, for
// packed calls with sinks.
//
// The first keys j < s of a sequence (s at most 128) stay visible to the queries i > j +
// wl whose window has passed them.  A kv tile's unit of the main kernels walks the
// queries that see it; with sinks in it, tile 0's would walk the whole sequence, alone,
// while the others walk a window.  So those kernels keep to the window, and these pairs
// go the other way round, a tile of 128 queries against the few sinks:
//   S = Q K_s^T, dP = dO V_s^T      (128 x N, N = s rounded up to 16)
//   P = 2^(S scale log2 e - LSE2), dS = P (dP - Delta), 0 where i - j <= wl or j >= s
//   dQ  = dS K_s                    stored as the accumulator's first value
//   dV_s += P^T dO, dK_s += dS^T Q  in TMEM over a run of tiles of one head and sequence
// with P and dS rounded to bf16 for the products, as in the main kernels.  It needs Q, dO
// and the row vectors once and writes dQ in fp32: 4 D + 4 D bytes per query and head, a
// memory-bound pass.  The list of (head, tile) positions is cut into one contiguous share
// per block, one or two of which an SM holds; a run ends with its sequence, head or share
// and leaves one fp32 part of dK_s and dV_s, which the last kernel of the call adds up.
//
// Measured, 16,384 tokens of 16 heads of 128, 16 sinks: 55 us, 4.8 TB/s of the 264 MB (of dQ
// half stays in L2); one block per SM (shared memory), a chain of load, products,
// exponentials, products and stores, 38% of DRAM busy.  Slower: two groups of warps with
// buffers of their own (65), or with the preprocess kernel's work in it (115 against 55 and
// 31 for both).  At head dimension 64, 4,099 tokens of 16 heads, two blocks per SM: 12 us,
// 16 with one.
//
// Warps 0-3: a query row per thread (TMEM lane); warp 4: TMA; warp 5: TMEM and MMAs.
// The dQ columns lie over those of S and dP, which are read before dQ is issued; the next
// tile's S waits until dQ has been read.  P and dS lie in shared memory [query][sinks]
// for both products: a K-major A operand for dQ, an MN-major one for dV_s and dK_s
// (128 sinks wide: rows from N on hold anything and are not read).
#include <cuda_bf16.h>

#include "bwd_common.cuh"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

// kWide: more than 64 sinks.
template <int D, bool kWide>
struct SinkSmem {
  static constexpr int kColBlocks = D / 64;
  static constexpr int kRowsKV = kWide ? 128 : 64;
  static constexpr int kKVBlock = kRowsKV * 128;
  static constexpr int kKVBytes = kKVBlock * kColBlocks;
  static constexpr int kQBlock = kTile * 128;
  static constexpr int kQBytes = kQBlock * kColBlocks;
  static constexpr int kStages = kWide ? 1 : 2;
  static constexpr int kPBlock = kTile * 128;  // 128 queries x 64 sinks
  static constexpr int kPBytes = kPBlock * (kWide ? 2 : 1);
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kKVBytes;
  static constexpr int kOffStage = kOffV + kKVBytes;  // Q, dO
  static constexpr int kOffP = kOffStage + kStages * 2 * kQBytes;
  static constexpr int kOffDS = kOffP + kPBytes;
  static constexpr int kOffBar = kOffDS + kPBytes;
  static constexpr int kBarKVFull = 0, kBarKVEmpty = 1;
  static constexpr int kBarQFull = 2, kBarQEmpty = kBarQFull + kStages;
  static constexpr int kBarSFull = kBarQEmpty + kStages;  // S and dP
  static constexpr int kBarPReady = kBarSFull + 1;
  static constexpr int kBarDQFull = kBarPReady + 1, kBarDQEmpty = kBarDQFull + 1;
  static constexpr int kBarAccFull = kBarDQEmpty + 1, kBarAccEmpty = kBarAccFull + 1;
  static constexpr int kBarDrain = kBarAccEmpty + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kBlocks = D == 64 && !kWide ? 2 : 1;  // per SM
  static constexpr uint32_t kColDP = kRowsKV, kColDV = 2 * kRowsKV < D ? D : 2 * kRowsKV,
                            kColDK = kColDV + D;
  static constexpr uint32_t kTmemCols = kColDK + D <= 256 ? 256 : 512;
  static_assert(kColDK + D <= 512 && kTmemCols * kBlocks <= 512, "TMEM columns");
  static_assert(kBlocks * (kBytes + 1024) <= 228 * 1024, "shared memory");
};

// A share's tiles that have sinks behind the window, in order.
struct SinkTile {
  VarItem it;
  int pad0, h;
  bool valid;
};
struct SinkWalk {
  long long x, end;
  int n_items;
  __device__ __forceinline__ SinkTile next(const BwdArgs& a) {
    SinkTile t;
    t.valid = false;
    for (; x < end; ++x) {
      t.h = (int)(x / n_items);
      const int item = (int)(x - (long long)t.h * n_items);
      t.it = load_item(a.items, item);
      if (sink_tile(a, t.it.len, t.it.tile)) {
        t.pad0 = a.items[item].pad0;
        t.valid = true;
        ++x;
        break;
      }
    }
    return t;
  }
};
__device__ __forceinline__ bool same_run(const SinkTile& a, const SinkTile& b) {
  return b.valid && a.h == b.h && a.it.b == b.it.b;
}

template <int D, bool kWide>
__global__ void __launch_bounds__(192, SinkSmem<D, kWide>::kBlocks)
    bwd_sink_kernel(const BwdArgs a, const __grid_constant__ Tails<true, 4> tails) {
  using L = SinkSmem<D, kWide>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (no room for two blocks of D = 64 with slack)
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::kOffBar + 8 * i; };
  if (threadIdx.x == 0) {
    mbar_init(bar(L::kBarKVFull), 1);
    mbar_init(bar(L::kBarKVEmpty), 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kBarQFull + s), 1);
      mbar_init(bar(L::kBarQEmpty + s), 1);
    }
    mbar_init(bar(L::kBarSFull), 1);
    mbar_init(bar(L::kBarPReady), 128);
    mbar_init(bar(L::kBarDQFull), 1);
    mbar_init(bar(L::kBarDQEmpty), 128);
    mbar_init(bar(L::kBarAccFull), 1);
    mbar_init(bar(L::kBarAccEmpty), 128);
    mbar_init(bar(L::kBarDrain), 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4) prefetch_tails(tails, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = *tmem_slot;
  const int group = a.Hq / a.Hkv;
  const int cols = (a.sinks + 15) & ~15;  // N
  SinkWalk walk;
  walk.n_items = *a.n_items;
  {
    const long long total = (long long)walk.n_items * a.Hq, share = sink_share(a, walk.n_items);
    walk.x = blockIdx.x * share;
    walk.end = walk.x + share < total ? walk.x + share : total;
  }
  if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0, runs = 0;
      bool ok = true, first = true;
      // rows .. of one tensor in pieces of at most 64 (kRows: all that are loaded)
      auto load = [&](uint32_t dst, uint32_t block, int kRows, int tensor, uint32_t b, int row,
                      int valid, int head) {
        for (int r = 0; r < kRows; r += 64)
          load_rows<64, L::kColBlocks>(dst + r * 128, block, &tails.of[tensor].box[0],
                                       tails.of[tensor], b, row + r, valid - r, a.T, head);
      };
      for (SinkTile t = walk.next(a); ok && t.valid;) {
        const int hk = t.h / group;
        if (first) {
          if (!mbar_wait(bar(L::kBarKVEmpty), (runs & 1) ^ 1, abort_flag)) break;
          mbar_arrive_expect_tx(bar(L::kBarKVFull), 2 * L::kKVBytes);
          // (zeros behind the sinks: what lies there is out of sight)
          const int keys = min(a.sinks, t.it.len);
          load(sbase + L::kOffK, L::kKVBlock, L::kRowsKV, 1, bar(L::kBarKVFull), t.it.row0, keys, hk);
          load(sbase + L::kOffV, L::kKVBlock, L::kRowsKV, 2, bar(L::kBarKVFull), t.it.row0, keys, hk);
          ++runs;
        }
        const uint32_t st = it % L::kStages;
        if (!mbar_wait(bar(L::kBarQEmpty + st), ((it / L::kStages) & 1) ^ 1, abort_flag)) break;
        const uint32_t dst = sbase + L::kOffStage + st * 2 * L::kQBytes;
        const int q0 = t.it.tile * kTile;
        mbar_arrive_expect_tx(bar(L::kBarQFull + st), 2 * L::kQBytes);
        load(dst, L::kQBlock, kTile, 0, bar(L::kBarQFull + st), t.it.row0 + q0, t.it.len - q0, t.h);
        load(dst + L::kQBytes, L::kQBlock, kTile, 3, bar(L::kBarQFull + st), t.it.row0 + q0,
             t.it.len - q0, t.h);
        ++it;
        const SinkTile n = walk.next(a);
        first = !same_run(t, n);
        t = n;
      }
      if (runs > 0) drain_wait_b(bar(L::kBarKVFull), (runs - 1) & 1);
      for (uint32_t n = (it > (uint32_t)L::kStages ? it - L::kStages : 0); n < it; ++n)
        drain_wait_b(bar(L::kBarQFull + n % L::kStages), (n / L::kStages) & 1);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_s = idesc_bf16_f32(kTile, cols, false, false);
      constexpr uint32_t kIdDQ = idesc_bf16_f32(kTile, D, false, true);
      constexpr uint32_t kIdAcc = idesc_bf16_f32(kTile, D, true, true);
      constexpr uint32_t kHi = sdesc_hi(1024);
      uint32_t it = 0, runs = 0;
      bool first = true;
      for (SinkTile t = walk.next(a); t.valid;) {
        const SinkTile n = walk.next(a);
        const bool last = !same_run(t, n);
        if (first && !mbar_wait(bar(L::kBarKVFull), runs & 1, abort_flag)) break;
        const uint32_t st = it % L::kStages;
        if (!mbar_wait(bar(L::kBarQFull + st), (it / L::kStages) & 1, abort_flag)) break;
        if (it > 0 && !mbar_wait(bar(L::kBarDQEmpty), (it - 1) & 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t q = sbase + L::kOffStage + st * 2 * L::kQBytes, g = q + L::kQBytes;
        // S = Q K_s^T, dP = dO V_s^T: both operands K-major
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t a_lo = sdesc_lo(x ? g : q, 16);
          const uint32_t b_lo = sdesc_lo(sbase + (x ? L::kOffV : L::kOffK), 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t oa = ((kk >> 2) * L::kQBlock + (kk & 3) * 32) >> 4;
            const uint32_t ob = ((kk >> 2) * L::kKVBlock + (kk & 3) * 32) >> 4;
            const uint32_t d = tmem + (x ? L::kColDP : 0);
            if (kk == 0)
              umma_ss_w<0>(d, a_lo + oa, kHi, b_lo + ob, kHi, id_s);
            else
              umma_ss_w<1>(d, a_lo + oa, kHi, b_lo + ob, kHi, id_s);
          }
        }
        umma_commit(bar(L::kBarSFull));
        if (!mbar_wait(bar(L::kBarPReady), it & 1, abort_flag)) break;
        // the accumulators, once the previous run's have been read
        if (first && runs > 0 && !mbar_wait(bar(L::kBarAccEmpty), (runs - 1) & 1, abort_flag)) break;
        tc_fence_after();
        {
          // dQ = dS K_s (K = sinks)
          const uint32_t a_lo = sdesc_lo(sbase + L::kOffDS, 16);
          const uint32_t b_lo = sdesc_lo(sbase + L::kOffK, L::kKVBlock);
          for (int kk = 0; kk < cols / 16; ++kk) {
            const uint32_t oa = ((kk >> 2) * L::kPBlock + (kk & 3) * 32) >> 4;
            const uint32_t ob = (kk * 16 * 128) >> 4;
            if (kk == 0)
              umma_ss_w<0>(tmem, a_lo + oa, kHi, b_lo + ob, kHi, kIdDQ);
            else
              umma_ss_w<1>(tmem, a_lo + oa, kHi, b_lo + ob, kHi, kIdDQ);
          }
          umma_commit(bar(L::kBarDQFull));
        }
        // dV_s += P^T dO, dK_s += dS^T Q (K = queries)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t a_lo = sdesc_lo(sbase + (x ? L::kOffDS : L::kOffP), kWide ? L::kPBlock : 0);
          const uint32_t b_lo = sdesc_lo(x ? q : g, L::kQBlock);
          const uint32_t d = tmem + (x ? L::kColDK : L::kColDV);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) {
            const uint32_t o = (kk * 16 * 128) >> 4;
            if (kk == 0 && first)
              umma_ss_w<0>(d, a_lo + o, kHi, b_lo + o, kHi, kIdAcc);
            else
              umma_ss_w<1>(d, a_lo + o, kHi, b_lo + o, kHi, kIdAcc);
          }
        }
        umma_commit(bar(L::kBarQEmpty + st));
        if (last) {
          umma_commit(bar(L::kBarKVEmpty));
          umma_commit(bar(L::kBarAccFull));
          ++runs;
        }
        ++it;
        first = last;
        t = n;
      }
      umma_commit(bar(L::kBarDrain));
      drain_wait_b(bar(L::kBarDrain), 0);
    }
  } else {
    // ------------------------------------------------------------ a query row per thread
    const int r = threadIdx.x;
    const uint32_t t_row = tmem + ((uint32_t)(warp * 32) << 16);
    uint8_t* p_row = smem + L::kOffP + r * 128;
    uint8_t* ds_row = smem + L::kOffDS + r * 128;
    uint32_t it = 0, runs = 0;
    bool first = true;
    int run_tile = 0;
    for (SinkTile t = walk.next(a); t.valid;) {
      if (first) run_tile = t.it.tile;
      const int i = t.it.tile * kTile + r;
      const bool real = i < t.it.len;
      float lse2 = INFINITY, delta = 0.f;
      if (real) {
        const size_t at = (size_t)t.h * a.T_pad + t.pad0 + i;
        lse2 = a.lse2[at];
        delta = a.delta[at];
      }
      const SinkTile n = walk.next(a);
      const bool last = !same_run(t, n);
      const int seen = real ? min(a.sinks, i - a.wl) : 0;  // sinks j < seen are behind the window
      if (!warp_wait_b(bar(L::kBarSFull), it & 1, abort_flag)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < cols; c += 16) {
        uint32_t s[16], d[16], wp[8], wd[8];
        __syncwarp();
        tmem_ld<16>(t_row + c, s);
        tmem_ld<16>(t_row + L::kColDP + c, d);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          float p[2], ds[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float x = ex2_mufu(fmaf(u2f(s[e + y]), a.scale_log2, -lse2));
            const bool live = c + e + y < seen;
            p[y] = live ? x : 0.f;
            ds[y] = live ? x * (u2f(d[e + y]) - delta) : 0.f;
          }
          wp[e / 2] = pack_bf16x2(p[0], p[1]);
          wd[e / 2] = pack_bf16x2(ds[0], ds[1]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int chunk = (c >> 3) + y;  // of 8 sinks; 8 chunks to a block
          const uint32_t off = (chunk >> 3) * L::kPBlock + (((chunk & 7) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(p_row + off) = make_uint4(wp[4 * y], wp[4 * y + 1], wp[4 * y + 2], wp[4 * y + 3]);
          *reinterpret_cast<uint4*>(ds_row + off) = make_uint4(wd[4 * y], wd[4 * y + 1], wd[4 * y + 2], wd[4 * y + 3]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bar(L::kBarPReady));
      if (!warp_wait_b(bar(L::kBarDQFull), it & 1, abort_flag)) break;
      tc_fence_after();
      // the tile's rows of dQ
      float* dst = a.dq_acc + ((size_t)t.h * a.T + t.it.row0 + t.it.tile * kTile) * D;
      const int rows = min(kTile, t.it.len - t.it.tile * kTile);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(t_row + c * 32, v);
        if (c == D / 32 - 1) {
          tc_fence_before();
          mbar_arrive(bar(L::kBarDQEmpty));
        }
        store_rows_f32(dst, c, D, v, 1.f, r & ~3, rows, lane);
      }
      ++it;
      if (last) {
        // the run's part of dK_s and dV_s: key rows now
        if (!warp_wait_b(bar(L::kBarAccFull), runs & 1, abort_flag)) break;
        tc_fence_after();
        if (warp * 32 < a.sinks) {
          const size_t base = ((size_t)t.h * a.sink_rows + sink_slot(a, t.it.row0, run_tile)) * D;
          const int keys = min(a.sinks, t.it.len);
#pragma unroll 1
          for (int pass = 0; pass < 2 * (D / 32); ++pass) {
            const int c = pass >> 1;
            const bool is_v = (pass & 1) != 0;
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(t_row + (is_v ? L::kColDV : L::kColDK) + c * 32, v);
            store_rows_f32((is_v ? a.sink_dv : a.sink_dk) + base, c, D, v, is_v ? 1.f : a.scale, r & ~3,
                           keys, lane);
          }
        }
        tc_fence_before();
        mbar_arrive(bar(L::kBarAccEmpty));
        ++runs;
      }
      first = last;
      t = n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicExch(a.status, (int)FA_ERR_TIMEOUT);
}

template <int D, bool kWide>
int launch(const BwdVarMaps& m, const BwdArgs& a, cudaStream_t stream) {
  using L = SinkSmem<D, kWide>;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  static bool attr_done[64] = {};
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(bwd_sink_kernel<D, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             L::kBytes) != cudaSuccess)
      return FA_ERR_CUDA;
    attr_done[dev] = true;
  }
  if (launch_pdl(bwd_sink_kernel<D, kWide>, dim3(a.sink_grid), dim3(192), L::kBytes, stream, a,
                 m.tails) != cudaSuccess)
    return FA_ERR_CUDA;
  return FA_OK;
}

}  // namespace

int bwd_sink_blocks(int D, int sinks, int sms) {
  return sms * (D == 64 && sinks <= 64 ? SinkSmem<64, false>::kBlocks : 1);
}

int launch_bwd_sink(const BwdVarMaps& m, const BwdArgs& a, cudaStream_t stream) {
  if (a.D == 128) return a.sinks > 64 ? launch<128, true>(m, a, stream) : launch<128, false>(m, a, stream);
  return a.sinks > 64 ? launch<64, true>(m, a, stream) : launch<64, false>(m, a, stream);
}

}  // namespace fa
