// fa_pages.cu -- page tables of a paged cache brought up to date on the device for the
// lengths that its sequences are about to have.
//
// Sequence b holds L = lens[b] tokens and will hold N = new_lens[b]; entry e of its table
// is the page of tokens e s .. e s + s - 1.  Under a window of wl tokens with sinks,
//   hidden(e) = (e + 1) s <= N - 1 - wl and e s >= sinks
// (no query from N - 1 on sees it), entries [hs, he).  With n0 = ceil(L / s), n1 = ceil(N / s):
//   back to the pool  e < n0 with a page of the pool, and hidden or e >= n1; becomes -1
//   from the pool     n0 <= e < n1, not hidden
// The pool is a stack; what comes back goes on top of it in (b, e) order, and what is taken
// then comes from the top, in that order too.  So all places are prefix sums over the
// sequences.  New tokens are packed in (b, position) order; a token's slot is page s +
// position % s, or -1 where its entry has no page.
//
// A few kilobytes move: the time is a launch and a chain of dependent steps.  One block or
// one cluster of blocks does all that the sums are needed for, so that no second launch
// stands between: a warp counts a sequence's entries (up to 32 warps share one where a block has
// few), the blocks' sums meet in shared memory of the cluster, and two barriers of the
// cluster stand where a page that came back may be taken by another block's sequence.  Only many new tokens' positions and slots take a
// second launch, for the whole GPU's stores.
//
// The hidden entries are read in every call, for any of them may still hold a page (it
// may have been taken without the window): 4 bytes for each page's tokens of the past.
//
// Measured: 64 sequences that grow by a token under a window of 4,096 (one block) 5.2 us, 8
// cold; 1,024 sequences, 244,000 new tokens, 15 us and 8 for the second launch (one launch
// for all: 48).
#include <cuda_runtime.h>

#include <climits>

#include "cache4.cuh"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kThreads = 1024;
constexpr int kMaxSequences = 65536;  // their sums lie in shared memory
// One block where a warp has at most two sequences and a window's hidden entries are not too
// many to read, else a cluster of the eight that every device grants.  Measured, us, one block / cluster, a window of 4,096:
// 64 sequences, tables of 524,352 entries in all 17.0 / 9.6, 131,136 9.5 / 8.3, 65,600 8.0 /
// 7.7, 16,448 5.7 / 7.6; one sequence of 65,537 6.4 / 9.3; 524,352 without a window 4.5 / 6.6.
constexpr int kOneBlock = 64, kCluster = 8;
constexpr long long kOneBlockEntries = 131072;
constexpr int kApart = 8192;  // more new tokens than this are written by a launch of their own

struct PageArgs {
  int* table;  // [B, width]
  int width, shift, B;
  int* stack;   // [pages]
  int* height;  // [1]
  int pages;
  const int *lens, *new_lens;
  int wl, sinks;
  int T;
  int* cu;           // [B + 1]
  int* pos;          // [T]
  long long* slots;  // [T]
  int* status;
  int apart;  // slot_kernel writes positions and slots
};

// What a sequence's lengths say about its entries.
struct Sequence {
  int L, N, n0, n1, hs, he;
  __device__ __forceinline__ bool hidden(int e) const { return e >= hs && e < he; }
  // entries taken from the pool: [n0, n1) without [hs, he)
  __device__ __forceinline__ int taken() const {
    const int all = max(0, n1 - n0), skip = max(0, min(he, n1) - max(hs, n0));
    return all - min(all, skip);
  }
};

__device__ __forceinline__ int cut_length(const PageArgs& a, int n) {
  const long long most = (long long)a.width << a.shift;
  return n < 0 ? 0 : (int)min((long long)n, most);
}

__device__ __forceinline__ Sequence make_sequence(const PageArgs& a, int L, int N) {
  Sequence s;
  s.L = L;
  s.N = N;
  const int page = 1 << a.shift;
  s.n0 = (s.L + page - 1) >> a.shift;
  s.n1 = (s.N + page - 1) >> a.shift;
  s.hs = s.he = 0;
  if (a.wl >= 0 && s.N - 1 - a.wl > 0) {
    s.hs = (int)(((long long)a.sinks + page - 1) >> a.shift);
    s.he = (s.N - 1 - a.wl) >> a.shift;
  }
  return s;
}

// Sums of entries taken and returned, and of new tokens (which stay at INT_MAX).
struct Sums {
  int taken, back, tokens;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return {x.taken + y.taken, x.back + y.back,
          (int)min((long long)x.tokens + y.tokens, (long long)INT_MAX)};
}
__device__ __forceinline__ Sums shfl_up(const Sums& x, int o) {
  return {__shfl_up_sync(0xffffffffu, x.taken, o), __shfl_up_sync(0xffffffffu, x.back, o),
          __shfl_up_sync(0xffffffffu, x.tokens, o)};
}

// The entries that may go back to the pool are hidden ones, [hs, min(he, n0)), and those
// behind the new length, [n1, n0) (he <= n1).  2^log warps share a sequence's: the first
// ones in equal parts, the others the last warp's.
struct Stretch {
  int lo, hi;
};
__device__ __forceinline__ Stretch stretch(const Sequence& s, int part, int slice, int log) {
  if (part) return slice == (1 << log) - 1 ? Stretch{s.n1, s.n0} : Stretch{0, 0};
  const long long n = max(0, min(s.he, s.n0) - s.hs);
  return {s.hs + (int)(n * slice >> log), s.hs + (int)(n * (slice + 1) >> log)};
}

// A lane loads several entries at a time, for it is the loads' latency that counts.
constexpr int kAtOnce = 8, kPieces = 4, kTakes = 4;

// The number of pages among them, by a whole warp, 16 bytes a load.
__device__ __forceinline__ int count_returned(const PageArgs& a, int b, const Sequence& s, int slice,
                                              int log) {
  const int lane = threadIdx.x & 31;
  const int* row = a.table + (size_t)b * a.width;
  int count = 0;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const Stretch x = stretch(s, part, slice, log);
    int lo = x.lo;
    const unsigned pages = a.pages;  // (a negative entry is none)
    if (x.hi - lo > 32 * kAtOnce) {
      // a long one: 16 bytes a load, behind the entries in front of the first such piece
      const int edge = (int)(-(reinterpret_cast<uintptr_t>(row + lo) >> 2) & 3);
      if (lane < edge) count += (unsigned)row[lo + lane] < pages;
      lo += edge;
#pragma unroll 1
      for (; lo + 128 * kPieces <= x.hi; lo += 128 * kPieces) {
        int4 page[kPieces];
#pragma unroll
        for (int y = 0; y < kPieces; ++y) page[y] = *reinterpret_cast<const int4*>(row + lo + 128 * y + 4 * lane);
#pragma unroll
        for (int y = 0; y < kPieces; ++y)
          count += ((unsigned)page[y].x < pages) + ((unsigned)page[y].y < pages) +
                   ((unsigned)page[y].z < pages) + ((unsigned)page[y].w < pages);
      }
    }
#pragma unroll 1
    for (; lo < x.hi; lo += 32 * kAtOnce) {
      int page[kAtOnce];
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) {
        const int e = lo + 32 * y + lane;
        page[y] = e < x.hi ? row[e] : -1;
      }
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) count += (unsigned)page[y] < pages;
    }
  }
  return __reduce_add_sync(0xffffffffu, count);
}

// Visits those entries in order, by a whole warp: f(e, page, rank) for the lanes that hold one.
template <typename F>
__device__ __forceinline__ void returned(const PageArgs& a, int b, const Sequence& s, int slice, int log,
                                         F f) {
  const int lane = threadIdx.x & 31;
  const int* row = a.table + (size_t)b * a.width;
  int count = 0;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const Stretch range = stretch(s, part, slice, log);
    const int lo = range.lo, hi = range.hi;
#pragma unroll 1
    for (int e0 = lo; e0 < hi; e0 += 32 * kAtOnce) {
      int page[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int e = e0 + 32 * x + lane;
        page[x] = e < hi ? row[e] : -1;
      }
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const bool on = page[x] >= 0 && page[x] < a.pages;
        const unsigned m = __ballot_sync(0xffffffffu, on);
        if (on) f(e0 + 32 * x + lane, page[x], count + __popc(m & ((1u << lane) - 1)));
        count += __popc(m);
      }
    }
  }
}

// The last of the ascending numbers x[lo .. lo + n - 1] that is at most t.
__device__ __forceinline__ int last_at_or_before(const int* x, int lo, int n, int t) {
  while (n > 1) {
    const int half = n >> 1;
    if (x[lo + half] <= t) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  return lo;
}

__device__ __forceinline__ void write_token(const PageArgs& a, int t, int b, int pos) {
  const int page = a.table[(size_t)b * a.width + (pos >> a.shift)];
  a.pos[t] = pos;
  a.slots[t] = page >= 0 ? ((long long)page << a.shift) + (pos & ((1 << a.shift) - 1)) : -1;
}
__device__ __forceinline__ void write_no_token(const PageArgs& a, int t) {
  a.pos[t] = -1;
  a.slots[t] = -1;
}

template <bool kOne>
__device__ __forceinline__ void sync_all() {
  if constexpr (kOne) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <bool kOne>
__global__ void __launch_bounds__(kThreads) page_kernel(const PageArgs a) {
  // [per] each: taken, back, tokens (counts, then sums before), lengths, of the block's sequences
  extern __shared__ int s_taken[];
  __shared__ Sums s_warp[32], s_total;
  __shared__ int s_slice[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank = 0;
  if constexpr (!kOne) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  constexpr int kBlocks = kOne ? 1 : kCluster;
  const int per = (a.B + kBlocks - 1) / kBlocks;
  int* s_back = s_taken + per;
  int* s_tokens = s_back + per;
  int* s_old = s_tokens + per;
  int* s_new = s_old + per;
  const int b0 = min(a.B, (int)rank * per), n = min(a.B, b0 + per) - b0;
  grid_dep_wait();
  grid_dep_launch();
  bool bad = false;
  int height = *a.height;
  if (height < 0 || height > a.pages) {
    bad = true;
    height = height < 0 ? 0 : a.pages;
  }
  for (int i = tid; i < n; i += kThreads) {
    const int l = a.lens[b0 + i], m = a.new_lens[b0 + i];
    s_old[i] = cut_length(a, l);
    s_new[i] = cut_length(a, m);
    bad |= s_old[i] != l || s_new[i] != m;
  }
  __syncthreads();
  auto sequence = [&](int i) { return make_sequence(a, s_old[i], s_new[i]); };
  // ---- counts, a warp per sequence, or a group of 2^log where the block has few
  int log = 0;
  while (n > 0 && log < 5 && (n << (log + 1)) <= 32) ++log;
  const int slice = warp & ((1 << log) - 1);
  for (int i = warp >> log; i < n; i += 32 >> log) {
    const Sequence s = sequence(i);
    const int back = count_returned(a, b0 + i, s, slice, log);
    if (lane == 0) {
      s_slice[warp] = back;
      if (slice == 0) {
        s_taken[i] = s.taken();
        s_back[i] = back;
        s_tokens[i] = max(0, s.N - s.L);
      }
    }
  }
  __syncthreads();
  if (log > 0) {  // (one sequence to a group)
    if (tid < n) {
      int sum = 0;
      for (int x = 0; x < 1 << log; ++x) sum += s_slice[(tid << log) + x];
      s_back[tid] = sum;
    }
    __syncthreads();
  }
  // ---- sums before each sequence, in the block
  const int each = (n + kThreads - 1) / kThreads, i0 = min(n, tid * each), i1 = min(n, i0 + each);
  Sums own = {0, 0, 0};
  for (int i = i0; i < i1; ++i) own = own + Sums{s_taken[i], s_back[i], s_tokens[i]};
  Sums inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y = shfl_up(inc, o);
    if (lane >= o) inc = y + inc;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Sums w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = shfl_up(w, o);
      if (lane >= o) w = y + w;
    }
    s_warp[lane] = w;
    if (lane == 31) s_total = w;
  }
  __syncthreads();
  sync_all<kOne>();
  // ... and over the blocks before it
  Sums before = {0, 0, 0}, total = {0, 0, 0};
  if constexpr (kOne) {
    total = s_total;
  } else {
    for (int r = 0; r < kBlocks; ++r) {
      Sums x;
      uint32_t at;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&s_total)), "r"(r));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x.taken) : "r"(at));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x.back) : "r"(at + 4));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x.tokens) : "r"(at + 8));
      if (r < (int)rank) before = before + x;
      total = total + x;
    }
  }
  // the sums before the thread's sequences: the warps before, the lanes before
  {
    Sums at = before;
    if (warp > 0) at = at + s_warp[warp - 1];
    const Sums lanes = shfl_up(inc, 1);
    if (lane > 0) at = at + lanes;
    for (int i = i0; i < i1; ++i) {
      const Sums x = {s_taken[i], s_back[i], s_tokens[i]};
      s_taken[i] = at.taken;
      s_back[i] = at.back;
      s_tokens[i] = at.tokens;
      a.cu[b0 + i] = min(at.tokens, a.T);
      at = at + x;
    }
  }
  if (rank == 0 && tid == 0) {
    a.cu[a.B] = min(total.tokens, a.T);
    bad |= total.tokens > a.T;
  }
  __syncthreads();
  // ---- back to the pool
  const Sums end = before + s_total;
  for (int i = warp >> log; i < n; i += 32 >> log) {
    if ((i + 1 < n ? s_back[i + 1] : end.back) == s_back[i]) continue;
    if (log > 0 && s_slice[warp] == 0) continue;
    const Sequence s = sequence(i);
    int* row = a.table + (size_t)(b0 + i) * a.width;
    int first = height + s_back[i];
    for (int x = 0; x < slice; ++x) first += s_slice[warp - slice + x];
    returned(a, b0 + i, s, slice, log, [&](int e, int page, int r) {
      if (first + r < a.pages) a.stack[first + r] = page;
      else bad = true;  // more pages than the pool has: one was held twice
      row[e] = -1;
    });
  }
  sync_all<kOne>();
  // ---- from the pool: the block's entries, dealt to its threads
  const int top = height + total.back;  // (both at most the pool's and the tables' entries)
#pragma unroll 1
  for (int y0 = before.taken + tid; y0 < end.taken; y0 += kTakes * kThreads) {
    int page[kTakes];
#pragma unroll
    for (int z = 0; z < kTakes; ++z) {
      const int y = y0 + z * kThreads, at = top - 1 - y;
      const bool there = at >= 0 && at < a.pages;
      page[z] = y < end.taken && there ? __ldcg(a.stack + at) : -1;
      bad |= y < end.taken && !there;
    }
#pragma unroll 1
    for (int z = 0; z < kTakes; ++z) {
      const int y = y0 + z * kThreads;
      if (y >= end.taken) break;
      const int i = last_at_or_before(s_taken, 0, n, y), x = y - s_taken[i];
      const Sequence s = sequence(i);
      // entries in front of the hidden ones, then those behind them
      const int lo1 = s.n0, hi1 = min(s.n1, max(s.n0, s.hs < s.he ? s.hs : s.n1));
      const int lo2 = s.hs < s.he ? max(s.n0, s.he) : s.n1;
      const int c1 = max(0, hi1 - lo1);
      a.table[(size_t)(b0 + i) * a.width + (x < c1 ? lo1 + x : lo2 + x - c1)] =
          z == 0 ? page[0] : z == 1 ? page[1] : z == 2 ? page[2] : page[3];
    }
  }
  if (rank == 0 && tid == 0) {
    const int left = top - total.taken;
    *a.height = left < 0 ? 0 : min(left, a.pages);
  }
  if (bad) atomicExch(a.status, 1);
  if (a.apart) return;
  __syncthreads();
  // ---- positions and slots of the block's new tokens
  const int lo = min(a.T, before.tokens), hi = n > 0 ? min(a.T, end.tokens) : lo;
  for (int t = lo + tid; t < hi; t += kThreads) {
    const int x = last_at_or_before(s_tokens, 0, n, t);
    write_token(a, t, b0 + x, s_old[x] + t - s_tokens[x]);
  }
  for (int t = min(a.T, total.tokens) + rank * kThreads + tid; t < a.T; t += kBlocks * kThreads)
    write_no_token(a, t);
}

// The same for many tokens, in a launch of its own over the whole GPU: a block takes 1024
// of them, whose sequences lie in a stretch of cu.
constexpr int kChunk = 1024, kStretch = 2048;

__global__ void __launch_bounds__(256) slot_kernel(const PageArgs a) {
  __shared__ int s_cu[kStretch];
  grid_dep_wait();
  grid_dep_launch();
  const int total = a.cu[a.B];
  const int t0 = blockIdx.x * kChunk, t1 = t0 + min(kChunk, total - t0);  // (up to INT_MAX)
  const int lane = threadIdx.x & 31;
  // the sequences of the first and the last token, each by a whole warp's search
  auto find = [&](int t) {
    int lo = 0, n = a.B;
    while (n > 1) {
      const int step = (n + 31) >> 5, at = lo + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, at < lo + n && a.cu[at] <= t);
      const int piece = 31 - __clz(m | 1);
      n = min(step, n - piece * step);
      lo += piece * step;
    }
    return lo;
  };
  int b0 = 0, b1 = 0;
  if (t0 < t1) {
    b0 = find(t0);
    b1 = find(t1 - 1);
  }
  const int n = b1 - b0 + 1;
  const bool near = n <= kStretch;
  for (int i = threadIdx.x; near && i < n; i += 256) s_cu[i] = a.cu[b0 + i];
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kChunk / 256; ++x) {
    const int t = t0 + 256 * x + threadIdx.x;
    if (t < t1) {
      const int i = last_at_or_before(near ? s_cu : a.cu + b0, 0, n, t);
      const int first = near ? s_cu[i] : a.cu[b0 + i];
      write_token(a, t, b0 + i, cut_length(a, a.lens[b0 + i]) + t - first);
    } else if (t < a.T) {
      write_no_token(a, t);
    }
  }
}

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" int fa_page_update(int* page_table, int table_width, int* free_pages, int* free_count,
                              int num_pages, const int* lens, const int* new_lens, int B, int page_size,
                              int window_left, int sinks, int T, int* cu_seqlens, int* positions,
                              int64_t* slots, fa_stream_t stream) {
  reset_launches();
  int rc = check_cache4(num_pages, 1, 64, page_size, B, table_width);
  if (rc) return rc;
  if (B > kMaxSequences || (long long)B * table_width >= (1LL << 30) || num_pages > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (T < 0 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (!page_table || !free_pages || !free_count || !lens || !new_lens || !cu_seqlens ||
      (T > 0 && (!positions || !slots)))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)free_pages, (const void*)free_count,
                        (const void*)lens, (const void*)new_lens, (const void*)cu_seqlens, (const void*)positions})
    if (misaligned(p, 4)) return FA_ERR_MISALIGNED;
  if (misaligned(slots, 8)) return FA_ERR_MISALIGNED;
  if ((rc = check_device())) return rc;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  int* status = cache4_status_word();
  if (!status) return FA_ERR_CUDA;
  const PageArgs a{page_table, table_width, c4_shift(page_size) + 4, B, free_pages, free_count, num_pages,
                   lens, new_lens, window_left < 0 ? -1 : window_left, sinks, T, cu_seqlens, positions,
                   reinterpret_cast<long long*>(slots), status, T > kApart ? 1 : 0};
  static bool attr_done[64] = {};
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(page_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             5 * (kMaxSequences / kCluster) * (int)sizeof(int)) != cudaSuccess)
      return FA_ERR_CUDA;
    attr_done[dev] = true;
  }
  const bool one =
      B <= kOneBlock && (window_left < 0 || (long long)B * table_width <= kOneBlockEntries);
  const int blocks = one ? 1 : kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 5 * (size_t)((B + blocks - 1) / blocks) * sizeof(int);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = one ? 1 : 2;
  if (cudaLaunchKernelEx(&cfg, one ? page_kernel<true> : page_kernel<false>, a) != cudaSuccess)
    return FA_ERR_CUDA;
  note_launches(1);
  if (a.apart) {
    if (launch_pdl(slot_kernel, dim3((unsigned)(((long long)T + kChunk - 1) / kChunk)), dim3(256), 0, cfg.stream, a) !=
        cudaSuccess)
      return FA_ERR_CUDA;
    note_launches(1);
  }
  return FA_OK;
}
