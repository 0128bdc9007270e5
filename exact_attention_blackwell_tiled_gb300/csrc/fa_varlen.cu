// fa_varlen.cu -- attention over packed sequences of different lengths: the plan
// kernel and the entry points fa_fwd_varlen / fa_bwd_varlen.
//
// Sequence b holds rows cu[b] .. cu[b+1]-1 of tensors [T, H, D]; a query sees
// keys of its own sequence only.  The attention kernels are the dense ones
// (fa_fwd.cu, fa_bwd.cu) with another walk over the work:
//   - The lengths are on the device, so a plan kernel lists the work there: one
//     item per pair of query tiles (forward) or kv tile (backward) that exists,
//     the longest first, as the dense causal calls deal theirs.  An item's place
//     is counted in closed form (the items before it, over all sequences), so
//     every item is written at once and no sort or scan runs.
//   - A tile may reach past its sequence's last row: it is loaded in pieces, zeros
//     behind the sequence's rows, by maps over the rows of all sequences (load_rows,
//     var_common.cuh).
// The plan costs one launch of a warp per sequence and no pass over the data; it
// overlaps the end of the kernel before it and the attention kernel's prologue.
// A few sequences are planned by every block of the call's first kernel for itself
// (plan_in_block, var_common.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "fa_internal.h"
#include "ptx.cuh"
#include "var_common.cuh"

namespace fa {

namespace {

constexpr int kPlanWarps = 4;
constexpr int kPlanCache = 4096;  // sequences whose lengths a block keeps

// One warp per sequence.  Bound by the latency of reading cu once and by the
// counting: B steps for every 32 items of a sequence (lanes are items), or B / 32
// for every item where a sequence has few (lanes are the other sequences).  With
// the lengths in shared memory 16384 tokens in 3 sequences take 3.6 us, 437 in short
// ones 3.7 (cold and alone), against 14-25 us when each item read them again.
__global__ void __launch_bounds__(kPlanWarps * 32) plan_kernel(const PlanArgs p) {
  __shared__ int s_len[kPlanCache], s_row0[kPlanWarps];
  __shared__ int s_total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_total = 0;
  __syncthreads();
  grid_dep_wait();  // the caller's kernels may have written cu
  grid_dep_launch();
  const int shift = p.item_rows == 256 ? 8 : 7;
  // every sequence ascending inside [0, T], or no work at all
  int bad = 0, items = 0;
  for (int i = threadIdx.x; i < p.B; i += kPlanWarps * 32) {
    const int lo = p.cu[i], hi = p.cu[i + 1];
    if (lo < 0 || hi < lo || hi > p.T) {
      bad = 1;
    } else {
      items += (hi - lo + p.item_rows - 1) >> shift;
      if (i < kPlanCache) s_len[i] = hi - lo;
      if (i / kPlanWarps == (int)blockIdx.x) s_row0[i % kPlanWarps] = lo;
    }
  }
  if (items && blockIdx.x == 0) atomicAdd(&s_total, items);
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.n_items = bad ? 0 : s_total;
    if (p.clear) {
      *p.status = bad ? (int)FA_ERR_INVALID_ARG : 0;
      *p.counter = 0;
    } else if (bad) {
      atomicExch(p.status, (int)FA_ERR_INVALID_ARG);
    }
  }
  const int b = blockIdx.x * kPlanWarps + warp;
  if (bad || b >= p.B) return;
  auto len_of = [&](int i) { return i < kPlanCache ? s_len[i] : p.cu[i + 1] - p.cu[i]; };
  const int row0 = s_row0[warp], len = len_of(b);
  if (len == 0) return;
  int pad0 = 0;
  for (int i = lane; i < b; i += 32) pad0 += (len_of(i) + p.pad - 1) & -p.pad;
  pad0 = warp_add(pad0);
  const int n_own = (len + p.item_rows - 1) >> shift, blk_own = (len + 63) >> 6;
  const int mode = plan_mode(p);
  auto count = [&](int t, int i) {
    const int n = len_of(i);
    return items_before(mode, t, n_own, blk_own, (n + p.item_rows - 1) >> shift, (n + 63) >> 6, i < b);
  };
  auto place = [&](int t, int before) {
    before += plan_descends(p) ? n_own - 1 - t : t;
    if (before >= p.max_items) return;
    int4* dst = reinterpret_cast<int4*>(p.items) + (p.narrow ? before : 2 * before);
    dst[0] = make_int4(row0, len, t, b);
    if (!p.narrow) dst[1] = make_int4(pad0, 0, 0, 0);
  };
  if (n_own < 8) {
    for (int t = 0; t < n_own; ++t) {
      int before = 0;
      for (int i = lane; i < p.B; i += 32)
        if (i != b) before += count(t, i);
      before = warp_add(before);
      if (lane == 0) place(t, before);
    }
  } else {
    for (int t = lane; t < n_own; t += 32) {
      int before = 0;
      for (int i = 0; i < p.B; ++i)
        if (i != b) before += count(t, i);
      place(t, before);
    }
  }
}

}  // namespace

int launch_plan(const PlanArgs& p, cudaStream_t stream) {
  const int grid = (p.B + kPlanWarps - 1) / kPlanWarps;
  if (launch_pdl(plan_kernel, dim3(grid), dim3(kPlanWarps * 32), 0, stream, p) != cudaSuccess)
    return FA_ERR_CUDA;
  note_launches(1);
  return FA_OK;
}

namespace {

constexpr size_t kHeader = 256;  // status word, item count (+64), unit counter (+128)

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

struct VarLayout {
  int max_items, groups;
  int pad;  // rows of the backward's query blocks
  long long t_pad;
  bool split;  // q heads are units of their own (BwdArgs::dk_part)
  long long sink_rows;  // BwdArgs::sink_rows
  size_t off_sink[4];
  size_t off_items, off_acc, off_delta, off_lse2, off_sem, off_dk, off_dv, total;
};

// Up to this many (kv tile, kv head) units a grouped backward splits its q heads:
// with u units a causal sequence's longest one is 304 / u of an SM's even share of
// 152, so below two to four units per SM the longest unit sets the time.  (The parts take
// 8 T Hq D bytes, at most 80 MB times the group at D = 128: T Hkv is below 77,824.)
constexpr long long kSplitUnits = 608;

// Whether a call with sinks takes those parts.  Under a window a unit has at most about (128 + wl
// + wr) / 64 blocks per head, and units are alike: what counts is how many an SM gets, and
// what each costs besides its blocks: its ends, its parts written and read again, some 4 blocks
// at D = 128, 2 at D = 64.  Measured, us of the whole backward, with parts / without: 4099
// tokens in 5 sequences, 16 / 4 heads, window 300, of 64 88.9 / 74.6, of 128 131.8 / 99.4;
// 9000 tokens in one 160 / 131 and 234 / 175, under 2000 350 / 360 (the rule's worst here)
// and 446 / 426; 4000 in two, 14 / 2 heads, 100, 66.8 / 72.8 (taken) and 122.8 / 92.1.
// (Calls without sinks keep theirs, and the order of their sums.)
bool split_pays(int max_items, int Hq, int Hkv, int T, int D, int wl, int wr, long long sms) {
  if (wr < 0) return true;  // (units of any number of blocks)
  const long long start = D == 128 ? 4 : 2;
  long long blocks = (128LL + wl + wr) / 64 + 1;
  if (blocks > T / 64 + 1) blocks = T / 64 + 1;
  const long long one = (max_items * (long long)Hkv + sms - 1) / sms * (Hq / Hkv * blocks + start);
  const long long parts = (max_items * (long long)Hq + sms - 1) / sms * (blocks + start);
  return parts < one;
}

int check_var(int B, int T, int Hq, int Hkv, int D) {
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (T > (1 << 30) || B > (1 << 18)) return FA_ERR_INVALID_ARG;  // the plan takes B^2 steps
  // units (item, head) and the packed rows over all heads are counted in 32 bits
  const long long t_pad = ((long long)T + 127) / 128 * 128 + 128LL * B;
  if (t_pad * Hq > INT32_MAX) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Forward calls under a window with an even number of q heads to a kv head: a unit is one
// tile of 128 query rows of two heads, not two tiles of one.  Its items are more, but of 16
// bytes, as many as the others' room holds.  Measured, us, two tiles / two heads, 4 sinks:
// 16384 tokens in one sequence, 32 / 8 heads, window 1024, of 128 299 / 273, of 64 259 / 234; 256
// 154 / 136 and 136 / 116; 4099 tokens in 5, 16 / 4 heads, 300, 31.5 / 28.1 and 27.2 / 24.2; 40 of
// 100 23.6 / 19.5 and 20.7 / 17.5; 437 in one, 8 / 1 heads 13.6 / 11.8 and 11.7 / 10.2.  Where
// sequences of one tile leave SMs without a unit, a unit of one head is done sooner: 10 of 44
// tokens, 4 / 2 heads, 8.0 / 9.1 and 6.8 / 7.5.
bool head_pairs(int B, int T, int Hq, int Hkv, int sms) {
  return Hq / Hkv % 2 == 0 && (T >= 128LL * B || (T / 256 + (long long)B) * Hq > sms);
}

// The sinks of a call that count: none where no window hides a key from any query.
int window_sinks(int sinks, int wl, int T) { return wl >= 0 && wl < T - 1 ? sinks : 0; }

VarLayout var_layout(int B, int T, int Hq, int Hkv, int D, bool backward, bool deterministic,
                     int wl, int sinks) {
  VarLayout L{};
  const int rows = backward ? 128 : 256;
  L.max_items = T / rows + B;
  L.off_items = kHeader;
  // (a workspace has room for a tensor map per sequence and tensor behind the items,
  // which nothing uses: its size is part of the interface)
  const size_t maps = (size_t)B * (backward ? 4 : 3) * sizeof(CUtensorMap);
  L.total = up256(up256(L.off_items + (size_t)L.max_items * sizeof(VarItem)) + maps);
  if (!backward) return L;
  // as many accumulators as a dense call of twice the mean length would take (at most;
  // the causal mask and D = 128 use fewer, sinks one, see fa_bwd_varlen_sink)
  const long long twice = 2LL * T / B + 1;
  L.groups = sinks > 0 ? 1 : dq_group_count((int)(twice < T ? twice : T), deterministic);
  L.pad = bwd_qblk_rows(D, deterministic);
  L.t_pad = ((long long)T + L.pad - 1) / L.pad * L.pad + (long long)L.pad * B;
  L.off_acc = L.total;
  L.off_delta = up256(L.off_acc + (size_t)L.groups * Hq * T * D * sizeof(float));
  L.off_lse2 = up256(L.off_delta + (size_t)Hq * L.t_pad * sizeof(float));
  L.off_sem = up256(L.off_lse2 + (size_t)Hq * L.t_pad * sizeof(float));
  L.total = L.off_sem;
  if (deterministic)
    L.total = up256(L.off_sem + (size_t)L.groups * Hq * (L.t_pad / L.pad) * sizeof(int));
  L.split = Hq > Hkv && (long long)L.max_items * Hkv <= kSplitUnits;
  if (L.split) {
    L.off_dk = L.total;
    L.off_dv = up256(L.off_dk + (size_t)Hq * T * D * sizeof(float));
    L.total = up256(L.off_dv + (size_t)Hq * T * D * sizeof(float));
  }
  if (sinks > 0) {
    L.sink_rows = sink_row_count(T, wl, sinks);
    for (int i = 0; i < 4; ++i) {  // dK, dV of the sinks' kernel; of the main kernel
      L.off_sink[i] = L.total;
      const int heads = i < 2 ? Hq : Hkv;
      L.total = up256(L.total + (size_t)heads * L.sink_rows * D * sizeof(float));
    }
  }
  return L;
}

// Rows and heads a tensor's elements are apart: null strides are contiguous.
int tensor_strides(const fa_packed_stride* s, int H, int D, long long* row, long long* head) {
  *row = s ? (long long)s->token : (long long)H * D;
  *head = s ? (long long)s->head : (long long)D;
  if (*row < D || *head < D || *row > (1LL << 36) || *head > (1LL << 36)) return FA_ERR_INVALID_ARG;
  if ((*row & 7) || (*head & 7)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

struct VarTensor {
  const void* p;
  const fa_packed_stride* s;
  int H, box_rows;
};

// A tensor's map over all its rows, in boxes of t.box_rows.
bool full_map(const VarTensor& t, int T, int D, CUtensorMap* map) {
  long long row, head;
  return tensor_strides(t.s, t.H, D, &row, &head) == FA_OK &&
         make_tmap_strided(map, t.p, t.H, T, D, row, head, t.box_rows);
}

// ... and in the pieces' boxes.
bool tail_maps(const VarTensor& t, int T, int D, TailMaps* maps) {
  for (int i = 0; i < kTailBoxes; ++i)
    if (!full_map({t.p, t.s, t.H, 64 >> (2 * i)}, T, D, &maps->box[i])) return false;
  return true;
}

int check_sinks(int sinks) {
  if (sinks < 0) return FA_ERR_INVALID_ARG;
  return sinks > kTile ? FA_ERR_UNSUPPORTED : FA_OK;  // the kernels keep them in one tile
}

int check_strides(const VarTensor* t, int n, int D) {
  for (int i = 0; i < n; ++i) {
    long long row, head;
    const int rc = tensor_strides(t[i].s, t[i].H, D, &row, &head);
    if (rc) return rc;
  }
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_varlen_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int backward,
                                 int deterministic) {
  if (check_var(B, T, Hq, Hkv, D) != FA_OK) return 0;
  return var_layout(B, T, Hq, Hkv, D, backward != 0, deterministic != 0, -1, 0).total;
}

size_t fa_varlen_sink_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int backward,
                                      int deterministic, int window_left, int sinks) {
  if (check_var(B, T, Hq, Hkv, D) != FA_OK || sinks < 0 || sinks > kTile) return 0;
  const int wl = window_side(window_left, T);
  return var_layout(B, T, Hq, Hkv, D, backward != 0, deterministic != 0, wl,
                    window_sinks(sinks, wl, T)).total;
}

int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                  const int* cu_seqlens, int B, int T, int Hq, int Hkv, int D,
                  const fa_packed_stride* q_stride, const fa_packed_stride* k_stride,
                  const fa_packed_stride* v_stride, int window_left, int window_right, float scale,
                  void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  return fa_fwd_varlen_sink(q, k, v, o, lse, cu_seqlens, B, T, Hq, Hkv, D, q_stride, k_stride,
                            v_stride, window_left, window_right, 0, scale, workspace,
                            workspace_bytes, stream);
}

int fa_fwd_varlen_sink(const void* q, const void* k, const void* v, void* o, float* lse,
                       const int* cu_seqlens, int B, int T, int Hq, int Hkv, int D,
                       const fa_packed_stride* q_stride, const fa_packed_stride* k_stride,
                       const fa_packed_stride* v_stride, int window_left, int window_right,
                       int sinks, float scale, void* workspace, size_t workspace_bytes,
                       fa_stream_t stream) {
  reset_launches();
  int rc = check_var(B, T, Hq, Hkv, D);
  if (rc) return rc;
  if ((rc = check_sinks(sinks))) return rc;
  if (!std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  const VarTensor t[3] = {{q, q_stride, Hq, kTile}, {k, k_stride, Hkv, kTile}, {v, v_stride, Hkv, kTile}};
  if ((rc = check_strides(t, 3, D))) return rc;
  if (T == 0) return FA_OK;
  if (!q || !k || !v || !o || !lse || !cu_seqlens) return FA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(lse, 4) || misaligned(cu_seqlens, 4))
    return FA_ERR_MISALIGNED;
  const int wl = window_side(window_left, T), wr = window_side(window_right, T);
  const int seen = window_sinks(sinks, wl, T);
  const VarLayout L = var_layout(B, T, Hq, Hkv, D, false, false, -1, 0);
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < L.total) return FA_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  CUtensorMap maps[3];
  Tails<true, 2> tails;  // of v and k
  for (int i = 0; i < 3; ++i)
    if (!full_map(t[i], T, D, &maps[i])) return FA_ERR_CUDA;
  // (k's are the sinks' in front of a window)
  if (!tail_maps(t[2], T, D, &tails.of[0])) return FA_ERR_CUDA;
  tails.of[1] = tails.of[0];
  if (seen && !tail_maps(t[1], T, D, &tails.of[1])) return FA_ERR_CUDA;
  PlanArgs p{};
  FwdArgs a{};
  a.wl = wl;
  a.wr = wr;
  a.causal = (wl < 0 && wr == 0) ? 1 : 0;
  a.sinks = seen;
  a.head_pairs = (wl >= 0 || wr > 0) && head_pairs(B, T, Hq, Hkv, info.sm_count) ? 1 : 0;
  p.cu = cu_seqlens;
  p.B = B;
  p.T = T;
  p.item_rows = a.head_pairs ? 128 : 256;
  p.pad = 64;
  p.causal = a.causal;
  p.items = reinterpret_cast<VarItem*>(ws + L.off_items);
  p.max_items = a.head_pairs ? T / 128 + B : L.max_items;
  p.narrow = a.head_pairs;
  p.n_items = reinterpret_cast<int*>(ws + 64);
  p.status = fwd_status_word();
  p.counter = reinterpret_cast<int*>(ws + 128);
  if (!p.status) return FA_ERR_CUDA;
  a.o = o;
  a.lse = lse;
  a.status = p.status;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.n_split = 1;
  a.items = p.items;
  a.n_items = p.n_items;
  a.T = T;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long units = (long long)p.max_items * Hq / (a.head_pairs ? 2 : 1);
  if (a.sinks && fwd_plan_fits_block(B, p.max_items, units))
    a.cu = cu_seqlens;
  else if ((rc = launch_plan(p, st)))
    return rc;
  return launch_fwd_var(maps[0], maps[1], maps[2], tails, a, D, p.max_items, st);
}

int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dO,
                  const float* lse, void* dq, void* dk, void* dv, const int* cu_seqlens, int B,
                  int T, int Hq, int Hkv, int D, const fa_packed_stride* q_stride,
                  const fa_packed_stride* k_stride, const fa_packed_stride* v_stride,
                  int window_left, int window_right, float scale, void* workspace,
                  size_t workspace_bytes, int deterministic, fa_stream_t stream) {
  return fa_bwd_varlen_sink(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, B, T, Hq, Hkv, D,
                            q_stride, k_stride, v_stride, window_left, window_right, 0, scale,
                            workspace, workspace_bytes, deterministic, stream);
}

int fa_bwd_varlen_sink(const void* q, const void* k, const void* v, const void* o, const void* dO,
                       const float* lse, void* dq, void* dk, void* dv, const int* cu_seqlens, int B,
                       int T, int Hq, int Hkv, int D, const fa_packed_stride* q_stride,
                       const fa_packed_stride* k_stride, const fa_packed_stride* v_stride,
                       int window_left, int window_right, int sinks, float scale, void* workspace,
                       size_t workspace_bytes, int deterministic, fa_stream_t stream) {
  reset_launches();
  int rc = check_var(B, T, Hq, Hkv, D);
  if (rc) return rc;
  if ((rc = check_sinks(sinks))) return rc;
  if (!std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  const int qrows = bwd_qblk_rows(D, deterministic);
  const VarTensor t[4] = {{q, q_stride, Hq, qrows}, {k, k_stride, Hkv, kTile},
                          {v, v_stride, Hkv, kTile}, {dO, nullptr, Hq, qrows}};
  if ((rc = check_strides(t, 4, D))) return rc;
  if (T == 0) return FA_OK;
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv || !cu_seqlens)
    return FA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(dO, 16) || misaligned(dq, 16) || misaligned(dk, 16) || misaligned(dv, 16) ||
      misaligned(lse, 4) || misaligned(cu_seqlens, 4))
    return FA_ERR_MISALIGNED;
  const int wl = window_side(window_left, T), seen = window_sinks(sinks, wl, T);
  const VarLayout L = var_layout(B, T, Hq, Hkv, D, true, deterministic != 0, wl, seen);
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < L.total) return FA_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  int dev;
  DeviceInfo info;
  if (!current_device(&dev, &info)) return FA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  BwdVarMaps m;
  CUtensorMap* const maps[4] = {&m.q, &m.k, &m.v, &m.dO};
  for (int i = 0; i < 4; ++i)
    if (!full_map(t[i], T, D, maps[i]) || !tail_maps(t[i], T, D, &m.tails.of[i])) return FA_ERR_CUDA;
  PlanArgs p{};
  BwdArgs a{};
  a.wl = wl;
  a.wr = window_side(window_right, T);
  a.causal = (a.wl < 0 && a.wr == 0) ? 1 : 0;
  p.cu = cu_seqlens;
  p.B = B;
  p.T = T;
  p.item_rows = 128;
  p.causal = a.causal;
  p.items = reinterpret_cast<VarItem*>(ws + L.off_items);
  p.max_items = L.max_items;
  p.n_items = reinterpret_cast<int*>(ws + 64);
  p.status = reinterpret_cast<int*>(ws);
  p.clear = 1;
  p.pad = L.pad;
  p.counter = reinterpret_cast<int*>(ws + 128);
  a.o = o;
  a.dO = dO;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dq_acc = reinterpret_cast<float*>(ws + L.off_acc);
  a.delta = reinterpret_cast<float*>(ws + L.off_delta);
  a.lse2 = reinterpret_cast<float*>(ws + L.off_lse2);
  a.sem = reinterpret_cast<int*>(ws + L.off_sem);
  const bool split = L.split && (seen == 0 || split_pays(L.max_items, Hq, Hkv, T, D, a.wl, a.wr, info.sm_count));
  if (split) {
    a.dk_part = reinterpret_cast<float*>(ws + L.off_dk);
    a.dv_part = reinterpret_cast<float*>(ws + L.off_dv);
  }
  if (seen > 0) {
    a.sinks = seen;
    a.sink_rows = L.sink_rows;
    a.sink_dk = reinterpret_cast<float*>(ws + L.off_sink[0]);
    a.sink_dv = reinterpret_cast<float*>(ws + L.off_sink[1]);
    a.sink_dk0 = reinterpret_cast<float*>(ws + L.off_sink[2]);
    a.sink_dv0 = reinterpret_cast<float*>(ws + L.off_sink[3]);
    if (deterministic) {
      // Under a window tile j adds to blocks from 2 j (64 rows) on: from the last tile down
      // the one before has been at a block two steps earlier, so that a chain never
      // waits; upwards each waits for the one before to be two blocks ahead, and the last
      // of those that run at a time for all of them (16384 tokens in one sequence, 32 heads
      // of 64 under 256: 690 us so, atomic 314).
      p.desc = a.desc = 1;
    }
  }
  a.status = p.status;
  a.unit_counter = p.counter;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.deterministic = deterministic ? 1 : 0;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (deterministic) {
    // Accumulators, at most: causal tiles of all heads, dealt together, reach a block
    // one after the other by themselves, so that more of them only cost the convert
    // its reads.  Read off two shapes, one choice for both.  Measured, us of the whole
    // backward, 1 / 2 / 4 accumulators: causal
    // 16 x 1024 tokens of 16 heads of 128 379 / 399 / 425, of 64 275 / 291 / 309; 5 x
    // 820 tokens, 16 / 4 heads, of 128 139 / 140 / 149, of 64 99 / 95 / 97; without a
    // mask of 128 555 / 545 / 567 and 186 / 181 / 187, of 64 493 / 474 / 439 and 148 /
    // 138 / 135.
    // (Sinks, whose chains do not wait: one, L.groups.  4099 tokens, 16 / 4 heads of 64 under
    // 300, 1 / 2 / 4: 87.7 / 90.1 / 93.2, of 128 1 / 4: 133 / 148.)
    const int most = a.causal ? (D == 128 ? 1 : 2) : (D == 128 ? 2 : 4);
    a.dq_groups = L.groups < most ? L.groups : most;
  } else {
    a.dq_groups = 1;
  }
  a.dq_group_stride = (size_t)Hq * T * D;
  a.n_qblk = (int)(L.t_pad / L.pad);
  a.sem_group_stride = Hq * a.n_qblk;
  a.qblk_rows = L.pad;
  {
    // kv heads dealt together, so that their q, dO, dQ accumulators and K / V stay
    // in L2, as in the dense call; in the deterministic mode all of them, since tiles
    // of one head that run side by side wait for each other (16384 tokens in 3
    // sequences, 16 heads of 64: 1,961 -> 1,670 us, before the waits were taken off
    // the adding warps, which made it 1,000)
    const double per_kv_head = (double)(Hq / Hkv) * T * D * (4.0 + 4.0) + (double)T * D * 4.0;
    const double fit = kBwdGroupBytes / per_kv_head;
    const int hg = deterministic || fit >= Hkv ? Hkv : (fit < 1.0 ? 1 : (int)fit);
    a.head_group = hg * (split ? Hq / Hkv : 1);
  }
  a.items = p.items;
  a.n_items = p.n_items;
  a.T = T;
  a.T_pad = (int)L.t_pad;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!bwd_plan_fits_block(B, L.max_items)) {
    if ((rc = launch_plan(p, st))) return rc;
    p.cu = nullptr;
  }
  return launch_bwd_var(m, a, p, L.max_items, st);
}

}  // extern "C"
