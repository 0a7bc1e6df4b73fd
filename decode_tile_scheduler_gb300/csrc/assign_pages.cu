// assign_pages.cu -- fia_assign_pages: a paged cache's block table and free list
// brought up to the sequences' lengths, and the slot and position of every new token.
//
// Two prefix sums over the sequences (pages that go back, pages that are missing) give
// every moved page its place on the free list, so that all of them move independently:
// the k-th missing page of the batch is the k-th from the end of the list with the
// returned ones on it, and where that is a returned one, it is read where it was, in its
// sequence's row of the table.  So nothing that the call writes is read by it (the counts
// apart, where they are changed in place), and its CTAs need not meet in between.
//
// The new tokens are taken in pieces, the rows of a sequence on one page (on 128 rows of
// it), counted by a third prefix sum: a lane finds the page of a piece, then its warp
// writes the rows.  (A search and a page per row bound the call by instructions: 1024
// sequences with 52 k rows 22.5 us.)
//
// Latency-bound: lengths, a scan, then pages (64 sequences of a token 6.1 us a call, 3.4 of
// them in the kernel: scan 0.9, pages 0.8, rows 1.1; 1024 sequences with 1 to 256 rows and
// pages that go back 10.4).  One CTA, or a cluster of sixteen for many rows (eight took
// 12.7 us, half of it the rows: few SMs issue their stores), each of which makes the prefix
// sums of all sequences for itself; past kWhole sequences each makes a slice, and they
// look into each other's shared memory.  (Its CTAs start together, on sixteen free SMs of one
// GPC: beside a kernel on another stream that holds the SMs, the call waits for them.)
#include <atomic>
#include <cstring>

#include "cluster.cuh"
#include "internal.h"

namespace fia {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCtas = 16, kPortable = 8;  // of a cluster: at most, on every device
constexpr int kWhole = 8192;  // sequences whose prefix sums every CTA holds (5000: 25 us, in slices 41)
constexpr int kPieceRows = 128;

struct PagesArgs {
  int B, bs, W, nb, layout, S, T;
  int per;               // sequences of a CTA's prefix sums (all of them up to kWhole)
  int pieces;            // of a page
  uint32_t magic;        // j / bs == (j * magic) >> shift, 0 <= j < 2^31
  int shift;
  const int32_t* lens;
  const int32_t* cu;     // null: S rows per sequence
  const int32_t* seen;
  int32_t* table;
  const int32_t* held;
  int32_t* held_out;
  int32_t* free_pages;
  const int32_t* count;
  int32_t* count_out;
  int32_t* slots;
  int32_t* positions;
  int32_t* status;
};

__device__ __forceinline__ int add_up(int v, int lane) {  // inclusive over a warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// largest i in [lo, hi) with prefix[i] <= x (lo where there is none)
__device__ __forceinline__ int last_at_most(const int32_t* prefix, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

enum { kGive, kTake, kPiece, kHeld, kLen, kArrays };

// The prefix sums as one array, whichever CTA holds them.
struct Sequences {
  // [5][per]: pages back, pages missing and pieces of rows before each; held, length
  const int32_t* smem;
  const int* totals;     // [3] of this CTA's slice
  int per, slices, rank;

  __device__ __forceinline__ int at(int what, int b) const {
    if (slices == 1) return smem[what * per + b];
    const int r = b / per;
    return peer_load(peer_addr(smem + what * per + (b - r * per), r)) + (what < kHeld ? before(what, r) : 0);
  }
  __device__ __forceinline__ int before(int what, int r) const {  // of the slices before r
    int n = 0;
    for (int k = 0; k < r; ++k) n += peer_load(peer_addr(totals + what, k));
    return n;
  }
  // The sequence that page (piece) m of all belongs to: the last one with at most m before
  // it (those without any share theirs with the next).
  __device__ __forceinline__ int of(int what, int B, int m) const {
    if (slices == 1) return last_at_most(smem + what * per, 0, B, m);
    int r = 0, n = 0;
    for (int k = 0; k + 1 < slices; ++k) {
      n += peer_load(peer_addr(totals + what, k));
      if (n <= m) r = k + 1;
    }
    m -= before(what, r);
    int lo = 0, hi = min(per, B - r * per);
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (peer_load(peer_addr(smem + what * per + mid, r)) <= m) lo = mid; else hi = mid;
    }
    return r * per + lo;
  }
};
__global__ void __launch_bounds__(kThreads) assign_pages_kernel(const PagesArgs a) {
  extern __shared__ int32_t smem[];         // Sequences' [kArrays][per], then cu_seqlens_q
  int32_t* s_cu = smem + kArrays * a.per;   // [B + 1] where B <= kWhole
  __shared__ int ws[3][kWarps];
  __shared__ int totals[3];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, threads = (int)blockDim.x;
  const int rank = (int)cluster_rank(), nc = (int)gridDim.x;
  const bool whole = a.B <= kWhole;
  const Sequences seq = {smem, totals, a.per, whole ? 1 : nc, rank};
  const int b0 = whole ? 0 : rank * a.per, n = max(0, min(a.B - b0, a.per));
  const int count = min(max(*a.count, 0), a.nb);
  if (a.cu && whole)
    for (int i = tid; i <= a.B; i += threads) s_cu[i] = __ldg(a.cu + i);
  const auto pages = [&](int64_t j) { return (int)(((uint64_t)(uint32_t)j * a.magic) >> a.shift); };
  const auto need_of = [&](int len) {  // (a length up to the capacity, below 2^31)
    return pages((int64_t)min(max((int64_t)len, (int64_t)0), (int64_t)a.W * a.bs) + a.bs - 1);
  };

  // A sequence's rows: key j of its first one (it may lie before the first key), their
  // number, and the first piece with a key and the pieces in all (one more for rows before
  // the first key).
  struct Rows {
    int64_t j;
    int n, first, pieces;
  };
  const auto piece_of = [&](int64_t j) {
    const int pg = pages(j);
    return a.pieces == 1 ? pg : pg * a.pieces + (int)(j - (int64_t)pg * a.bs) / kPieceRows;
  };
  const auto rows_of = [&](int b, int len) {
    Rows r;
    r.n = a.cu ? max(__ldg(a.cu + b + 1) - __ldg(a.cu + b), 0) : a.S;
    r.j = (int64_t)len - r.n;
    r.first = r.pieces = 0;
    if (r.n > 0 && a.T > 0) {
      if (len > 0) {
        r.first = piece_of(max(r.j, (int64_t)0));
        r.pieces = piece_of(len - 1) - r.first + 1;
      }
      if (r.j < 0) ++r.pieces;
    }
    return r;
  };

  // ---- prefix sums ----
  int carry[3] = {0, 0, 0};
  for (int base = 0; base < n; base += threads) {
    const int i = base + tid;
    int held = 0, need = 0, len = 0, rows = 0;
    if (i < n) {
      held = min(max(a.held[b0 + i], 0), a.W);
      len = __ldg(a.lens + b0 + i);
      need = need_of(len);
      rows = rows_of(b0 + i, len).pieces;
    }
    const int x[3] = {max(held - need, 0), max(need - held, 0), rows};
    int incl[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      incl[k] = add_up(x[k], lane);
      if (lane == 31) ws[k][wid] = incl[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int wv = add_up(32 * lane < threads ? ws[k][lane] : 0, lane);
      const int before = carry[k] + (wid > 0 ? __shfl_sync(0xffffffffu, wv, max(wid - 1, 0)) : 0);
      carry[k] += __shfl_sync(0xffffffffu, wv, 31);
      if (i < n) smem[k * a.per + i] = before + incl[k] - x[k];
    }
    if (i < n) {
      smem[kHeld * a.per + i] = held;
      smem[kLen * a.per + i] = len;
    }
    __syncthreads();
  }
  int all[3] = {carry[0], carry[1], carry[2]};  // pages back, pages missing, pieces
  if (!whole) {
    if (tid < 3) totals[tid] = carry[tid];
    cluster_bar_arrive();
    cluster_bar_wait();
#pragma unroll
    for (int k = 0; k < 3; ++k) all[k] = seq.before(k, nc);
  }
  // This CTA has read the counts: they may be written behind the wait.  (One CTA: the scan's
  // barriers lie between.)
  if (nc > 1) cluster_bar_arrive();
  bool bad = false;
  const int64_t top = min((int64_t)count + all[0], (int64_t)a.nb);  // the list's length after the returns
  // Entry `at` of that list, -1 below its start.
  const auto listed = [&](int64_t at) {
    if (at < 0) return -1;
    if (at < count) return __ldg(a.free_pages + at);
    const int m = (int)(at - count), b = seq.of(kGive, a.B, m);
    return __ldg(a.table + (int64_t)b * a.W + need_of(seq.at(kLen, b)) + m - seq.at(kGive, b));
  };

  // ---- pages that go back, and missing ones ----
  // (threads are counted warp by warp over the CTAs; pages from the last ones on, and the
  // rows below from the first, so that a small call does both at once)
  const int warps = nc * threads / 32, me = (wid * nc + rank) * 32 + lane, everyone = 32 * warps;
  for (int64_t m = everyone - 1 - me; m < all[0]; m += everyone) {
    if (count + m < a.nb) a.free_pages[count + m] = listed(count + m);
    else bad = true;
  }
  for (int64_t m = everyone - 1 - me; m < all[1]; m += everyone) {
    const int b = seq.of(kTake, a.B, (int)m);
    const int page = listed(top - 1 - m);
    bad = bad || top - 1 - m < 0;
    a.table[(int64_t)b * a.W + seq.at(kHeld, b) + (int)m - seq.at(kTake, b)] = page;
  }

  // ---- the tokens' slots and positions: up to 32 pieces to a warp ----
  const int per = min(32, max(1, (all[2] + warps / 2 - 1) / (warps / 2)));
  const int32_t* cu = whole ? s_cu : a.cu;
  for (int64_t m0 = (int64_t)per * (me >> 5); m0 < all[2]; m0 += (int64_t)per * warps) {
    const int64_t m = lane < per ? m0 + lane : all[2];
    // the piece's rows, and the slot (-1: of all of them) and position (kNone: -1 for all)
    // of its first
    constexpr int kNone = INT32_MIN;
    int t = 0, rows = 0, slot = -1, position = kNone;
    if (m < all[2]) {
      const int b = seq.of(kPiece, a.B, (int)m), len = seq.at(kLen, b);
      const Rows r = rows_of(b, len);
      int k = (int)m - seq.at(kPiece, b);
      t = a.cu ? cu[b] : b * a.S;
      if (r.j < 0 && k == 0) {  // before the first key
        rows = (int)min(-r.j, (int64_t)r.n);
      } else {
        k += r.first - (r.j < 0 ? 1 : 0);
        const int pg = a.pieces == 1 ? k : k / a.pieces, at = (k - pg * a.pieces) * kPieceRows;
        const int64_t start = (int64_t)pg * a.bs;
        const int64_t ja = max(max(r.j, (int64_t)0), start + at);
        rows = (int)(min(min((int64_t)len, start + a.bs), start + at + (a.pieces == 1 ? a.bs : kPieceRows)) - ja);
        t += (int)(ja - r.j);
        position = a.seen ? __ldg(a.seen + b) - (int)(len - ja) : (int)ja;
        int page = -1;
        if ((uint32_t)pg < (uint32_t)a.W) {  // (cu_seqlens_q that does not ascend: anything)
          const int held = seq.at(kHeld, b);
          page = pg < held ? __ldg(a.table + (int64_t)b * a.W + pg)
                           : listed(top - 1 - seq.at(kTake, b) - (pg - held));
        }
        if (page >= 0 && page < a.nb) slot = page * a.bs + (int)(ja - start);
        else bad = true;
      }
    }
    const auto write = [&](int to, int i, int s0, int p0) {
      if (to >= 0 && to < a.T) {
        if (a.slots) a.slots[to] = s0 < 0 ? -1 : s0 + i;
        if (a.positions) a.positions[to] = p0 == kNone ? -1 : p0 + i;
      }
    };
    if (rows == 1) write(t, 0, slot, position);
    for (uint32_t left = __ballot_sync(0xffffffffu, rows > 1); left; left &= left - 1) {
      const int l = __ffs(left) - 1;
      const int t1 = __shfl_sync(0xffffffffu, t, l), n1 = __shfl_sync(0xffffffffu, rows, l);
      const int s1 = __shfl_sync(0xffffffffu, slot, l), p1 = __shfl_sync(0xffffffffu, position, l);
      for (int i = lane; i < n1; i += 32) write(t1 + i, i, s1, p1);
    }
  }
  if (a.cu) {  // rows of no sequence
    const int first = min(max(cu[0], 0), a.T), end = min(max(cu[a.B], 0), a.T);
    for (int t = me; t < first + a.T - end; t += everyone) {
      const int to = t < first ? t : t - first + end;
      if (a.slots) a.slots[to] = -1;
      if (a.positions) a.positions[to] = -1;
    }
  }
  if (bad && a.status) atomicExch(a.status, 3);

  // ---- counts ----
  if (nc > 1) cluster_bar_wait();
  for (int b = me; b < a.B; b += everyone) {
    const int need = need_of(seq.at(kLen, b)), held = seq.at(kHeld, b);
    const int64_t left = max(top - seq.at(kTake, b), (int64_t)0);
    a.held_out[b] = need <= held ? need : held + (int)min((int64_t)(need - held), left);
  }
  if (me == 0) *a.count_out = (int)max(top - all[1], (int64_t)0);
  if (!whole) {  // (the peers' reads of this CTA's memory)
    cluster_bar_arrive();
    cluster_bar_wait();
  }
}

// CTAs of a large call's cluster, and the kernel made ready for them, once a device.
cudaError_t pages_ctas(int dev, int* n) {
  static std::atomic<int> known[256];
  std::atomic<int>& mine = known[dev & 255];
  *n = mine.load();
  if (*n) return cudaSuccess;
  constexpr int smem = 4 * (kArrays * kWhole + kWhole + 1);
  static_assert(smem >= 4 * kArrays * (65536 / kPortable), "a slice of the largest batch");
  cudaError_t e = cudaFuncSetAttribute(assign_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  *n = kPortable;
  if (cudaFuncSetAttribute(assign_pages_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, assign_pages_kernel, &cfg) == cudaSuccess && fit > 0) *n = kMaxCtas;
  }
  cudaGetLastError();  // (a device without such clusters is no error)
  mine.store(*n);
  return cudaSuccess;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

}  // namespace fia

extern "C" size_t fia_sizeof_pages_params(void) { return sizeof(fia_pages_params); }

extern "C" fia_status fia_assign_pages(const fia_pages_params* p, void* stream) {
  fia::NvtxRange range("fia_assign_pages");
  using namespace fia;
  if (!p) return FIA_ERR_NULL_ARG;
  for (int i = 0; i < 8; ++i)
    if (p->reserved[i] != 0) return FIA_ERR_BAD_SHAPE;
  if (p->batch < 1 || p->batch > 65536) return FIA_ERR_BAD_SHAPE;
  if (p->block_size <= 0 || p->block_size % 16 || p->block_size > 1024) return FIA_ERR_BAD_SHAPE;
  if (p->num_blocks <= 0 || p->max_blocks_per_seq <= 0) return FIA_ERR_BAD_SHAPE;
  if ((int64_t)p->num_blocks * p->block_size > INT32_MAX) return FIA_ERR_BAD_SHAPE;
  if ((int64_t)p->max_blocks_per_seq * p->block_size > 20971520) return FIA_ERR_BAD_SHAPE;
  if ((int64_t)p->batch * p->max_blocks_per_seq > INT32_MAX) return FIA_ERR_BAD_SHAPE;
  if (p->layout != FIA_LAYOUT_BSND && p->layout != FIA_LAYOUT_TND) return FIA_ERR_BAD_SHAPE;
  const bool tnd = p->layout == FIA_LAYOUT_TND;
  if (tnd ? p->total_q < 0 : p->seqlen_q < 0 || p->seqlen_q > 20971520) return FIA_ERR_BAD_SHAPE;
  if (tnd && !p->cu_seqlens_q) return FIA_ERR_NULL_ARG;
  if (!p->seqused_kv || !p->block_table || !p->pages_held || !p->pages_held_out || !p->free_pages ||
      !p->free_count || !p->free_count_out)
    return FIA_ERR_NULL_ARG;
  for (const void* q : {(const void*)p->seqused_kv, (const void*)p->cu_seqlens_q,
                        (const void*)p->tokens_seen, (const void*)p->block_table,
                        (const void*)p->pages_held, (const void*)p->pages_held_out,
                        (const void*)p->free_pages, (const void*)p->free_count,
                        (const void*)p->free_count_out, (const void*)p->slots,
                        (const void*)p->positions, (const void*)p->status})
    if (!aligned4(q)) return FIA_ERR_BAD_SHAPE;
  // (counts that overlap in part: a sequence's would be read after another's was written)
  if (rows_overlap(p->pages_held, p->pages_held_out, 1, p->batch, p->batch)) return FIA_ERR_BAD_SHAPE;
  const int64_t rows = tnd ? p->total_q : (int64_t)p->batch * p->seqlen_q;
  // (counted in 32 bits, in strides of all threads)
  if (rows > INT32_MAX - kMaxCtas * kThreads) return FIA_ERR_BAD_SHAPE;
  PagesArgs a;
  memset(&a, 0, sizeof a);
  a.B = p->batch;
  a.bs = p->block_size;
  a.W = p->max_blocks_per_seq;
  a.nb = p->num_blocks;
  a.layout = p->layout;
  a.S = p->seqlen_q;
  a.T = p->slots || p->positions ? (int)rows : 0;
  a.pieces = (p->block_size + kPieceRows - 1) / kPieceRows;
  int l = 0;
  while ((1 << l) < a.bs) ++l;
  a.magic = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint64_t)a.bs + 1);
  a.shift = 31 + l;
  a.lens = p->seqused_kv;
  a.cu = tnd ? p->cu_seqlens_q : nullptr;
  a.seen = p->tokens_seen;
  a.table = p->block_table;
  a.held = p->pages_held;
  a.held_out = p->pages_held_out;
  a.free_pages = p->free_pages;
  a.count = p->free_count;
  a.count_out = p->free_count_out;
  a.slots = p->slots;
  a.positions = p->positions;
  a.status = p->status;
  int dev = 0, most = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || pages_ctas(dev, &most) != cudaSuccess) return FIA_ERR_CUDA;
  // (1024 sequences, 6.5 k pages back: eight CTAs 13.1 us with 49 k rows; one 14.5 with 800)
  const int nc = a.B > kThreads / 2 || a.T > 2 * kThreads ? most : 1;
  a.per = a.B <= kWhole ? a.B : (a.B + nc - 1) / nc;
  const size_t smem = 4 * (kArrays * (size_t)a.per + (a.cu && a.B <= kWhole ? a.B + 1 : 0));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc);
  // (a small call's barriers and launch are shorter with fewer warps)
  cfg.blockDim = dim3(nc > 1 || a.B > 256 || a.T > 512 ? kThreads : 256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = nc > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, assign_pages_kernel, a) == cudaSuccess ? FIA_OK : FIA_ERR_CUDA;
}
