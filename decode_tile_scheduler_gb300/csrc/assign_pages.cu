// assign_pages.cu -- fia_assign_pages: a paged cache's block table and free list
// brought up to the sequences' lengths, and the slot and position of every new token.
//
// Two prefix sums over the sequences (pages that go back, pages that are missing) give
// every moved page its place on the free list, so that all of them move independently:
// the k-th missing page of the batch is the k-th from the end of the list with the
// returned ones on it.  A token's slot needs no table entry that this call writes: a
// page it takes is found on the list.
//
// Latency-bound (lengths, then a scan, then pages): one CTA, or a cluster of eight for
// many sequences or rows, each CTA with a slice of the sequences whose prefixes lie in
// its shared memory, where the others read them.  (A grid would have to meet between
// the returns and the takes; a cluster's barrier is the cheaper one.)
#include <atomic>
#include <cstring>

#include "cluster.cuh"
#include "internal.h"

namespace fia {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kCuMax = 4096;  // sequences whose cu_seqlens_q is kept in shared memory

struct PagesArgs {
  int B, bs, W, nb, layout, S, T;
  int per;               // sequences of a CTA
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

// largest i with prefix[i] <= x (prefix[0] <= x)
__device__ __forceinline__ int last_at_most(const int32_t* prefix, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) assign_pages_kernel(const PagesArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* s_give = smem;                // [per] pages given back before each sequence of the slice
  int32_t* s_take = smem + a.per;        // [per] pages missing before it
  int32_t* s_held = smem + 2 * a.per;    // [per] pages held, clamped
  int32_t* s_cu = smem + 3 * a.per;      // [B + 1] where B <= kCuMax
  __shared__ int ws[2][kWarps];
  __shared__ int mine[2];  // the slice's pages back, and missing
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)cluster_rank(), nc = (int)gridDim.x;
  const int b0 = rank * a.per, n = max(0, min(a.B - b0, a.per));
  const int count = min(max(__ldg(a.count), 0), a.nb);
  const bool cu_here = a.cu && a.B <= kCuMax;
  if (cu_here)
    for (int i = tid; i <= a.B; i += kThreads) s_cu[i] = __ldg(a.cu + i);
  const auto pages = [&](int64_t j) { return (int)(((uint64_t)(uint32_t)j * a.magic) >> a.shift); };
  const auto need_of = [&](int len) {  // (a length up to the capacity, below 2^31)
    return pages((int64_t)min(max((int64_t)len, (int64_t)0), (int64_t)a.W * a.bs) + a.bs - 1);
  };

  // ---- prefix sums of the slice ----
  int carry[2] = {0, 0};
  for (int base = 0; base < a.per; base += kThreads) {
    const int i = base + tid;
    int held = 0, need = 0;
    if (i < n) {
      held = min(max(a.held[b0 + i], 0), a.W);
      need = need_of(__ldg(a.lens + b0 + i));
    }
    const int x[2] = {max(held - need, 0), max(need - held, 0)};
    int incl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      incl[k] = add_up(x[k], lane);
      if (lane == 31) ws[k][wid] = incl[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int wv = add_up(ws[k][lane], lane);
      const int before = carry[k] + (wid > 0 ? __shfl_sync(0xffffffffu, wv, max(wid - 1, 0)) : 0);
      carry[k] += __shfl_sync(0xffffffffu, wv, 31);
      if (i < n) (k ? s_take : s_give)[i] = before + incl[k] - x[k];
    }
    if (i < n) s_held[i] = held;
    __syncthreads();
  }
  if (tid == 0) {
    mine[0] = carry[0];
    mine[1] = carry[1];
  }
  cluster_bar_arrive();
  cluster_bar_wait();  // (every count and held has been read: they may be written now)
  int give0 = 0, take0 = 0, gives = 0, takes = 0;  // before this slice, and in all
  for (int r = 0; r < nc; ++r) {
    const int g = peer_load(peer_addr(&mine[0], r)), k = peer_load(peer_addr(&mine[1], r));
    if (r < rank) {
      give0 += g;
      take0 += k;
    }
    gives += g;
    takes += k;
  }
  bool bad = false;

  // ---- pages that go back ----
  // (B * W below 2^31 bounds every count; m steps past it by less than kThreads)
  for (int64_t m = tid; m < carry[0]; m += kThreads) {
    const int i = last_at_most(s_give, n, (int)m);
    // (sequences without returns share their prefix with the one behind: the last is it)
    const int need = need_of(__ldg(a.lens + b0 + i));
    const int64_t at = (int64_t)count + give0 + m;
    if (at < a.nb) a.free_pages[at] = a.table[(int64_t)(b0 + i) * a.W + need + ((int)m - s_give[i])];
    else bad = true;
  }
  const int64_t top = min((int64_t)count + gives, (int64_t)a.nb);  // the list's length then
  if (gives > 0) {
    cluster_bar_arrive();
    cluster_bar_wait();
  }

  // ---- missing pages ----
  for (int64_t m = tid; m < carry[1]; m += kThreads) {
    const int i = last_at_most(s_take, n, (int)m);
    const int64_t at = top - 1 - take0 - m;
    int page = -1;
    if (at >= 0) page = __ldcg(a.free_pages + at); else bad = true;
    a.table[(int64_t)(b0 + i) * a.W + s_held[i] + ((int)m - s_take[i])] = page;
  }
  for (int i = tid; i < n; i += kThreads) {
    const int need = need_of(__ldg(a.lens + b0 + i)), held = s_held[i];
    const int64_t left = max(top - take0 - s_take[i], (int64_t)0);
    a.held_out[b0 + i] = need <= held ? need : held + (int)min((int64_t)(need - held), left);
  }
  if (rank == 0 && tid == 0) *a.count_out = (int)max(top - takes, (int64_t)0);

  // ---- the tokens' slots and positions ----
  if (a.slots || a.positions) {
    for (int t = rank * kThreads + tid; t < a.T; t += nc * kThreads) {
      int b, i, q_len;
      if (a.cu) {
        const int32_t* cu = cu_here ? s_cu : a.cu;
        b = last_at_most(cu, a.B, t);
        i = t - cu[b];
        q_len = cu[b + 1] - cu[b];
      } else {
        b = t / a.S;
        i = t - b * a.S;
        q_len = a.S;
      }
      int slot = -1, position = -1;
      const int len = __ldg(a.lens + b);
      const int64_t j = (int64_t)len - q_len + i;
      if (i >= 0 && i < q_len && j >= 0) {
        position = a.seen ? __ldg(a.seen + b) - q_len + i : (int)j;
        int page = -1;
        if (j < (int64_t)a.W * a.bs) {
          const int pg = pages(j), r = b / a.per, k = b - r * a.per;
          const int held = r == rank ? s_held[k] : peer_load(peer_addr(s_held + k, r));
          if (pg < held) {
            page = a.table[(int64_t)b * a.W + pg];
          } else {
            int before = take0;
            if (r != rank) {
              before = 0;
              for (int k2 = 0; k2 < r; ++k2) before += peer_load(peer_addr(&mine[1], k2));
            }
            const int take = r == rank ? s_take[k] : peer_load(peer_addr(s_take + k, r));
            const int64_t at = top - 1 - before - take - (pg - held);
            if (at >= 0) page = __ldcg(a.free_pages + at);
          }
          if (page >= 0 && page < a.nb) slot = page * a.bs + (int)(j - (int64_t)pg * a.bs);
        }
        bad = bad || slot < 0;
      }
      if (a.slots) a.slots[t] = slot;
      if (a.positions) a.positions[t] = position;
    }
  }
  if (bad && a.status) atomicExch(a.status, 3);
  if (nc > 1) {  // (the peers' reads of this CTA's memory)
    cluster_bar_arrive();
    cluster_bar_wait();
  }
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
  if (rows > INT32_MAX - 8192) return FIA_ERR_BAD_SHAPE;  // (counted in 32 bits, in strides of 8192)
  PagesArgs a;
  memset(&a, 0, sizeof a);
  a.B = p->batch;
  a.bs = p->block_size;
  a.W = p->max_blocks_per_seq;
  a.nb = p->num_blocks;
  a.layout = p->layout;
  a.S = p->seqlen_q;
  a.T = (int)rows;
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
  const int nc = a.B > kThreads || a.T > 2 * kThreads ? kMaxCtas : 1;
  a.per = (a.B + nc - 1) / nc;
  const size_t smem = 4 * (3 * (size_t)a.per + (a.cu && a.B <= kCuMax ? a.B + 1 : 0));
  static std::atomic<uint64_t> done_mask[4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FIA_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask[(dev >> 6) & 3].load() & bit)) {
    if (cudaFuncSetAttribute(assign_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * (3 * (65536 / kMaxCtas) + kCuMax + 1)) != cudaSuccess)
      return FIA_ERR_CUDA;
    done_mask[(dev >> 6) & 3].fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, assign_pages_kernel, a) == cudaSuccess ? FIA_OK : FIA_ERR_CUDA;
}
