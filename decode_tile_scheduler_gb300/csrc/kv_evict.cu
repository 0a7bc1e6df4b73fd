// kv_evict.cu -- fia_kv_evict: a KV cache cut down to `budget` keys per
// (sequence, KV head).
//
// Which keys stay: each slot's (protected, weight) pair becomes one 32-bit key
// that orders the same way (floats order like their bits once negative ones
// are complemented and the others have their top bit set; a protected key is
// the largest value, a NaN weight 0), and the budget-th largest key T is found
// by radix selection: three histograms of 11, 11 and 10 bits, each over the keys
// that share the digits found so far, ending early where a digit's keys all
// stay.  Keys above T stay, and of those equal to T the lowest slots, as many as
// the budget has left.
//
// Compaction moves what has to move and nothing else: the k-th kept slot at or
// past the budget into the k-th evicted slot below it.  Sources and targets
// are disjoint, so the moves are independent of each other.
//
// One cluster of 1 to 8 CTAs per (sequence, KV head), each a contiguous slice of
// its slots.  A slice's keys are read once into shared memory; a CTA adds the few
// bins of its histogram that are not empty to every peer's joined one, and reads
// the peers' counts, in their shared memory, so the weights travel once and
// nothing but the list of moves passes through global memory.
//
// Bound by latency: a short chain of passes over shared memory between one read of
// the weights and positions and one copy of the moved rows.  256 heads of 2049 to
// 2176 keys cut to 2048: 16.4 us (length and weights 4.9, selection 2.3, ranks 2.1,
// moves 4.2 of them, 81 rows a head); 32 FP8 heads of 8 to 32 k keys 24.7 us, 1880
// rows a head.
#include <algorithm>
#include <atomic>

#include "cluster.cuh"
#include "kv_cache.cuh"

namespace fia {

namespace {

struct EvictArgs {
  CacheView c;
  const int32_t* seqused;
  int32_t* seqused_out;
  const int32_t* seen;
  const float* w_in;
  float* w_out;
  const int32_t* p_in;
  int32_t* p_out;
  int64_t stride;
  int budget, first, recent;
  int32_t* status;
  int2* moves;         // [B * KVN][max_moves] (hole, tail)
  int max_moves;
};

__device__ __forceinline__ uint32_t order_key(float w, int pos, int first, int64_t newest) {
  if (pos < first || pos >= newest) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // (-0 becomes 0)
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kRanked = kThreads;  // keys with one first digit ranked directly, at most
constexpr int kListedMax = 2048;   // moves listed in shared memory, at most
constexpr int kStagedMax = 40 * 1024;  // keys of a slice kept in shared memory, at most
constexpr int kPages = 2 * kThreads;   // table entries kept in shared memory, at most
constexpr int kInFlight = 4;           // rows of a lane in flight

// The cluster's barrier in two halves; alone, the CTA's.
template <int CS>
__device__ __forceinline__ void cluster_arrive() {
  if constexpr (CS > 1) cluster_bar_arrive();
}
template <int CS>
__device__ __forceinline__ void cluster_wait() {
  if constexpr (CS == 1)
    __syncthreads();
  else
    cluster_bar_wait();
}
template <int CS>
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive<CS>();
  cluster_wait<CS>();
}
__device__ __forceinline__ void peer_add(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v)
               : "memory");
}
// Sum of x over the block's threads before this one (exclusive), `total` over
// all; two barriers.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[wid] = incl;
  __syncthreads();
  uint32_t v = lane < kWarps ? warp_sums[lane] : 0u;
  uint32_t before = lane < wid ? v : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  __syncthreads();
  *total = v;
  return before + incl - x;
}

template <int CS>
__global__ void __launch_bounds__(kThreads, 2) kv_evict_kernel(const EvictArgs a, int staged,
                                                                int listed) {
  extern __shared__ uint32_t skey[];  // the slice's keys, with `staged` places
  int2* slist = reinterpret_cast<int2*>(skey + staged);  // CS = 1: the moves, with `listed` places
  __shared__ int32_t pages[kPages];  // the sequence's first table entries
  // this CTA's histogram of a pass, and each pass's over the cluster (alone: its own)
  __shared__ __align__(16) uint32_t mine_h[CS > 1 ? kBins : 4];
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ uint32_t warp_sums[kWarps], found[3];
  __shared__ int totals[3];   // of this CTA: keys at the threshold, kept keys, kept below the budget
  __shared__ int warp_cnt[3][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = CS == 1 ? 0u : cluster_rank();
  const int pair = blockIdx.x / CS, b = pair / a.c.KVN, hk = pair - b * a.c.KVN;
  const float* w = a.w_in + pair * a.stride;
  const int32_t* pin = a.p_in ? a.p_in + pair * a.stride : nullptr;
  // everything whose place does not depend on the length is fetched beside it (the
  // weights of slots behind the length among them: rows have the capacity's places)
  const int n_raw = __ldg(a.seqused + b), seen_raw = a.seen ? __ldg(a.seen + b) : 0;
  const int32_t* table = a.c.bt ? a.c.bt + (int64_t)b * a.c.max_blocks : nullptr;
  const int npages = table ? min(a.c.max_blocks, kPages) : 0;
  int32_t page[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    page[i] = tid + i * kThreads < npages ? __ldg(table + tid + i * kThreads) : 0;
  constexpr int U = 4;  // loads in flight
  float wv[U];
  int pv[U];
  auto fetch = [&](int j0, int end) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kThreads;
      wv[u] = j < end ? w[j] : 0.f;
      pv[u] = j < end && pin ? pin[j] : j;
    }
  };
  if (CS == 1) fetch(tid, a.c.cap);
  const int n = min(max(n_raw, 0), a.c.cap);
  const int m = min(n, a.budget);
  if (hk == 0 && rank == 0 && tid == 0) a.seqused_out[b] = m;
  float* wo = a.w_out + pair * a.stride;
  int32_t* po = a.p_out ? a.p_out + pair * a.stride : nullptr;
  const int slice = ((n + CS - 1) / CS + 31) & ~31;  // n <= 20M: no overflow
  const int lo = min(n, (int)rank * slice), hi = min(n, lo + slice);
  if (n <= a.budget) {  // (the whole cluster leaves)
    for (int j = lo + tid; j < hi; j += kThreads) {
      if (wo != w) wo[j] = w[j];
      if (po && po != pin) po[j] = pin ? pin[j] : j;
    }
    return;
  }
  if (CS > 1) fetch(lo + tid, hi);
  const int64_t newest = (int64_t)(a.seen ? seen_raw : n) - a.recent;
  auto key_at = [&](int j) { return order_key(w[j], pin ? pin[j] : j, a.first, newest); };
  const bool in_smem = slice <= staged;
  auto key_of = [&](int j) { return in_smem ? skey[j - lo] : key_at(j); };

  // ---- the budget-th largest key ----
  for (int i = tid; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = 0u;
  if (CS > 1)
    for (int i = tid; i < kBins; i += kThreads) mine_h[i] = 0u;
  if (tid == 0) totals[0] = 0;
  __syncthreads();
  cluster_arrive<CS>();  // (peers may add to the joined histograms once all are clear)
  uint32_t prefix = 0, known = 0, left = (uint32_t)a.budget;
  bool ties = true;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    uint32_t* h0 = CS > 1 ? mine_h : hist[pass];
    auto count = [&](uint32_t k, bool mine) {
      // protected keys fall into one bin: one count per warp
      const uint32_t safe = __ballot_sync(0xffffffffu, mine && k == 0xffffffffu);
      if (mine && k != 0xffffffffu) atomicAdd(&h0[(k >> shift) & digits], 1u);
      if (safe && lane == 0) atomicAdd(&h0[digits], (uint32_t)__popc(safe));
    };
    const int end = lo + ((hi - lo + 31) & ~31);  // (whole warps)
    if (pass == 0) {
      for (int j0 = lo + tid; j0 < end; j0 += U * kThreads) {
        if (j0 != lo + tid) fetch(j0, hi);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * kThreads;
          const uint32_t k = order_key(wv[u], pv[u], a.first, newest);
          if (j < hi && in_smem) skey[j - lo] = k;
          // every slot below the new length starts with its own values; those
          // of the holes are overwritten by the moves, after the last barrier
          if (j < min(hi, m)) {
            if (wo != w) wo[j] = wv[u];
            if (po && po != pin) po[j] = pv[u];
          }
          count(k, j < hi);  // (past `end` for a whole warp: nothing)
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (tid + i * kThreads < npages) pages[tid + i * kThreads] = page[i];
    } else {
      for (int j = lo + tid; j < end; j += kThreads) {
        const uint32_t k = j < hi ? key_of(j) : 0u;
        count(k, j < hi && (k & known) == prefix);
      }
    }
    __syncthreads();
    // bins in falling order, four to a thread
    const int top = kBins - 4 - 4 * tid;
    if constexpr (CS > 1) {
      const uint4 x = *reinterpret_cast<const uint4*>(&mine_h[top]);
      *reinterpret_cast<uint4*>(&mine_h[top]) = make_uint4(0u, 0u, 0u, 0u);
      if (pass == 0) cluster_wait<CS>();
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (xs[i]) {
#pragma unroll
          for (int r = 0; r < CS; ++r) peer_add(peer_addr(&hist[pass][top + i], r), xs[i]);
        }
      cluster_sync<CS>();
    }
    const uint4 h = *reinterpret_cast<const uint4*>(&hist[pass][top]);
    uint32_t total;
    uint32_t above = block_scan(h.x + h.y + h.z + h.w, warp_sums, &total);
    const uint32_t c[4] = {h.w, h.z, h.y, h.x};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < left && left <= above + c[i]) {
        found[0] = (uint32_t)(top + 3 - i);
        found[1] = left - above;
        found[2] = c[i];
      }
      above += c[i];
    }
    __syncthreads();
    prefix |= found[0] << shift;
    known |= digits << shift;
    left = found[1];
    ties = left != found[2];
    if (!ties) break;  // every key with these digits stays
    if (CS == 1 && pass == 0 && in_smem && found[2] <= kRanked && found[0] != digits) {
      // few keys share the first digit: rank them among themselves, each by a
      // thread, instead of two more passes and a count of ties (the newest keys
      // often have equal weights, of no query yet).  Those that stay become the
      // largest key, the others the smallest.
      const int few = (int)found[2];
      uint2* cand = reinterpret_cast<uint2*>(&hist[1][0]);
      for (int j = lo + tid; j < hi; j += kThreads) {
        const uint32_t k = skey[j - lo];
        if ((k & known) == prefix) cand[atomicAdd(&totals[0], 1)] = make_uint2(k, (uint32_t)j);
      }
      __syncthreads();
      if (tid < few) {
        const uint2 mine = cand[tid];
        uint32_t better = 0;
#pragma unroll 8
        for (int i = 0; i < few; ++i) {
          const uint2 o = cand[i];
          better += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
        }
        skey[(int)mine.y - lo] = better < left ? 0xffffffffu : 0u;
      }
      __syncthreads();
      prefix += 1u << shift;
      ties = false;
      break;
    }
  }
  // (with ties the threshold is a whole key, and `left` of its keys stay)

  // ---- ranks in slot order: each warp a contiguous part of the slice ----
  const int part = (((hi - lo) + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = min(hi, lo + wid * part), w1 = min(hi, w0 + part);
  int eq_base = 0;
  if (ties) {
    int c = 0;
    for (int j0 = w0; j0 < w1; j0 += 32) {
      const int j = j0 + lane;
      c += __popc(__ballot_sync(0xffffffffu, j < w1 && key_of(j) == prefix));
    }
    if (lane == 0) warp_cnt[0][wid] = c;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int x = warp_cnt[0][i];
      before += i < wid ? x : 0;
      all += x;
    }
    if (CS > 1) {
      if (tid == 0) totals[0] = all;
      cluster_sync<CS>();
      for (int r = 0; r < (int)rank; ++r) before += peer_load(peer_addr(&totals[0], r));
    }
    eq_base = before;
  }
  // whether the key of lane's slot stays; `eq` runs over the warp's part
  auto keeps = [&](int j, int& eq) {
    const uint32_t k = j < w1 ? key_of(j) : 0u;
    const uint32_t d = k & known;
    if (!ties) return j < w1 && d >= prefix;
    const bool is = j < w1 && d == prefix;
    const uint32_t me = __ballot_sync(0xffffffffu, is);
    const bool stay = j < w1 && (d > prefix || (is && eq + __popc(me & ((1u << lane) - 1)) < (int)left));
    eq += __popc(me);
    return stay;
  };
  {
    int kept = 0, low = 0, eq = eq_base;
    for (int j0 = w0; j0 < w1; j0 += 32) {
      const int j = j0 + lane;
      const bool stay = keeps(j, eq);
      kept += __popc(__ballot_sync(0xffffffffu, stay));
      low += __popc(__ballot_sync(0xffffffffu, stay && j < m));
    }
    if (lane == 0) warp_cnt[1][wid] = kept, warp_cnt[2][wid] = low;
    __syncthreads();
  }
  int kept = 0, low = 0;  // kept before this warp's part; kept below the budget, in all
  {
    int all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int x = warp_cnt[1][i];
      kept += i < wid ? x : 0;
      all += x;
      low += warp_cnt[2][i];
    }
    if (CS > 1) {
      if (tid == 0) totals[1] = all, totals[2] = low;
      cluster_sync<CS>();
      low = 0;
      for (int r = 0; r < CS; ++r) {
        if (r < (int)rank) kept += peer_load(peer_addr(&totals[1], r));
        low += peer_load(peer_addr(&totals[2], r));
      }
    }
  }
  const int moves = min(m - low, a.max_moves);
  // a hole's rank is its slot less the kept slots before it, a tail's the kept
  // slots before it less those below the budget
  const bool in_list = CS == 1 && listed > 0;
  int2* mv = in_list ? slist : a.moves + (int64_t)pair * a.max_moves;
  {
    int eq = eq_base;
    for (int j0 = w0; j0 < w1; j0 += 32) {
      const int j = j0 + lane;
      const bool stay = keeps(j, eq);
      const uint32_t mk = __ballot_sync(0xffffffffu, stay);
      const int before = kept + __popc(mk & ((1u << lane) - 1));
      if (j < w1) {
        if (j < m && !stay && j - before < a.max_moves) mv[j - before].x = j;
        if (j >= m && stay && before - low < a.max_moves) mv[before - low].y = j;
      }
      kept += __popc(mk);
    }
  }
  cluster_sync<CS>();

  // ---- the moves ----
  // A warp takes up to 32 at a time.  Each lane finds the rows of one move and
  // makes its small copies (weight, position, scales); then the warp copies the
  // rows, 16 bytes of K or V per lane, kInFlight moves in flight.  (With every lane
  // finding the rows of every move the address arithmetic bound the phase.)
  // 16-byte pieces of a K row: 16 or 8 (bf16), 8 (FP8), 4 (MXFP4)
  const int row_pieces = a.c.D * (a.c.mx ? 1 : a.c.fp8 ? 2 : 4) / 32;
  const int per = 16 / row_pieces;           // moves a warp makes side by side: 1, 2, 4
  const int grp = lane / (2 * row_pieces), x = lane % (2 * row_pieces);
  uint4* pool = reinterpret_cast<uint4*>(x >= row_pieces ? a.c.v : a.c.k) + x % row_pieces;
  auto row_of = [&](int j) {
    if (!table) return cache_row(a.c, b, hk, j);
    const int pg = cache_page(a.c, j);
    return page_row(a.c, hk, j, pg, pg < kPages ? pages[pg] : __ldg(table + pg));
  };
  constexpr int kAll = CS * kWarps;  // warps of the cluster
  for (int i0 = (int)rank * kWarps + wid; i0 < moves; i0 += 32 * kAll) {
    const int i = i0 + lane * kAll;
    int2 ht = make_int2(0, 0);
    if (i < moves) ht = in_list ? slist[i] : __ldcg(mv + i);
    int64_t to = 0, from = 0;  // rows, in pieces
    bool ok = false;
    float weight = 0.f;
    int position = 0;
    float2 ks = make_float2(0.f, 0.f), vs = ks;
    int64_t scale_to = 0;
    if (i < moves) {
      const RowAt t = row_of(ht.x), f = row_of(ht.y);
      ok = t.ok && f.ok;
      to = t.row * row_pieces;
      from = f.row * row_pieces;
      weight = w[ht.y];
      if (po) position = pin ? pin[ht.y] : ht.y;
      scale_to = t.srow;
      if (a.c.fp8 && ok) {  // (D = 128: two scales a row)
        ks = reinterpret_cast<const float2*>(a.c.ks)[f.srow];
        vs = reinterpret_cast<const float2*>(a.c.vs)[f.srow];
      } else if (a.c.mx && ok) {  // (four bytes)
        ks.x = a.c.ks[f.srow];
        vs.x = a.c.vs[f.srow];
      }
    }
    const uint32_t fine = __ballot_sync(0xffffffffu, ok);
    for (int c0 = 0; c0 < 32 && i0 + c0 * kAll < moves; c0 += kInFlight * per) {
      uint4 v[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int c = c0 + u * per + grp;
        const int64_t at = __shfl_sync(0xffffffffu, from, c);
        if ((fine >> c) & 1u) v[u] = pool[at];
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int c = c0 + u * per + grp;
        const int64_t at = __shfl_sync(0xffffffffu, to, c);
        if ((fine >> c) & 1u) pool[at] = v[u];
      }
    }
    if (i < moves) {
      wo[ht.x] = weight;
      if (po) po[ht.x] = position;
      if (a.c.fp8 && ok) {
        reinterpret_cast<float2*>(a.c.ks)[scale_to] = ks;
        reinterpret_cast<float2*>(a.c.vs)[scale_to] = vs;
      } else if (a.c.mx && ok) {
        a.c.ks[scale_to] = ks.x;
        a.c.vs[scale_to] = vs.x;
      }
      if (!ok && a.status) atomicExch(a.status, 3);
    }
  }
}

template <int CS>
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  auto kern = kv_evict_kernel<CS>;
  const int slice = (((a.c.cap + CS - 1) / CS) + 31) & ~31;
  const int staged = slice <= kStagedMax ? slice : 0;
  const int listed = CS == 1 && a.max_moves <= kListedMax ? a.max_moves : 0;
  static std::atomic<uint64_t> done_mask[4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask[(dev >> 6) & 3].load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * kStagedMax + 8 * kListedMax);
    if (e != cudaSuccess) return e;
    done_mask[(dev >> 6) & 3].fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.c.B * a.c.KVN * CS);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 4 * (size_t)staged + 8 * (size_t)listed;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CS;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, staged, listed);
}

// At most min(budget, capacity - budget) keys of a head move.
int64_t max_moves_of(const fia_evict_params* p) {
  return std::max<int64_t>(1, std::min<int64_t>(p->budget, cache_capacity(p->cache) - p->budget));
}

fia_status check_evict(const fia_evict_params* p) {
  if (!p) return FIA_ERR_NULL_ARG;
  for (int i = 0; i < 8; ++i)
    if (p->reserved[i] != 0) return FIA_ERR_BAD_SHAPE;
  fia_status st = check_cache(p->cache);
  if (st != FIA_OK) return st;
  if (!p->seqused_kv || !p->seqused_out || !p->weights_in || !p->weights_out)
    return FIA_ERR_NULL_ARG;
  if (p->positions_in && !p->positions_out) return FIA_ERR_NULL_ARG;
  if (p->seqused_out == p->seqused_kv) return FIA_ERR_BAD_SHAPE;
  for (const void* q : {(const void*)p->seqused_kv, (const void*)p->seqused_out,
                        (const void*)p->tokens_seen, (const void*)p->weights_in,
                        (const void*)p->weights_out, (const void*)p->positions_in,
                        (const void*)p->positions_out, (const void*)p->status})
    if (!aligned_to(q, 4)) return FIA_ERR_BAD_SHAPE;
  const int64_t cap = cache_capacity(p->cache);
  if (p->state_stride < cap) return FIA_ERR_BAD_SHAPE;
  const int64_t rows = (int64_t)p->cache.batch * p->cache.num_kv_heads;
  if (rows_overlap(p->weights_in, p->weights_out, rows, p->state_stride, cap) ||
      rows_overlap(p->positions_in, p->positions_out, rows, p->state_stride, cap) ||
      rows_overlap(p->seqused_kv, p->seqused_out, 1, p->cache.batch, p->cache.batch))
    return FIA_ERR_BAD_SHAPE;
  if (p->budget < 1 || p->budget > cap) return FIA_ERR_BAD_SHAPE;
  if (p->first_tokens < 0 || p->recent_tokens < 0 ||
      (int64_t)p->first_tokens + p->recent_tokens > p->budget)
    return FIA_ERR_BAD_SHAPE;
  return FIA_OK;
}

}  // namespace

}  // namespace fia

extern "C" size_t fia_sizeof_evict_params(void) { return sizeof(fia_evict_params); }

extern "C" fia_status fia_get_evict_workspace_size(const fia_evict_params* p, size_t* bytes) {
  if (!bytes) return FIA_ERR_NULL_ARG;
  const fia_status st = fia::check_evict(p);
  if (st != FIA_OK) return st;
  *bytes = (size_t)(sizeof(int2) * p->cache.batch * p->cache.num_kv_heads *
                    fia::max_moves_of(p));
  return FIA_OK;
}

extern "C" fia_status fia_kv_evict(const fia_evict_params* p, void* ws, size_t ws_bytes,
                                   void* stream) {
  fia::NvtxRange range("fia_kv_evict");
  using namespace fia;
  size_t need;
  const fia_status st = fia_get_evict_workspace_size(p, &need);
  if (st != FIA_OK) return st;
  if (!ws || ws_bytes < need) return FIA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned_to(ws, 8)) return FIA_ERR_BAD_SHAPE;
  EvictArgs a;
  memset(&a, 0, sizeof a);
  a.c = cache_view(p->cache);
  a.seqused = p->seqused_kv;
  a.seqused_out = p->seqused_out;
  a.seen = p->tokens_seen;
  a.w_in = p->weights_in;
  a.w_out = p->weights_out;
  a.p_in = p->positions_in;
  a.p_out = p->positions_out;
  a.stride = p->state_stride;
  a.budget = p->budget;
  a.first = p->first_tokens;
  a.recent = p->recent_tokens;
  a.status = p->status;
  a.moves = static_cast<int2*>(ws);
  a.max_moves = (int)max_moves_of(p);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FIA_ERR_CUDA;
  // CTAs per head: while they have a few thousand slots each, as many as run at
  // once (two to an SM)
  const int64_t pairs = (int64_t)a.c.B * a.c.KVN;
  int cs = 8;
  while (cs > 1 && (pairs * cs > 2 * sms || a.c.cap < 2048 * cs)) cs /= 2;
  const cudaError_t e = cs == 8   ? launch_evict<8>(a, s)
                        : cs == 4 ? launch_evict<4>(a, s)
                        : cs == 2 ? launch_evict<2>(a, s)
                                  : launch_evict<1>(a, s);
  return e == cudaSuccess ? FIA_OK : FIA_ERR_CUDA;
}
