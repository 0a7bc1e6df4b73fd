// kv_evict.cu -- fia_kv_evict: a KV cache cut down to `budget` keys per
// (sequence, KV head).
//
// Which keys stay: each slot's (protected, weight) pair becomes one 32-bit key
// that orders the same way (floats order like their bits once negative ones
// are complemented and the others have their top bit set; a protected key is
// the largest value, a NaN weight 0), and the budget-th largest key T is found
// by radix selection, a histogram of the next digit over the keys that share
// the digits found so far.  Keys above T stay, and of those equal to T the
// lowest slots, as many as the budget has left.
//
// Compaction moves what has to move and nothing else: the k-th kept slot at or
// past the budget into the k-th evicted slot below it.  Sources and targets
// are disjoint, so the moves are independent of each other.
#include <algorithm>

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

constexpr int kThreads = 1024;

__global__ void __launch_bounds__(kThreads) kv_evict_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_digit, s_left;
  __shared__ int s_sum[3][32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int pair = blockIdx.x, b = pair / a.c.KVN, hk = pair - b * a.c.KVN;
  const int n = min(max(__ldg(a.seqused + b), 0), a.c.cap);
  const int m = min(n, a.budget);
  if (hk == 0 && tid == 0) a.seqused_out[b] = m;
  const float* w = a.w_in + pair * a.stride;
  const int32_t* pin = a.p_in ? a.p_in + pair * a.stride : nullptr;
  float* wo = a.w_out + pair * a.stride;
  int32_t* po = a.p_out ? a.p_out + pair * a.stride : nullptr;
  if (n <= a.budget) {
    for (int j = tid; j < n; j += kThreads) {
      if (wo != w) wo[j] = w[j];
      if (po && po != pin) po[j] = pin ? pin[j] : j;
    }
    return;
  }
  const int64_t newest = (int64_t)(a.seen ? __ldg(a.seen + b) : n) - a.recent;
  auto key_of = [&](int j) { return order_key(w[j], pin ? pin[j] : j, a.first, newest); };
  // the budget-th largest key
  uint32_t prefix = 0, left = (uint32_t)a.budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t known = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = tid; j < n; j += kThreads) {
      const uint32_t k = key_of(j);
      if ((k & known) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t l = left;
      int d = 255;
      for (; d > 0 && hist[d] < l; --d) l -= hist[d];
      s_digit = (uint32_t)d;
      s_left = l;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    left = s_left;
  }
  // in slot order: which keys equal to the threshold stay, then the holes and
  // tails and their ranks
  int2* mv = a.moves + (int64_t)pair * a.max_moves;
  int eq_before = 0, holes = 0, tails = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int j = base + tid;
    const uint32_t k = j < n ? key_of(j) : 0u;
    const bool eq = j < n && k == prefix;
    const uint32_t me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_sum[0][wid] = __popc(me);
    __syncthreads();
    int eq_rank = eq_before + __popc(me & ((1u << lane) - 1));
    for (int i = 0; i < 32; ++i) {
      if (i < wid) eq_rank += s_sum[0][i];
      eq_before += s_sum[0][i];
    }
    const bool keep = j < n && (k > prefix || (eq && eq_rank < (int)left));
    const bool hole = j < m && !keep, tail = j >= m && keep;
    const uint32_t mh = __ballot_sync(0xffffffffu, hole), mt = __ballot_sync(0xffffffffu, tail);
    if (lane == 0) s_sum[1][wid] = __popc(mh), s_sum[2][wid] = __popc(mt);
    __syncthreads();
    int rh = holes + __popc(mh & ((1u << lane) - 1)), rt = tails + __popc(mt & ((1u << lane) - 1));
    for (int i = 0; i < 32; ++i) {
      if (i < wid) rh += s_sum[1][i], rt += s_sum[2][i];
      holes += s_sum[1][i];
      tails += s_sum[2][i];
    }
    if (hole && rh < a.max_moves) mv[rh].x = j;
    if (tail && rt < a.max_moves) mv[rt].y = j;
    if (keep && j < m) {
      if (wo != w) wo[j] = w[j];
      if (po && po != pin) po[j] = pin ? pin[j] : j;
    }
    __syncthreads();
  }
  // the moves (holes == tails)
  const int es = a.c.fp8 ? 1 : 2;
  const int pieces = a.c.D * es / 16;
  for (int64_t x = tid; x < (int64_t)holes * pieces; x += kThreads) {
    const int i = (int)(x / pieces), pc = (int)(x % pieces);
    const int2 ht = mv[i];
    const RowAt to = cache_row(a.c, b, hk, ht.x), of = cache_row(a.c, b, hk, ht.y);
    if (pc == 0) {
      wo[ht.x] = w[ht.y];
      if (po) po[ht.x] = pin ? pin[ht.y] : ht.y;
    }
    if (!to.ok || !of.ok) {
      if (a.status) atomicExch(a.status, 3);
      continue;
    }
    const int64_t t0 = to.row * a.c.D * es + pc * 16, f0 = of.row * a.c.D * es + pc * 16;
    *reinterpret_cast<uint4*>(a.c.k + t0) = *reinterpret_cast<const uint4*>(a.c.k + f0);
    *reinterpret_cast<uint4*>(a.c.v + t0) = *reinterpret_cast<const uint4*>(a.c.v + f0);
    if (a.c.fp8 && pc < a.c.D / 64) {
      const int nt = a.c.D / 64;
      a.c.ks[to.srow * nt + pc] = a.c.ks[of.srow * nt + pc];
      a.c.vs[to.srow * nt + pc] = a.c.vs[of.srow * nt + pc];
    }
  }
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
  kv_evict_kernel<<<a.c.B * a.c.KVN, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FIA_OK : FIA_ERR_CUDA;
}
