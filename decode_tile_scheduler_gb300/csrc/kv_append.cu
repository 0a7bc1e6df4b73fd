// kv_append.cu -- fia_kv_append: the K and V rows of new tokens written to
// their places in a paged or contiguous cache, quantised to E4M3 with one fp32
// scale per 64 elements where the cache is FP8, and the per-key state (weight
// and position) of their slots set.
//
// Row i of a sequence's q_len new rows goes to slot kv_len - q_len + i.  FP8:
// scale = amax / 448 and code = rn(x / scale), both divisions in fp32 as IEEE
// rounds them (the format's definition; a reciprocal would move codes that lie
// near a rounding border).
//
// Memory-bound: every new element is read once and written once.  A thread
// takes 16 bytes of a K row and the same 16 bytes of the V row (bf16), or 16
// elements of each (FP8; the four threads of a 64-element tile share its
// largest magnitude by shuffles), so both loads are in flight together and the
// stores are 16 bytes wide.  20,642 rows of 8 heads of 128 in bf16 (170 MB): 29.5 us,
// 5.8 TB/s, 0.85 of the measured copy rate.
#include <algorithm>

#include "kv_cache.cuh"

namespace fia {

namespace {

struct AppendArgs {
  CacheView c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t k_stride, v_stride;
  const int32_t* cu;       // null: BSND, S rows per sequence
  const int32_t* seqused;
  const int32_t* seen;
  float* weights;
  int32_t* positions;
  int64_t stride;
  int32_t* status;
  int T, S;                // new rows, in all and (BSND) per sequence
};

constexpr float kFp8Max = 448.f;
constexpr float kBf16Max = 3.38953139e38f;  // largest finite bf16 value

// Largest magnitude among the 16 bf16 values of a and b, NaN left out.
__device__ __forceinline__ float amax16(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = fmaxf(m, fabsf(__uint_as_float(w[i] << 16)));
    m = fmaxf(m, fabsf(__uint_as_float(w[i] & 0xffff0000u)));
  }
  return m;
}

__device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, float scale) {
  const float x0 = __fdiv_rn(__uint_as_float(w0 << 16), scale);
  const float x1 = __fdiv_rn(__uint_as_float(w0 & 0xffff0000u), scale);
  const float x2 = __fdiv_rn(__uint_as_float(w1 << 16), scale);
  const float x3 = __fdiv_rn(__uint_as_float(w1 & 0xffff0000u), scale);
  uint32_t r;  // (the first source of a pair lands in its upper byte)
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// The 16 elements of a and b as codes at dst, the tile's scale from its first
// thread (lanes 4k .. 4k + 3 of a warp hold one tile).
__device__ __forceinline__ void store_fp8(uint8_t* dst, float* scale_dst, const uint4& a,
                                          const uint4& b, bool ok, bool first) {
  float m = amax16(a, b);
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = fminf(m, kBf16Max);
  const float scale = m > 0.f ? __fdiv_rn(m, kFp8Max) : 1.f;
  if (!ok) return;
  *reinterpret_cast<uint4*>(dst) = make_uint4(quant4(a.x, a.y, scale), quant4(a.z, a.w, scale),
                                              quant4(b.x, b.y, scale), quant4(b.z, b.w, scale));
  if (first) *scale_dst = scale;
}

template <bool FP8>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
  constexpr int E = FP8 ? 16 : 8;         // elements per thread
  // eight threads are a group, one or two groups a (row, head): one 32-bit
  // division finds a thread's place (64-bit ones made the kernel issue-bound,
  // 72 % of its issue slots at half of the DRAM rate)
  const uint32_t two = a.c.D / E == 16;
  const uint32_t u = blockIdx.x * 32u + threadIdx.x / 8, per_row = (uint32_t)a.c.KVN << two;
  const uint32_t row = u / per_row, in_row = u - row * per_row;
  // (FP8: a tile's four threads are past the end together, and take part in
  // its shuffles)
  const bool inside = row < (uint32_t)a.T;
  const int t = inside ? (int)row : 0;
  const int hk = (int)(in_row >> two);
  const int part = (int)(((in_row & two) << 3) | (threadIdx.x & 7));
  // sequence, and the row's place counted from the sequence's end (negative; else
  // the row is no sequence's, and nothing is done with it)
  int b, back;
  if (a.cu) {
    int lo = 0, hi = a.c.B;  // largest b with cu[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid;
    }
    b = lo;
    back = t >= __ldg(a.cu + b) ? t - __ldg(a.cu + b + 1) : 0;
  } else {
    b = t / a.S;
    back = t - (b + 1) * a.S;
  }
  const int64_t slot = (int64_t)__ldg(a.seqused + b) + back;
  bool ok = inside && back < 0 && slot >= 0 && slot < a.c.cap;
  RowAt r = {0, 0, false};
  if (ok) r = cache_row(a.c, b, hk, (int)slot);
  ok = ok && r.ok;
  if (inside && back < 0 && !ok && part == 0 && a.status) atomicExch(a.status, 3);
  const int64_t src = (int64_t)hk * a.c.D + part * E;
  const uint4* ks = reinterpret_cast<const uint4*>(a.k_new + (int64_t)t * a.k_stride + src);
  const uint4* vs = reinterpret_cast<const uint4*>(a.v_new + (int64_t)t * a.v_stride + src);
  if constexpr (FP8) {
    const uint4 k0 = __ldg(ks), k1 = __ldg(ks + 1), v0 = __ldg(vs), v1 = __ldg(vs + 1);
    const int64_t dst = r.row * a.c.D + part * E;
    const int64_t sc = r.srow * (a.c.D / 64) + part / 4;
    store_fp8(a.c.k + dst, a.c.ks + sc, k0, k1, ok, part % 4 == 0);
    store_fp8(a.c.v + dst, a.c.vs + sc, v0, v1, ok, part % 4 == 0);
  } else {
    const uint4 kw = __ldg(ks), vw = __ldg(vs);
    if (ok) {
      const int64_t dst = 2 * (r.row * a.c.D + part * E);
      *reinterpret_cast<uint4*>(a.c.k + dst) = kw;
      *reinterpret_cast<uint4*>(a.c.v + dst) = vw;
    }
  }
  if (ok && part == 0) {
    const int64_t at = ((int64_t)b * a.c.KVN + hk) * a.stride + slot;
    if (a.weights) a.weights[at] = 0.f;
    if (a.positions)
      a.positions[at] = a.seen ? __ldg(a.seen + b) + back : (int32_t)slot;
  }
}

}  // namespace

}  // namespace fia

extern "C" size_t fia_sizeof_append_params(void) { return sizeof(fia_append_params); }

extern "C" fia_status fia_kv_append(const fia_append_params* p, void* stream) {
  fia::NvtxRange range("fia_kv_append");
  using namespace fia;
  if (!p) return FIA_ERR_NULL_ARG;
  for (int i = 0; i < 8; ++i)
    if (p->reserved[i] != 0) return FIA_ERR_BAD_SHAPE;
  fia_status st = check_cache(p->cache);
  if (st != FIA_OK) return st;
  if (p->layout != FIA_LAYOUT_BSND && p->layout != FIA_LAYOUT_TND) return FIA_ERR_BAD_SHAPE;
  const bool tnd = p->layout == FIA_LAYOUT_TND;
  if (tnd ? p->total_q < 0 : p->seqlen_q < 0 || p->seqlen_q > 20971520) return FIA_ERR_BAD_SHAPE;
  if (tnd && !p->cu_seqlens_q) return FIA_ERR_NULL_ARG;
  const int64_t rows = tnd ? p->total_q : (int64_t)p->cache.batch * p->seqlen_q;
  // (a tensor of no rows has no address)
  if ((rows && (!p->k_new || !p->v_new)) || !p->seqused_kv) return FIA_ERR_NULL_ARG;
  if (!aligned_to(p->k_new, 16) || !aligned_to(p->v_new, 16)) return FIA_ERR_BAD_SHAPE;
  const int64_t nd = (int64_t)p->cache.num_kv_heads * p->cache.head_dim;
  for (const int64_t s : {p->k_token_stride, p->v_token_stride})
    if (s && (s < nd || s % 8)) return FIA_ERR_BAD_SHAPE;
  for (const void* q : {(const void*)p->cu_seqlens_q, (const void*)p->seqused_kv,
                        (const void*)p->tokens_seen, (const void*)p->weights,
                        (const void*)p->positions, (const void*)p->status})
    if (!aligned_to(q, 4)) return FIA_ERR_BAD_SHAPE;
  if ((p->weights || p->positions) && p->state_stride < cache_capacity(p->cache))
    return FIA_ERR_BAD_SHAPE;
  AppendArgs a;
  memset(&a, 0, sizeof a);
  a.c = cache_view(p->cache);
  a.k_new = static_cast<const uint16_t*>(p->k_new);
  a.v_new = static_cast<const uint16_t*>(p->v_new);
  a.k_stride = p->k_token_stride ? p->k_token_stride : nd;
  a.v_stride = p->v_token_stride ? p->v_token_stride : nd;
  a.cu = tnd ? p->cu_seqlens_q : nullptr;
  a.seqused = p->seqused_kv;
  a.seen = p->tokens_seen;
  a.weights = p->weights;
  a.positions = p->positions;
  a.stride = p->state_stride;
  a.status = p->status;
  a.S = p->seqlen_q;
  if (rows == 0) return FIA_OK;
  const int64_t grid = (rows * a.c.KVN * (a.c.D / (a.c.fp8 ? 16 : 8)) + 255) / 256;
  // (the kernel counts rows, and groups of eight threads, in 32 bits)
  if (rows > INT32_MAX || grid >= (1 << 27)) return FIA_ERR_BAD_SHAPE;
  a.T = (int)rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.c.fp8) kv_append_kernel<true><<<(int)grid, 256, 0, s>>>(a);
  else kv_append_kernel<false><<<(int)grid, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FIA_OK : FIA_ERR_CUDA;
}
