// norm_rope.cu -- fia_norm_rope_append: the heads of new queries and keys normed and
// rotated to their positions in one pass, the queries stored, the keys and values
// written to their slots of the cache in its type.
//
// Memory-bound: every element is read once and written once.  A head's D / 8 lanes
// take 16 bytes each; the sum of squares is joined by shuffles, the other value of a
// rotated pair comes from the lane D's half away as the 16 bytes that it loaded.  A warp
// keeps its token, and with it the cosines and sines and both weights, for kHeads
// rounds of heads, whose loads are in flight together.
#include <cmath>

#include "kv_cache.cuh"
#include "kv_quant.cuh"

namespace fia {

namespace {

constexpr int kRounds = 4;  // rounds of heads a warp takes

struct RopeArgs {
  CacheView c;
  int T, QN, rot, P;
  float eps;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride, out_stride;
  uint16_t* out;
  const uint16_t* qw;
  const uint16_t* kw;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* slots;
  int32_t* status;
  int unit;              // rows of a page, or of a contiguous cache's sequence
  int64_t pool;          // rows of the cache
  int groups;            // warps of a token
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                    pack_bf16(y[6], y[7]));
}

// The eight values of a lane to its place in a row of the cache (bf16 caches: `bits`);
// every lane of the warp takes part in the shuffles, those without `ok` store nothing.
template <int D, int F>
__device__ __forceinline__ void store_row(uint8_t* pool, float* scales, int64_t row, int64_t srow,
                                          int chunk, float (&y)[8], const uint4& bits, bool ok) {
  if constexpr (F == 0) {
    if (ok) *reinterpret_cast<uint4*>(pool + 2 * (row * D + 8 * chunk)) = bits;
  } else {
    float m = 0.f;
    int nan = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = fmaxf(m, fabsf(y[i]));  // (a NaN is left out)
      nan |= y[i] != y[i];
    }
#pragma unroll
    for (int o = 1; o < (F == 1 ? 8 : 4); o <<= 1) {  // the lanes of one scale
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (F == 2) nan |= __shfl_xor_sync(0xffffffffu, nan, o);
    }
    if (F == 2 && m > kBf16Max) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(y[i], -kBf16Max), kBf16Max);
    }
    m = fminf(m, kBf16Max);
    if (!ok) return;
    if constexpr (F == 1) {
      const float scale = m > 0.f ? __fdiv_rn(m, kFp8Max) : 1.f;
      *reinterpret_cast<uint2*>(pool + row * D + 8 * chunk) =
          make_uint2(e4m3x4(y[0], y[1], y[2], y[3], scale), e4m3x4(y[4], y[5], y[6], y[7], scale));
      if (chunk % 8 == 0) scales[srow * (D / 64) + chunk / 8] = scale;
    } else {
      const int e = nan ? 255 : mx_scale(m);
      uint32_t codes = 0u;
      if (!nan) codes = e2m1x8(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7], mx_inverse(e));
      *reinterpret_cast<uint32_t*>(pool + (row * D + 8 * chunk) / 2) = codes;
      if (chunk % 4 == 0)
        reinterpret_cast<uint8_t*>(scales)[srow * (D / 32) + chunk / 4] = (uint8_t)e;
    }
  }
}

template <int D, int F, bool PAIRS>
__global__ void __launch_bounds__(256) norm_rope_kernel(const RopeArgs a) {
  constexpr int L = D / 8, H = 32 / L;  // lanes of a head, heads side by side
  const int lane = threadIdx.x & 31, chunk = lane % L;
  const uint32_t w = blockIdx.x * 8u + (threadIdx.x >> 5);
  const uint32_t t = w / (uint32_t)a.groups, grp = w - t * a.groups;
  if (t >= (uint32_t)a.T) return;  // whole warps
  const int KVN = a.c.KVN, heads = a.QN + 2 * KVN;
  const int h0 = (int)grp * (kRounds * H) + lane / L;
  // the heads' loads first
  uint4 x[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int h = h0 + r * H;
    x[r] = make_uint4(0u, 0u, 0u, 0u);
    if (h < heads) {
      const uint16_t* src = h < a.QN ? a.q + t * a.q_stride + (int64_t)h * D
                            : h < a.QN + KVN ? a.k + t * a.k_stride + (int64_t)(h - a.QN) * D
                                             : a.v + t * a.v_stride + (int64_t)(h - a.QN - KVN) * D;
      x[r] = *(reinterpret_cast<const uint4*>(src) + chunk);
    }
  }
  const int position = __ldg(a.positions + t), slot = __ldg(a.slots + t);
  const bool inside = slot >= 0 && slot < a.pool;
  if (position < 0 || (position >= a.P && a.rot > 0)) {
    if (position >= 0 && lane == 0 && a.status) atomicExch(a.status, 3);
    return;
  }
  if (!inside && lane == 0 && a.status) atomicExch(a.status, 3);
  const int page = inside ? slot / a.unit : 0, in_page = inside ? slot - page * a.unit : 0;

  // the rotation of this lane's eight elements: y' = y cos + other * sin, with the sine's
  // sign of the pair's half in it
  const int half = a.rot / 2, e0 = 8 * chunk;
  const bool turned = e0 < a.rot;
  float cs[8], sn[8];
  if (turned) {
    const float* row = a.cos_sin + (int64_t)position * a.rot;
    if constexpr (PAIRS) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + e0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + e0 / 2));
      cs[0] = cs[1] = c4.x; cs[2] = cs[3] = c4.y; cs[4] = cs[5] = c4.z; cs[6] = cs[7] = c4.w;
      sn[0] = -s4.x; sn[1] = s4.x; sn[2] = -s4.y; sn[3] = s4.y;
      sn[4] = -s4.z; sn[5] = s4.z; sn[6] = -s4.w; sn[7] = s4.w;
    } else {
      const bool second = e0 >= half;
      const int i0 = second ? e0 - half : e0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + i0) + i);
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + i0) + i);
        cs[4 * i] = c4.x; cs[4 * i + 1] = c4.y; cs[4 * i + 2] = c4.z; cs[4 * i + 3] = c4.w;
        sn[4 * i] = second ? s4.x : -s4.x; sn[4 * i + 1] = second ? s4.y : -s4.y;
        sn[4 * i + 2] = second ? s4.z : -s4.z; sn[4 * i + 3] = second ? s4.w : -s4.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
  }
  // the lane with the other values of this one's pairs
  const int step = half / 8;
  const int other = PAIRS || !turned ? lane : lane + (e0 >= half ? -step : step);
  const int other_chunk = other % L;

#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int h = h0 + r * H;
    const int kind = h < a.QN ? 0 : h < a.QN + KVN ? 1 : 2;  // query, key, value
    float y[8];
    unpack8(x[r], y);
    uint4 xo = x[r];
    if constexpr (!PAIRS) {
      xo.x = __shfl_sync(0xffffffffu, x[r].x, other);
      xo.y = __shfl_sync(0xffffffffu, x[r].y, other);
      xo.z = __shfl_sync(0xffffffffu, x[r].z, other);
      xo.w = __shfl_sync(0xffffffffu, x[r].w, other);
    }
    float o[8];
    unpack8(xo, o);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
#pragma unroll
    for (int d = 1; d < L; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if (kind < 2) {
      const uint16_t* weight = kind ? a.kw : a.qw;
      if (weight) {
        const float f = 1.f / sqrtf(ss * (1.f / D) + a.eps);
        float wy[8], wo[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(weight) + chunk), wy);
        unpack8(__ldg(reinterpret_cast<const uint4*>(weight) + other_chunk), wo);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = y[i] * f * wy[i];
          o[i] = o[i] * f * wo[i];
        }
      }
      if (turned) {
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = y[i] * cs[i] + (PAIRS ? y[i ^ 1] : o[i]) * sn[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = z[i];
      }
      if (kind == 0 && h < heads)
        *(reinterpret_cast<uint4*>(a.out + t * a.out_stride + (int64_t)h * D) + chunk) = pack8(y);
    }
    const int hk = kind == 2 ? h - a.QN - KVN : h - a.QN;
    const int64_t srow = ((int64_t)page * KVN + hk) * a.unit + in_page;
    const int64_t row = a.c.head_major ? srow : (int64_t)slot * KVN + hk;
    store_row<D, F>(kind == 2 ? a.c.v : a.c.k, kind == 2 ? a.c.vs : a.c.ks, row, srow, chunk, y,
                    kind == 2 ? x[r] : pack8(y), inside && kind > 0 && h < heads);
  }
}

template <int D, int F>
cudaError_t launch_rope(const RopeArgs& a, bool pairs, int grid, cudaStream_t s) {
  if (pairs) norm_rope_kernel<D, F, true><<<grid, 256, 0, s>>>(a);
  else norm_rope_kernel<D, F, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

}  // namespace fia

extern "C" size_t fia_sizeof_norm_rope_params(void) { return sizeof(fia_norm_rope_params); }

extern "C" fia_status fia_norm_rope_append(const fia_norm_rope_params* p, void* stream) {
  fia::NvtxRange range("fia_norm_rope_append");
  using namespace fia;
  if (!p) return FIA_ERR_NULL_ARG;
  for (int i = 0; i < 8; ++i)
    if (p->reserved[i] != 0) return FIA_ERR_BAD_SHAPE;
  fia_status st = check_cache(p->cache);
  if (st != FIA_OK) return st;
  const int D = p->cache.head_dim, KVN = p->cache.num_kv_heads;
  if (p->tokens < 0 || p->num_q_heads < 0 || p->num_q_heads > 256) return FIA_ERR_BAD_SHAPE;
  if (p->rotary_dim < 0 || p->rotary_dim > D || p->rotary_dim % 16) return FIA_ERR_BAD_SHAPE;
  if (p->interleaved != 0 && p->interleaved != 1) return FIA_ERR_BAD_SHAPE;
  if (p->max_positions < 0 || !std::isfinite(p->eps) || p->eps < 0.f) return FIA_ERR_BAD_SHAPE;
  // (tensors of no rows, or no heads, have no address)
  if (p->tokens && (!p->k || !p->v || !p->positions || !p->slots)) return FIA_ERR_NULL_ARG;
  if (p->tokens && p->num_q_heads && (!p->q || !p->q_out)) return FIA_ERR_NULL_ARG;
  if (p->tokens && p->rotary_dim && !p->cos_sin) return FIA_ERR_NULL_ARG;
  for (const void* q : {p->q, p->k, p->v, (const void*)p->q_out, p->q_weight, p->k_weight,
                        (const void*)p->cos_sin})
    if (!aligned_to(q, 16)) return FIA_ERR_BAD_SHAPE;
  for (const void* q : {(const void*)p->positions, (const void*)p->slots, (const void*)p->status})
    if (!aligned_to(q, 4)) return FIA_ERR_BAD_SHAPE;
  const int64_t qd = (int64_t)p->num_q_heads * D, kd = (int64_t)KVN * D;
  RopeArgs a;
  memset(&a, 0, sizeof a);
  a.q_stride = p->q_token_stride ? p->q_token_stride : qd;
  a.k_stride = p->k_token_stride ? p->k_token_stride : kd;
  a.v_stride = p->v_token_stride ? p->v_token_stride : kd;
  a.out_stride = p->q_out_token_stride ? p->q_out_token_stride : qd;
  if (a.q_stride < qd || a.out_stride < qd || a.k_stride < kd || a.v_stride < kd) return FIA_ERR_BAD_SHAPE;
  if (a.q_stride % 8 || a.k_stride % 8 || a.v_stride % 8 || a.out_stride % 8) return FIA_ERR_BAD_SHAPE;
  if (p->q && p->q == p->q_out && a.q_stride != a.out_stride) return FIA_ERR_BAD_SHAPE;
  a.c = cache_view(p->cache);
  a.T = p->tokens;
  a.QN = p->num_q_heads;
  a.rot = p->rotary_dim;
  a.P = p->max_positions;
  a.eps = p->eps;
  a.q = static_cast<const uint16_t*>(p->q);
  a.k = static_cast<const uint16_t*>(p->k);
  a.v = static_cast<const uint16_t*>(p->v);
  a.out = static_cast<uint16_t*>(p->q_out);
  a.qw = static_cast<const uint16_t*>(p->q_weight);
  a.kw = static_cast<const uint16_t*>(p->k_weight);
  a.cos_sin = p->cos_sin;
  a.positions = p->positions;
  a.slots = p->slots;
  a.status = p->status;
  a.unit = a.c.bt ? a.c.bs : a.c.cap;
  a.pool = a.c.bt ? a.c.num_blocks * a.c.bs : (int64_t)a.c.B * a.c.cap;
  if (a.T == 0) return FIA_OK;
  const int per = kRounds * (256 / D);  // heads of a warp
  a.groups = (a.QN + 2 * KVN + per - 1) / per;
  const int64_t grid = ((int64_t)a.T * a.groups + 7) / 8;
  if (grid > INT32_MAX / 8) return FIA_ERR_BAD_SHAPE;  // (warps are counted in 32 bits)
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool pairs = p->interleaved != 0;
  cudaError_t e;
  if (a.c.mx) e = launch_rope<128, 2>(a, pairs, (int)grid, s);
  else if (a.c.fp8) e = launch_rope<128, 1>(a, pairs, (int)grid, s);
  else if (D == 64) e = launch_rope<64, 0>(a, pairs, (int)grid, s);
  else e = launch_rope<128, 0>(a, pairs, (int)grid, s);
  return e == cudaSuccess ? FIA_OK : FIA_ERR_CUDA;
}
