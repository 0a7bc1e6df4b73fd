// norm_rope.cu -- fia_norm_rope_append: the heads of new queries and keys normed and
// rotated to their positions in one pass, the queries stored, the keys and values
// written to their slots of the cache in its type.
//
// Memory-bound: every element is read once and written once.  A head's D / 8 lanes
// take 16 bytes each; the sum of squares is joined by shuffles, the other value of a
// rotated pair comes from the lane D's half away as the 16 bytes that it loaded.  A warp
// keeps its token and one kind of head (query, key, value) for kRounds rounds of heads,
// whose loads are in flight together: weights times cosines and weights times sines are
// made once for all of them, which leaves an element a product, a product and sum, and
// the head's factor, in packed pairs of fp32.
//
// Measured: 8 prompts of 256 to 4096 tokens, 32 + 8 + 8 heads (375 MB) 70.2 us, 5.3 TB/s,
// 0.79 of the measured copy rate; 4 of 256 to 2048 with 64 query heads into an FP8 cache
// (122 MB) 29.1 us; 32 tokens 4.1 us, a launch.  Four rounds in blocks of 128 threads, at
// least eight to an SM: blocks of 256 threads 73.5 us, of 64 71.6; with five or six blocks
// of 256 to an SM for fewer registers 79.5 and 90.3; eight rounds 80, two 96.
#include <cmath>

#include "kv_cache.cuh"
#include "kv_quant.cuh"

namespace fia {

namespace {

constexpr int kRounds = 4, kThreads = 128;  // rounds of heads a warp takes; of a block

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
  int q_groups, kv_groups, groups;  // warps of a token's queries, of its keys (values), in all
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
// Pairs of fp32 in one instruction.
union Pair {
  float f[2];
  unsigned long long u;
};
__device__ __forceinline__ Pair pair_of(uint32_t w) {  // two bf16
  Pair p;
  p.f[0] = __uint_as_float(w << 16);
  p.f[1] = __uint_as_float(w & 0xffff0000u);
  return p;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return d;
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
__global__ void __launch_bounds__(kThreads, 8) norm_rope_kernel(const RopeArgs a) {
  constexpr int L = D / 8, H = 32 / L;  // lanes of a head, heads side by side
  const int lane = threadIdx.x & 31, chunk = lane % L;
  const uint32_t w = blockIdx.x * (kThreads / 32u) + (threadIdx.x >> 5);
  const uint32_t t = w / (uint32_t)a.groups;
  int grp = (int)(w - t * a.groups);
  if (t >= (uint32_t)a.T) return;  // whole warps
  // the warp's kind of head, and its first one
  const int KVN = a.c.KVN;
  const int kind = grp < a.q_groups ? 0 : grp < a.q_groups + a.kv_groups ? 1 : 2;
  const int heads = kind == 0 ? a.QN : KVN;
  grp -= kind == 0 ? 0 : a.q_groups + (kind - 1) * a.kv_groups;
  const int h0 = grp * (kRounds * H) + lane / L;
  const uint16_t* src = kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
  src += (int64_t)h0 * D + 8 * chunk;
  uint4 x[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    x[r] = make_uint4(0u, 0u, 0u, 0u);
    if (h0 + r * H < heads) x[r] = *reinterpret_cast<const uint4*>(src + r * H * D);
  }
  const int position = __ldg(a.positions + t), slot = __ldg(a.slots + t);
  if (position < 0 || (position >= a.P && a.rot > 0)) {
    if (position >= 0 && lane == 0 && a.status) atomicExch(a.status, 3);
    return;
  }
  const bool inside = slot >= 0 && slot < a.pool;
  if (!inside && lane == 0 && a.status) atomicExch(a.status, 3);
  // the place of KV head 0's row in the cache, and from head to head
  int64_t row = 0, srow = 0;
  int step = 0, sstep = 0;
  if (kind > 0 && inside) {
    const int page = slot / a.unit, in_page = slot - page * a.unit;
    srow = (int64_t)page * KVN * a.unit + in_page;
    sstep = a.unit;
    row = a.c.head_major ? srow : (int64_t)slot * KVN;
    step = a.c.head_major ? a.unit : 1;
  }
  if (kind == 2) {  // values: as they are
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int h = h0 + r * H;
      float y[8];
      unpack8(x[r], y);
      store_row<D, F>(a.c.v, a.c.vs, row + (int64_t)h * step, srow + (int64_t)h * sstep, chunk, y, x[r],
                      inside && h < heads);
    }
    return;
  }

  // What this lane's eight elements are multiplied by, their own values and the others of
  // their pairs (the sine with the sign of the pair's half), both with the norm's weights.
  const int half = a.rot / 2, e0 = 8 * chunk;
  const bool turned = e0 < a.rot, second = e0 >= half;
  // the lane with the other values of this one's pairs
  const int other = PAIRS || !turned ? lane : lane + (second ? -half / 8 : half / 8);
  const uint16_t* weight = kind ? a.kw : a.qw;
  Pair own[4], oth[4];
  {
    uint4 wy = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), wo = wy;  // ones
    if (weight) {
      wy = __ldg(reinterpret_cast<const uint4*>(weight) + chunk);
      wo = __ldg(reinterpret_cast<const uint4*>(weight) + other % L);
    }
    const uint32_t y4[4] = {wy.x, wy.y, wy.z, wy.w}, o4[4] = {wo.x, wo.y, wo.z, wo.w};
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
    if (turned) {
      const float* table = a.cos_sin + (int64_t)position * a.rot;
      if constexpr (PAIRS) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(table + e0 / 2));
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(table + half + e0 / 2));
        cs[0] = cs[1] = c4.x; cs[2] = cs[3] = c4.y; cs[4] = cs[5] = c4.z; cs[6] = cs[7] = c4.w;
        sn[0] = -s4.x; sn[1] = s4.x; sn[2] = -s4.y; sn[3] = s4.y;
        sn[4] = -s4.z; sn[5] = s4.z; sn[6] = -s4.w; sn[7] = s4.w;
      } else {
        const int i0 = second ? e0 - half : e0;
        const float sign = second ? 1.f : -1.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 c4 = __ldg(reinterpret_cast<const float4*>(table + i0) + i);
          const float4 s4 = __ldg(reinterpret_cast<const float4*>(table + half + i0) + i);
          cs[4 * i] = c4.x; cs[4 * i + 1] = c4.y; cs[4 * i + 2] = c4.z; cs[4 * i + 3] = c4.w;
          sn[4 * i] = sign * s4.x; sn[4 * i + 1] = sign * s4.y;
          sn[4 * i + 2] = sign * s4.z; sn[4 * i + 3] = sign * s4.w;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Pair py = pair_of(y4[i]), po = PAIRS ? py : pair_of(o4[i]);
      own[i].f[0] = py.f[0] * cs[2 * i];
      own[i].f[1] = py.f[1] * cs[2 * i + 1];
      oth[i].f[0] = po.f[PAIRS ? 1 : 0] * sn[2 * i];
      oth[i].f[1] = po.f[PAIRS ? 0 : 1] * sn[2 * i + 1];
    }
  }

#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int h = h0 + r * H;
    const uint32_t xw[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
    Pair y[4], z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = pair_of(xw[i]);
    float f = 1.f;
    if (weight) {
      Pair ss = mul2(y[0], y[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) ss = fma2(y[i], y[i], ss);
      float s = ss.f[0] + ss.f[1];
#pragma unroll
      for (int d = 1; d < L; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      f = rsqrtf(s * (1.f / D) + a.eps);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Pair o;
      if constexpr (PAIRS) {
        o.f[0] = y[i].f[1];
        o.f[1] = y[i].f[0];
      } else {
        o = pair_of(__shfl_sync(0xffffffffu, xw[i], other));
      }
      if (!turned) o.u = 0;  // (an infinite value is no NaN of it)
      z[i] = fma2(o, oth[i], mul2(y[i], own[i]));
      if (weight) {
        const Pair ff = {{f, f}};
        z[i] = mul2(z[i], ff);
      }
    }
    float v[8] = {z[0].f[0], z[0].f[1], z[1].f[0], z[1].f[1], z[2].f[0], z[2].f[1], z[3].f[0], z[3].f[1]};
    if (kind == 0) {
      if (h < heads)
        *(reinterpret_cast<uint4*>(a.out + t * a.out_stride + (int64_t)h * D) + chunk) = pack8(v);
    } else {
      store_row<D, F>(a.c.k, a.c.ks, row + (int64_t)h * step, srow + (int64_t)h * sstep, chunk, v, pack8(v),
                      inside && h < heads);
    }
  }
}

template <int D, int F>
cudaError_t launch_rope(const RopeArgs& a, bool pairs, int grid, cudaStream_t s) {
  if (pairs) norm_rope_kernel<D, F, true><<<grid, kThreads, 0, s>>>(a);
  else norm_rope_kernel<D, F, false><<<grid, kThreads, 0, s>>>(a);
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
  a.q_groups = (a.QN + per - 1) / per;
  a.kv_groups = (KVN + per - 1) / per;
  a.groups = a.q_groups + 2 * a.kv_groups;
  const int64_t grid = ((int64_t)a.T * a.groups + kThreads / 32 - 1) / (kThreads / 32);
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
