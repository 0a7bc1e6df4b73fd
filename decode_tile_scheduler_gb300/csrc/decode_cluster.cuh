// decode_cluster.cuh -- decode calls of few units and few keys in one kernel (part of
// decode.cu): a cluster of eight CTAs per unit instead of plan, chunks, partials in
// global memory and a combine.  For a window with first tokens, for key weights, and for
// MXFP4 caches.
//
// A unit is (sequence, KV head, 8 columns (query row, head)).  Its warps, 64 in the
// cluster, take 16 keys at a time, straight from global memory into the fragments of
// mma.m16n8k16: the order of a contraction is free, so a lane's 16-byte piece of a K
// row is used as it lies, with Q's elements loaded in the same order, and the pieces
// of V rows are paired by byte permutes.  S = K Q^T has the keys as rows; the columns'
// maximum and sum are kept per warp, P^T comes from 8 x 8 transposes in registers,
// and O^T = V^T P stays in registers to the end.  Then the warps' (m, l, O) are folded
// in shared memory, the CTAs' through distributed shared memory, each CTA an eighth
// of D.  Key weights need no second look at K: a warp keeps its scores in shared
// memory until the columns' lse is known.
//
// MXFP4: a warp's 16 rows go through its part of shared memory, and from there as in
// decode_mx.cuh, windows of V scales and far groups too (a warp's own, of all four groups).
//
// Bound by latency: lengths and page table, then K and V, then two folds.  One sequence,
// 8 KV heads, a window of 1024 and 4 first tokens: 7.7 us a call in a graph (plan, decode
// and combine 12.4); two contexts of up to 777 keys with key weights 8.7 us (14.3).  At
// 188 registers, one CTA to an SM, 16 clusters of eight did not fit at once: 12.7 us.
#pragma once

#include "cluster.cuh"
#include "kv_cache.cuh"

namespace fia {
namespace {

// V scale factors (fp16) of rows 2k, 2k + 1 (lanes) as pairs: groups 0 and 1 from the even
// lane, 2 and 3 from the odd one.
__device__ __forceinline__ uint2 mx_scale_pairs(uint32_t h01, uint32_t h23, int lane) {
  const uint32_t theirs = __shfl_xor_sync(0xffffffffu, lane & 1 ? h01 : h23, 1);
  const uint32_t even = lane & 1 ? theirs : h01, odd = lane & 1 ? h23 : theirs;
  return make_uint2(__byte_perm(even, odd, 0x5410), __byte_perm(even, odd, 0x7632));
}
// The row of a block of 16 whose address this lane gives the transposing ldmatrix of V:
// matrices (keys 0, 8, 2, 10, 4, ..., even group), (1, 9, 3, 11, ..., even), and of the odd
// group.  A lane's first register then holds keys 2q and 2q + 8, its second 2q + 1 and
// 2q + 9, and one mask pairs the neighbours of both.
__device__ __forceinline__ int mx_v_row(int lane) {
  return 2 * ((lane & 7) >> 1) + 8 * (lane & 1) + ((lane >> 3) & 1);
}

constexpr int kFewCtas = 8, kFewWarps = 8, kFewThreads = 32 * kFewWarps;
constexpr int kFewKeys = 16;                               // keys of a warp's step
constexpr int kFewSpan = kFewCtas * kFewWarps;             // steps side by side
constexpr int kFewKept = kFewKeys * 8 + kFewKeys;          // floats kept per step (weights)
constexpr int kFewMaxRounds = 8;                           // steps of a warp, at most
constexpr int kFewMaxKept = 4;                             // the same with key weights
constexpr int kFewPages = 4 * kFewThreads;                 // table entries in shared memory

// The pairs (a.e, b.e) and (a.e+1, b.e+1) of four codes' bytes as two bf16 pairs.
__device__ __forceinline__ void codes_bf16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  uint32_t l, h;
  e4m3x4_to_f16x2x2(codes, l, h);  // (exact in either format)
  const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&l));
  const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&h));
  lo = pack_bf16(fl.x, fl.y);
  hi = pack_bf16(fh.x, fh.y);
}

enum FewFormat { kFewBf16, kFewFp8, kFewMx };

template <int D, int F, bool WT>
__global__ void __cluster_dims__(kFewCtas, 1, 1) __launch_bounds__(kFewThreads, 2)
    decode_few_kernel(const DecodeArgs a, const CacheView c, const KeyWeightsOut o, int groups,
                      int planned) {
  constexpr bool FP8 = F == kFewFp8, MX = F == kFewMx;
  constexpr int NK = FP8 ? 4 : D / 32;   // 16-byte pieces of a lane's Q row
  constexpr int NV = D / 64;             // pieces of a V row per lane, 8 elements each
  extern __shared__ float kept[];        // WT: per step of a warp, 16 keys x 8 scores, 16 old weights
  __shared__ __align__(16) float o_warp[kFewWarps][8][D];
  __shared__ __align__(16) float o_cta[8][D];
  __shared__ __align__(8) float2 ml_warp[kFewWarps][8];
  __shared__ __align__(8) float2 ml_cta[8];
  __shared__ float share[8][kFewCtas];   // what a CTA's O counts for, per column
  __shared__ float nl[8];                // -lse, log2 units
  __shared__ int32_t pages[kFewPages];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const int rank = (int)cluster_rank();
  const int unit = blockIdx.x / kFewCtas, grp = unit % groups, pair = unit / groups;
  const int b = pair / a.KVN, hk = pair - b * a.KVN;
  if (planned) {  // (else the plan is being built beside this kernel)
    pdl_wait();
    if (a.sched[5] != kDecodePlanMark || a.sched[6] != a.B || a.sched[7] != a.num_ctas ||
        *a.prefill_mark == kPrefillPlanMark) {
      if (blockIdx.x == 0 && tid == 0) atomicExch(a.err, 2);
      return;  // the whole grid
    }
  }
  const int32_t* table = c.bt ? c.bt + (int64_t)b * c.max_blocks : nullptr;
  int32_t page[kFewPages / kFewThreads];  // fetched beside the lengths
#pragma unroll
  for (int i = 0; i < kFewPages / kFewThreads; ++i)
    page[i] = table && tid + i * kFewThreads < c.max_blocks ? __ldg(table + tid + i * kFewThreads) : 0;
  int64_t qrow, ql, kl64;
  batch_lengths(a, b, &qrow, &ql, &kl64);
  const int kl = (int)min(max(kl64, (int64_t)0), (int64_t)a.S_kv);
  const UnitInfo r = unit_from(a, b, hk * a.HG, (int)qrow, ql, kl);
  const bool fits = r.q_len == 0 || lengths_fit(a, qrow, r.q_len, kl64);
  const int c0 = 8 * grp, ncols = fits ? min(8, r.q_len * a.G - c0) : 0;
  float* w_out = WT ? o.w_out + (int64_t)pair * o.stride : nullptr;
  const float* w_in = WT && o.w_in ? o.w_in + (int64_t)pair * o.stride : nullptr;

  // steps of 16 keys that some row sees: nwin from step s0 on, then 0, 1, ... (the
  // first tokens, where steps that no row sees lie between)
  int s0 = 0, nwin = 0, steps = 0;
  if (ncols > 0 && kl > 0) {
    const int nf = (min(a.first_tokens, r.hi + 1) + kFewKeys - 1) / kFewKeys;
    nwin = steps = nf;
    if (r.hi >= r.lo) {
      s0 = r.lo / kFewKeys;
      if (nf >= s0) {
        s0 = 0;
        nwin = steps = r.hi / kFewKeys + 1;
      } else {
        nwin = r.hi / kFewKeys - s0 + 1;
        steps = nwin + nf;
      }
    }
  }

  // Q in the order of the K pieces: lane (g, q4) holds column g's
  uint4 q[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    q[i] = make_uint4(0u, 0u, 0u, 0u);
    if (g < ncols) {
      const int col = c0 + g, row = col / a.G, h = hk * a.G + col - row * a.G;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (qrow + row) * a.q_stride + (int64_t)h * D);
      // bf16: piece q4 + 4i of 8 elements; FP8: the two halves of piece q4 + 4 (i / 2) of 16
      // (MXFP4: as bf16: the eight elements of group i at 8 q4)
      q[i] = __ldg(src + (FP8 ? 2 * (q4 + 4 * (i >> 1)) + (i & 1) : q4 + 4 * i));
    }
  }
  // MXFP4: Q in fp16, each column times a power of two, K's 2 k-steps a group, the score
  // factors (all as in decode_mx_kernel)
  float slc[2];
  uint32_t win = kMxWindow * 0x1010101u, far = 0u;  // a byte a group: its window's top; 0x80: far
  if constexpr (MX) {
    uint32_t emax = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) emax = max(emax, max((w[k] >> 7) & 0xffu, (w[k] >> 23) & 0xffu));
    }
    const int sh = column_shift(emax);
    const float up = __int_as_float((127 + sh) << 23);
    const float down = a.scale_log2 * __int_as_float((127 - sh) << 23);
    slc[0] = __shfl_sync(0xffffffffu, down, 8 * q4);
    slc[1] = __shfl_sync(0xffffffffu, down, 8 * q4 + 4);
    const auto half = [&](uint32_t w) {
      return pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
    };
#pragma unroll
    for (int i = 0; i < NK; ++i) q[i] = make_uint4(half(q[i].x), half(q[i].y), half(q[i].z), half(q[i].w));
  }
  // the bounds of this lane's two columns
  int lo[2], hi[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    lo[e] = 0;
    hi[e] = -1;
    const int col = 2 * q4 + e;
    if (col < ncols) row_bounds(a, r.q_len, kl, (c0 + col) / a.G, &lo[e], &hi[e]);
  }
#pragma unroll
  for (int i = 0; i < kFewPages / kFewThreads; ++i)
    if (table) pages[tid + i * kFewThreads] = page[i];
  __syncthreads();

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // FP8: the windows of the halves' V scales, 16 bits apart (0x8000 beside: far); O over
  // 2^(top - 140), far over 2^(top - 127 - kFar)
  uint32_t win8 = kFp8Window * 0x10001u;
  float O[NV][4][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) O[i][t][k] = 0.f;
  const int64_t row_bytes = MX ? D / 2 : (int64_t)D * (FP8 ? 1 : 2);
  const int64_t key_bytes = c.head_major ? row_bytes : row_bytes * a.KVN;
  for (int n = 0, t = wid * kFewCtas + rank; t < steps; ++n, t += kFewSpan) {
    const int j0 = (t < nwin ? s0 + t : t - nwin) * kFewKeys;
    RowAt at;  // (16 keys lie in one page)
    if (!table) {
      at = cache_row(c, b, hk, j0);
    } else {
      const int pg = cache_page(c, j0);
      at = page_row(c, hk, j0, pg, pg < kFewPages ? pages[pg] : __ldg(table + pg));
    }
    const int end = at.ok ? kl - j0 : 0;  // keys of the step that exist
    const uint8_t* kb = c.k + (at.ok ? at.row : 0) * row_bytes;
    const uint8_t* vb = c.v + (at.ok ? at.row : 0) * row_bytes;
    // keys that no row sees count as zeros in O too, whatever they hold
    const auto seen = [&](int k) {
      return k < end && j0 + k <= r.hi && (j0 + k >= r.lo || j0 + k < a.first_tokens);
    };
    // (MXFP4: 16-byte pieces of rows on their way to shared memory, piece lane % 4 of rows
    // lane / 4 and 8 more; the scales of row lane)
    uint8_t* rows = reinterpret_cast<uint8_t*>(o_warp[wid]);  // K, V, the scales as products take them
    uint4 kt[2], vt[2];
    uint32_t ksw = 0u, vsw = 0u;
    if constexpr (MX) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        kt[k] = vt[k] = make_uint4(0u, 0u, 0u, 0u);
        if (seen(g + 8 * k)) {
          kt[k] = __ldg(reinterpret_cast<const uint4*>(kb + (g + 8 * k) * key_bytes) + q4);
          vt[k] = __ldg(reinterpret_cast<const uint4*>(vb + (g + 8 * k) * key_bytes) + q4);
        }
      }
      if (lane < kFewKeys && seen(lane)) {
        ksw = __ldg(reinterpret_cast<const uint32_t*>(c.ks) + at.srow + lane);
        vsw = __ldg(reinterpret_cast<const uint32_t*>(c.vs) + at.srow + lane);
      }
    }
    uint4 kx[2][FP8 ? 2 : NK];
#pragma unroll
    for (int k = 0; k < 2 && !MX; ++k)
#pragma unroll
      for (int i = 0; i < (FP8 ? 2 : NK); ++i) {
        kx[k][i] = make_uint4(0u, 0u, 0u, 0u);
        if (seen(g + 8 * k))
          kx[k][i] = __ldg(reinterpret_cast<const uint4*>(kb + (g + 8 * k) * key_bytes) + q4 + 4 * i);
      }
    uint4 vx[4][NV];  // FP8: the first 8 bytes of each
#pragma unroll
    for (int k = 0; k < 4 && !MX; ++k) {
      const int key = 2 * q4 + (k & 1) + 8 * (k >> 1);
      const bool on = seen(key);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        vx[k][i] = make_uint4(0u, 0u, 0u, 0u);
        if (on) {
          if constexpr (FP8) {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(vb + key * key_bytes) + g + 8 * i);
            vx[k][i].x = x.x;
            vx[k][i].y = x.y;
          } else {
            vx[k][i] = __ldg(reinterpret_cast<const uint4*>(vb + key * key_bytes) + g + 8 * i);
          }
        }
      }
    }
    float2 ksc[2], vsc[2];  // FP8: the scales of keys g and g + 8
    if constexpr (FP8) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ksc[k] = vsc[k] = make_float2(0.f, 0.f);
        if (seen(g + 8 * k)) {
          ksc[k] = __ldg(reinterpret_cast<const float2*>(c.ks) + at.srow + g + 8 * k);
          vsc[k] = __ldg(reinterpret_cast<const float2*>(c.vs) + at.srow + g + 8 * k);
        }
      }
    }
    float* keep = kept + (n * kFewWarps + wid) * kFewKept;
    if (WT && lane < kFewKeys)
      keep[kFewKeys * 8 + lane] = w_in && j0 + lane < kl ? w_in[j0 + lane] : 0.f;

    // ---- scores ----
    float x[4];  // keys g, g, g + 8, g + 8; columns 2 q4, 2 q4 + 1, ...
    if constexpr (MX) {
      __syncwarp();  // (the step before has read its rows)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<uint4*>(rows + sw64(g + 8 * k, q4)) = kt[k];
        *reinterpret_cast<uint4*>(rows + 1024 + sw64(g + 8 * k, q4)) = vt[k];
      }
      float kf[4];
      e8m0x4_to_f32x4(ksw, kf);
      const bool counts = lane < kFewKeys && seen(lane);
      if (!counts) vsw = win - 0x04040404u;            // (in the windows)
      const uint32_t fct = vsw + (0x10101010u - win);  // 2^(1 - d): fp16 exponents 16 - d
      uint32_t h01 = __byte_perm(fct, 0u, 0x4140) << 10, h23 = __byte_perm(fct, 0u, 0x4342) << 10;
      const uint32_t out = n == 0 ? __vsub4(win - 0x04040404u, vsw) & 0xf8f8f8f8u : __vsub4(win, vsw) & 0xf0f0f0f0u;
      if (__any_sync(0xffffffffu, (out | far) != 0u)) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t code = vsw >> (8 * j) & 255u;
          const bool was = far >> (8 * j + 7) & 1u;
          const uint32_t most = __reduce_max_sync(0xffffffffu, !counts || code == 255u ? 0u : code);
          const uint32_t least = __reduce_min_sync(0xffffffffu, !counts || code == 0u ? 255u : code);
          const uint32_t top = n == 0 ? scale_window(least, most, kMxWindow) : win >> (8 * j) & 255u;
          const bool is = was || most > top || least + 15 < top;
          const uint32_t now = is ? max(top, most) : top;
          if (is) {
            const int e = (int)(top - now) - (was ? kFar : 1) + kFar;
            const float f0 = pow2_of(e / 2), f1 = pow2_of(e - e / 2);
#pragma unroll
            for (int i = 2 * (j & 1); i < 2 * (j & 1) + 2; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) O[j >> 1][i][k] = O[j >> 1][i][k] * f0 * f1;
            far |= 0x80u << (8 * j);
          }
          win = (win & ~(255u << (8 * j))) | now << (8 * j);
          h[j] = is ? 0u : code == 255u ? 0x7e00u : (uint32_t)max((int)(code + 16u - now), 0) << 10;
        }
        h01 = h[0] | h[1] << 16;
        h23 = h[2] | h[3] << 16;
      }
      const uint2 pairs = mx_scale_pairs(h01, h23, lane);
      if (lane < kFewKeys) {
        *reinterpret_cast<float4*>(rows + 2048 + lane * 16) = make_float4(kf[0], kf[1], kf[2], kf[3]);
        *reinterpret_cast<uint2*>(rows + 2304 + lane * 8) = pairs;
        *reinterpret_cast<uint32_t*>(rows + 2432 + lane * 4) = vsw;
      }
      __syncwarp();
      const float4 f0 = *reinterpret_cast<const float4*>(rows + 2048 + g * 16);
      const float4 f1 = *reinterpret_cast<const float4*>(rows + 2048 + (g + 8) * 16);
      const float fa[4] = {f0.x, f0.y, f0.z, f0.w}, fb[4] = {f1.x, f1.y, f1.z, f1.w};
      x[0] = x[1] = x[2] = x[3] = 0.f;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        uint32_t w[4];
        ldsm_x4(smem_u32(rows) + sw64(lane & 15, 2 * jj + (lane >> 4)), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = 2 * jj + k;
          uint32_t ka[2][4];
          e2m1x8_to_f16x2x4(w[2 * k], ka[0][0], ka[0][2], ka[1][0], ka[1][2]);
          e2m1x8_to_f16x2x4(w[2 * k + 1], ka[0][1], ka[0][3], ka[1][1], ka[1][3]);
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(s4, ka[0], q[j].x, q[j].y);
          mma_f16(s4, ka[1], q[j].z, q[j].w);
          x[0] += s4[0] * fa[j];
          x[1] += s4[1] * fa[j];
          x[2] += s4[2] * fb[j];
          x[3] += s4[3] * fb[j];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] *= slc[k & 1];
    } else if constexpr (FP8) {
      float h[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // the halves of D apart: each has its scale
#pragma unroll
        for (int k = 0; k < 4; ++k) h[i][k] = 0.f;
        const uint32_t w0[4] = {kx[0][i].x, kx[0][i].y, kx[0][i].z, kx[0][i].w};
        const uint32_t w1[4] = {kx[1][i].x, kx[1][i].y, kx[1][i].z, kx[1][i].w};
        const uint32_t qw[8] = {q[2 * i].x, q[2 * i].y, q[2 * i].z, q[2 * i].w,
                                q[2 * i + 1].x, q[2 * i + 1].y, q[2 * i + 1].z, q[2 * i + 1].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t f[4];
          codes_bf16(w0[k], f[0], f[2]);
          codes_bf16(w1[k], f[1], f[3]);
          mma_bf16(h[i], f, qw[2 * k], qw[2 * k + 1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[k] = a.scale_log2 * (ksc[k >> 1].x * h[0][k] + ksc[k >> 1].y * h[1][k]);
    } else {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint32_t f0[4] = {kx[0][i].x, kx[1][i].x, kx[0][i].y, kx[1][i].y};
        const uint32_t f1[4] = {kx[0][i].z, kx[1][i].z, kx[0][i].w, kx[1][i].w};
        mma_bf16(s, f0, q[i].x, q[i].y);
        mma_bf16(s, f1, q[i].z, q[i].w);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = a.scale_log2 * s[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + g + 8 * (k >> 1), e = k & 1;
      if (!(j <= hi[e] && (j >= lo[e] || j < a.first_tokens))) x[k] = -INFINITY;
    }
    if (WT) {
      *reinterpret_cast<float2*>(keep + g * 8 + 2 * q4) = make_float2(x[0], x[1]);
      *reinterpret_cast<float2*>(keep + (g + 8) * 8 + 2 * q4) = make_float2(x[2], x[3]);
    }

    // ---- softmax: this warp's running maximum and sum ----
    // FP8: P times its V scale is multiplied in fp16 (the codes are fp16 values, and
    // bf16 would drop three bits of P) over the top of a window of scales, or in two terms.
    float over[2];
    if constexpr (FP8) {
      uint32_t e[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) e[k] = seen(g + 8 * k) ? exponents2(vsc[k]) : win8 - 0x40004u;  // (inside)
      const uint32_t high = n == 0 ? win8 - 0x40004u : win8, out = n == 0 ? 0xfff8fff8u : 0xfff0fff0u;
      if (__any_sync(0xffffffffu, (((high - e[0]) | (high - e[1])) & out) != 0u)) {
        uint32_t next = 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t u = seen(g) ? e[0] >> (16 * i) & 0xffu : 0u, v = seen(g + 8) ? e[1] >> (16 * i) & 0xffu : 0u;
          const uint32_t most = __reduce_max_sync(0xffffffffu, max(u == 255u ? 0u : u, v == 255u ? 0u : v));
          const uint32_t least = __reduce_min_sync(0xffffffffu, min(u == 0u ? 255u : u, v == 0u ? 255u : v));
          const uint32_t top = n == 0 ? scale_window(least, most, kFp8Window) : win8 >> (16 * i) & 0xffu;
          const bool was = win8 >> (16 * i + 15) & 1u, is = was || most > top || least + 15 < top;
          const uint32_t now = is ? max(top, most) : top;
          if (is) {
            const int by = (int)(top - now) - (was ? kFar : 13) + kFar;
            const float f0 = pow2_of(by / 2), f1 = pow2_of(by - by / 2);
#pragma unroll
            for (int t4 = 0; t4 < 4; ++t4)
#pragma unroll
              for (int k = 0; k < 4; ++k) O[i][t4][k] = O[i][t4][k] * f0 * f1;
          }
          next |= (now | (is ? 0x8000u : 0u)) << (16 * i);
        }
        win8 = next;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)  // (far: O's products are made apart)
        over[i] = win8 >> (16 * i + 15) & 1u ? 0.f : pow2_of(140 - (int)(win8 >> (16 * i) & 0xffu));
    }
    float p[4], mus[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // (MXFP4: the reference lies 13 lower, which keeps P's bits in fp16)
      float mx = fmaxf(m[e], fmaxf(x[e], x[2 + e]) - (MX ? 13.f : 0.f));
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mu = mx == -INFINITY ? 0.f : mx;
      mus[e] = mu;
      const float corr = fast_exp2(m[e] - mu);  // (m = -inf: 0)
      m[e] = mx;
      p[e] = fast_exp2(x[e] - mu);
      p[2 + e] = fast_exp2(x[2 + e] - mu);
      l[e] = l[e] * corr + (p[e] + p[2 + e]);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          O[i][k][e] *= corr;
          O[i][k][2 + e] *= corr;
        }
    }

    // ---- O^T += V^T P: P is rounded to bf16 here (FP8: to fp16, see above) ----
    uint32_t b0, b1;
    if constexpr (MX) {
      const uint32_t p0 = movmatrix_t(pack_f16(p[0], p[1])), p1 = movmatrix_t(pack_f16(p[2], p[3]));
      const uint4 s0 = *reinterpret_cast<const uint4*>(rows + 2304 + q4 * 16);
      const uint4 s1 = *reinterpret_cast<const uint4*>(rows + 2304 + (q4 + 4) * 16);
      const uint32_t sa[4] = {s0.x, s0.y, s0.z, s0.w}, sb[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        uint32_t w[4];
        ldsm_x4_t(smem_u32(rows) + 1024 + sw64(mx_v_row(lane), 2 * jj + (lane >> 4)), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // group 2 jj + k: O's m-tiles 2 k and 2 k + 1 of half jj
          uint32_t va[2][4];
          mx_v_fragments(w[2 * k], w[2 * k + 1], va);
          b0 = mul_f16x2(p0, sa[2 * jj + k]);
          b1 = mul_f16x2(p1, sb[2 * jj + k]);
          mma_f16(O[jj][2 * k], va[0], b0, b1);
          mma_f16(O[jj][2 * k + 1], va[1], b0, b1);
        }
      }
      if (far) {  // P times its scale from the scores, as two terms in bf16
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!(far >> (8 * j + 7) & 1u)) continue;
          const int top = (int)(win >> (8 * j) & 255u) - kFar;
          const int c0 = rows[2432 + g * 4 + j], c1 = rows[2432 + (g + 8) * 4 + j];
          const float s0 = c0 == 255 ? __int_as_float(0x7fffffff) : (float)(c0 - top);
          const float s1 = c1 == 255 ? __int_as_float(0x7fffffff) : (float)(c1 - top);
          const float t0 = fast_exp2(x[0] - mus[0] + s0), t1 = fast_exp2(x[1] - mus[1] + s0);
          const float t2 = fast_exp2(x[2] - mus[0] + s1), t3 = fast_exp2(x[3] - mus[1] + s1);
          uint32_t w[4], va[2][4];
          ldsm_x4_t(smem_u32(rows) + 1024 + sw64(mx_v_row(lane), 2 * (j >> 1) + (lane >> 4)), w[0], w[1], w[2], w[3]);
          mx_v_fragments(w[2 * (j & 1)], w[2 * (j & 1) + 1], va);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int y = 0; y < 4; ++y) va[i][y] = f16x2_to_bf16x2(va[i][y]);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            b0 = movmatrix_t(bf16_term(t0, t1, y));
            b1 = movmatrix_t(bf16_term(t2, t3, y));
            mma_bf16(O[j >> 1][2 * (j & 1)], va[0], b0, b1);
            mma_bf16(O[j >> 1][2 * (j & 1) + 1], va[1], b0, b1);
          }
        }
      }
    } else if constexpr (!FP8) {
      b0 = movmatrix_t(pack_bf16(p[0], p[1]));
      b1 = movmatrix_t(pack_bf16(p[2], p[3]));
    }
#pragma unroll
    for (int i = 0; i < NV && !MX; ++i) {
      if constexpr (FP8) {
        const float v0 = (i ? vsc[0].y : vsc[0].x) * over[i], v1 = (i ? vsc[1].y : vsc[1].x) * over[i];
        b0 = movmatrix_t(pack_f16(p[0] * v0, p[1] * v0));
        b1 = movmatrix_t(pack_f16(p[2] * v1, p[3] * v1));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t f[4];
        if constexpr (FP8) {
          const uint32_t sel = k & 1 ? 0x7362u : 0x5140u;  // bytes (a.e, b.e, a.e+1, b.e+1)
          const uint32_t y0 = k < 2 ? vx[0][i].x : vx[0][i].y, y1 = k < 2 ? vx[1][i].x : vx[1][i].y;
          const uint32_t y2 = k < 2 ? vx[2][i].x : vx[2][i].y, y3 = k < 2 ? vx[3][i].x : vx[3][i].y;
          e4m3x4_to_f16x2x2(__byte_perm(y0, y1, sel), f[0], f[1]);
          e4m3x4_to_f16x2x2(__byte_perm(y2, y3, sel), f[2], f[3]);
          mma_f16(O[i][k], f, b0, b1);
        } else {
          const auto word = [&](const uint4& y) { return k == 0 ? y.x : k == 1 ? y.y : k == 2 ? y.z : y.w; };
          f[0] = __byte_perm(word(vx[0][i]), word(vx[1][i]), 0x5410);
          f[1] = __byte_perm(word(vx[0][i]), word(vx[1][i]), 0x7632);
          f[2] = __byte_perm(word(vx[2][i]), word(vx[3][i]), 0x5410);
          f[3] = __byte_perm(word(vx[2][i]), word(vx[3][i]), 0x7632);
          mma_bf16(O[i][k], f, b0, b1);
        }
      }
    }
    if (FP8 && (win8 & 0x80008000u)) {  // P times its scale from the scores, as two terms in bf16
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!(win8 >> (16 * i + 15) & 1u)) continue;
        const int top = (int)(win8 >> (16 * i) & 0xffu);
        float t4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          t4[k] = far_product(x[k] - mus[k & 1], i ? vsc[k >> 1].y : vsc[k >> 1].x, top);
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          b0 = movmatrix_t(bf16_term(t4[0], t4[1], term));
          b1 = movmatrix_t(bf16_term(t4[2], t4[3], term));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t f[4];
            const uint32_t sel = k & 1 ? 0x7362u : 0x5140u;
            const uint32_t y0 = k < 2 ? vx[0][i].x : vx[0][i].y, y1 = k < 2 ? vx[1][i].x : vx[1][i].y;
            const uint32_t y2 = k < 2 ? vx[2][i].x : vx[2][i].y, y3 = k < 2 ? vx[3][i].x : vx[3][i].y;
            codes_bf16(__byte_perm(y0, y1, sel), f[0], f[1]);
            codes_bf16(__byte_perm(y2, y3, sel), f[2], f[3]);
            mma_bf16(O[i][k], f, b0, b1);
          }
        }
      }
    }
  }

  // ---- the CTA's warps ----
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
    const int lower = MX ? mx_lower(m[e], l[e]) : 0;
    if (g == 0) ml_warp[wid][2 * q4 + e] = make_float2(m[e], l[e]);
    if constexpr (MX) {
      if (e == 0) __syncwarp();  // (o_warp held the last step's rows)
#pragma unroll
      for (int t = 0; t < 8; ++t) {  // group t / 2, elements 4g + 2 (t % 2) and the next
        const int back = (int)(win >> (4 * (t & 6)) & 255u) - lower -
                         (far >> (4 * (t & 6) + 7) & 1u ? 127 + kFar : 128);
        const float back0 = pow2_of(back / 2), back1 = pow2_of(back - back / 2);
        *reinterpret_cast<float2*>(&o_warp[wid][2 * q4 + e][32 * (t >> 1) + 4 * g + 2 * (t & 1)]) =
            make_float2(O[t >> 2][t & 3][e] * back0 * back1, O[t >> 2][t & 3][2 + e] * back0 * back1);
      }
    }
#pragma unroll
    for (int i = 0; i < NV && !MX; ++i) {
      const int by = FP8 ? (int)(win8 >> (16 * i) & 0xffu) - (win8 >> (16 * i + 15) & 1u ? 127 + kFar : 140) : 0;
      const float back0 = FP8 ? pow2_of(by / 2) : 1.f, back1 = FP8 ? pow2_of(by - by / 2) : 1.f;
#pragma unroll
      for (int k = 0; k < 4; ++k)  // elements 2k and 2k + 1 of piece g + 8i
        *reinterpret_cast<float2*>(&o_warp[wid][2 * q4 + e][(g + 8 * i) * 8 + 2 * k]) =
            make_float2(back0 * O[i][k][e] * back1, back0 * O[i][k][2 + e] * back1);
    }
  }
  __syncthreads();
  {
    // a warp per column
    const float2 ml = lane < kFewWarps ? ml_warp[lane][wid] : make_float2(-INFINITY, 0.f);
    float M = ml.x;
#pragma unroll
    for (int d = 1; d < kFewWarps; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    M = __shfl_sync(0xffffffffu, M, 0);
    // (scores that are all NaN leave m = -inf and l = NaN)
    const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : exp2f(ml.x - M);
    float L = ml.y * f;
#pragma unroll
    for (int d = 1; d < kFewWarps; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    if (lane == 0) ml_cta[wid] = make_float2(M, L);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int d = 2 * lane + 64 * i;
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kFewWarps; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k);
        const float2 v = *reinterpret_cast<const float2*>(&o_warp[k][wid][d]);
        if (fk != 0.f) {  // (a warp without keys)
          s.x += fk * v.x;
          s.y += fk * v.y;
        }
      }
      *reinterpret_cast<float2*>(&o_cta[wid][d]) = s;
    }
  }
  cluster_bar_arrive();
  cluster_bar_wait();

  // ---- the cluster's CTAs: a warp per column finds what each counts for ----
  {
    const float2 ml = lane < kFewCtas ? peer_load2(peer_addr(&ml_cta[wid], lane))
                                      : make_float2(-INFINITY, 0.f);
    float M = ml.x;
#pragma unroll
    for (int d = 1; d < kFewCtas; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    M = __shfl_sync(0xffffffffu, M, 0);
    const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : exp2f(ml.x - M);
    float L = ml.y * f;
#pragma unroll
    for (int d = 1; d < kFewCtas; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    L = __shfl_sync(0xffffffffu, L, 0);
    if (wid < ncols) {
      const int col = c0 + wid, i = col / a.G, h = hk * a.G + col - i * a.G;
      float scl, lse;
      finish_head(a, h, L != L ? 0.f : M, L, &scl, &lse);
      if (lane < kFewCtas) share[wid][lane] = f * scl;
      if (lane == 0) {
        nl[wid] = -1.4426950408889634f * lse;
        if (rank == 0 && a.lse)
          a.lse[a.layout == 1 ? (qrow + i) * a.QN + h : ((int64_t)b * a.QN + h) * a.S_q + i] = lse;
      }
    }
  }
  __syncthreads();
  constexpr int PER = D / kFewCtas / 2;  // pairs of elements of a column in this CTA
  if (tid < 8 * PER && tid / PER < ncols) {
    const int cl = tid / PER, d = rank * (D / kFewCtas) + 2 * (tid % PER);
    float2 v[kFewCtas];
#pragma unroll
    for (int k = 0; k < kFewCtas; ++k) v[k] = peer_load2(peer_addr(&o_cta[cl][d], k));
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kFewCtas; ++k) {
      const float f = share[cl][k];
      if (f != 0.f) {
        s.x += f * v[k].x;
        s.y += f * v[k].y;
      }
    }
    const int col = c0 + cl, i = col / a.G, h = hk * a.G + col - i * a.G;
    *reinterpret_cast<uint32_t*>(a.out + (qrow + i) * a.out_stride + (int64_t)h * D + d) =
        pack_bf16(s.x, s.y);
  }
  __syncwarp();
  cluster_bar_arrive();  // (the peers' reads of this CTA's memory)

  if constexpr (WT) {
    // two lanes a key, four columns each
    const int key = lane >> 1, q = 4 * (lane & 1);
    for (int n = 0, t = wid * kFewCtas + rank; t < steps; ++n, t += kFewSpan) {
      const int j = (t < nwin ? s0 + t : t - nwin) * kFewKeys + key;
      const float* keep = kept + (n * kFewWarps + wid) * kFewKept;
      float w = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = keep[key * 8 + q + e];
        // (a hidden pair adds nothing, whatever its row's lse)
        if (q + e < ncols && x != -INFINITY) w += fast_exp2(x + nl[q + e]);
      }
      w += __shfl_xor_sync(0xffffffffu, w, 1);
      if (q == 0 && j < kl) w_out[j] = keep[kFewKeys * 8 + key] + w;
    }
    // keys of the steps that no row sees
    for (int j = rank * kFewThreads + tid; j < kl; j += kFewCtas * kFewThreads) {
      const int s = j / kFewKeys;
      if (!((s >= s0 && s < s0 + nwin) || s < steps - nwin)) w_out[j] = w_in ? w_in[j] : 0.f;
    }
  }
  cluster_bar_wait();
  pdl_wait();  // (without a wait for the plan above: nothing behind this kernel overtakes it)
  if (!fits && rank == 0 && tid == 0) atomicExch(a.err, 2);  // (behind the plan, which clears it)
}

// Steps of 16 keys that a row of the call can see, at most.
int64_t few_steps(const DecodeArgs& a) {
  const int64_t all = ((int64_t)a.S_kv + kFewKeys - 1) / kFewKeys;
  if (a.mask_mode != 4) return all;
  // (a window and the first tokens, each cut at both ends)
  const int64_t keys = (int64_t)a.pre_tokens + a.next_tokens + a.S_max + a.first_tokens;
  return std::min(all, keys / kFewKeys + 3);
}

template <int D, int F, bool WT>
cudaError_t launch_few_t(const DecodeArgs& a, const CacheView& c, const KeyWeightsOut* w,
                         bool planned, cudaStream_t s) {
  const int groups = (a.S_max * a.G + 7) / 8;
  const size_t smem = WT ? 4 * (size_t)kFewKept * kFewWarps * ((few_steps(a) + kFewSpan - 1) / kFewSpan) : 0;
  const KeyWeightsOut o = WT ? *w : KeyWeightsOut{};
  auto kern = decode_few_kernel<D, F, WT>;
  static std::atomic<uint64_t> done_mask[4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask[(dev >> 6) & 3].load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * kFewKept * kFewWarps * kFewMaxKept);
    if (e != cudaSuccess) return e;
    done_mask[(dev >> 6) & 3].fetch_or(bit);
  }
  return launch_pdl(kern, dim3(a.B * a.KVN * groups * kFewCtas),
                    dim3(kFewThreads), smem, s, a, c, o, groups, planned ? 1 : 0);
}

}  // namespace

// The rule: clusters that run at once (two CTAs to an SM; 16 clusters of 8 fit with
// one to an SM), and rounds up to which this kernel was the faster.  Measured (us a
// call, here / plan, decode and combine; 4 query heads per KV head, bf16): 4 units,
// window 1000 7.3 / 12.4, 8000 14.4 / 16.8; 32 units, 1000 9.5 / 15.7, 8000 27.0 /
// 32.4; 48 units, 1000 16.8 / 16.8.  With key weights 4 units of 1000 keys 8.3 / 13.9,
// of 4000 14.1 / 14.5, of 8000 22.3 / 17.5; 32 units 10.8 / 17.6, 18.8 / 26.3, 37.3 /
// 36.1; 48 units of 2000 keys 24.1 / 23.3.  FP8 gains more.  MXFP4 takes it for calls
// without a window too: 8 units, 300 keys 9.7 / 14.5, 2000 10.8 / 16.4, 4000 14.2 / 16.8,
// 8000 18.5 / 21.8; 32 units, 300 10.3 / 14.8, 4000 16.5 / 24.0, 8000 24.6 / 26.8.  (With
// FIA_DEBUG the other kernels run: they report pages outside the pool.)
bool decode_is_few(const DecodeArgs& a, bool weights) {
  const int sms = a.mx ? a.num_ctas / decode_mx_ctas() : a.num_ctas;
  if ((a.first_tokens == 0 && !weights && !a.mx) || a.mask || a.debug || sms < kFewCtas) return false;
  const int64_t groups = (a.S_max * a.G + 7) / 8;
  if (weights && groups > 1) return false;  // (a key's weight is a sum within one unit)
  return (int64_t)a.B * a.KVN * groups * 9 <= 2 * sms &&
         few_steps(a) <= kFewSpan * (weights ? kFewMaxKept : kFewMaxRounds);
}

cudaError_t launch_decode_few(const DecodeArgs& a, const fia_kv_cache& cache, const KeyWeightsOut* w,
                              bool planned, cudaStream_t s) {
  const CacheView c = cache_view(cache);
  if (c.mx)
    return w ? launch_few_t<128, kFewMx, true>(a, c, w, planned, s)
             : launch_few_t<128, kFewMx, false>(a, c, w, planned, s);
  if (c.fp8)
    return w ? launch_few_t<128, kFewFp8, true>(a, c, w, planned, s)
             : launch_few_t<128, kFewFp8, false>(a, c, w, planned, s);
  if (a.D == 64)
    return w ? launch_few_t<64, kFewBf16, true>(a, c, w, planned, s)
             : launch_few_t<64, kFewBf16, false>(a, c, w, planned, s);
  return w ? launch_few_t<128, kFewBf16, true>(a, c, w, planned, s)
           : launch_few_t<128, kFewBf16, false>(a, c, w, planned, s);
}

}  // namespace fia
