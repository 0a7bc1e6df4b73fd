// key_weights.cu -- how much attention weight each cached key received: for key
// j of KV head g, the probabilities exp(scale * q_ih . k_j - lse_ih) summed over
// the query rows i and the heads h of g's group that see it, added to what the
// key had.  It runs behind the attention kernels, whose lse it takes.
#include "kv_cache.cuh"
#include "internal.h"

namespace fia {

namespace {

// First token row, query length and KV length of batch b.
__device__ __forceinline__ void lengths(const WeightsArgs& a, int b, int64_t* qrow, int* ql,
                                        int* kl) {
  if (a.cu_seqlens_q) {
    *qrow = a.cu_seqlens_q[b];
    *ql = a.cu_seqlens_q[b + 1] - a.cu_seqlens_q[b];
  } else {
    *qrow = (int64_t)b * a.S_q;
    *ql = a.S_q;
  }
  *kl = min(a.seqused_kv ? a.seqused_kv[b] : a.S_kv, a.S_kv);
}

__device__ __forceinline__ bool sees(const WeightsArgs& a, int ql, int kl, int b, int i, int j) {
  const int64_t p = (int64_t)(a.mask_mode == 2 ? 0 : kl - ql) + i;
  if (a.mask_mode == 2 || a.mask_mode == 3) return j <= p;
  if (a.mask_mode == 4)
    return j <= p + a.next_tokens && (j >= p - a.pre_tokens || j < a.first_tokens);
  return !a.mask || a.mask[(int64_t)b * a.mask_bstride + (int64_t)i * a.mask_rstride + j] == 0;
}

// A thread per key: its row in registers, the query rows one after another.
template <int D>
__global__ void __launch_bounds__(128) key_weights_kernel(const WeightsArgs a, const CacheView c) {
  if (a.err && *a.err == 2) return;  // no plan of these arguments: the attention did not run
  const int b = blockIdx.z, hk = blockIdx.y, j = blockIdx.x * 128 + threadIdx.x;
  int64_t qrow;
  int ql, kl;
  lengths(a, b, &qrow, &ql, &kl);
  if (j >= kl) return;
  float k[D];
  const RowAt r = cache_row(c, b, hk, j);
  for (int d = 0; d < D; ++d) {
    if (!r.ok) k[d] = 0.f;
    else if (c.fp8) {
      uint16_t h = c.k[r.row * D + d];
      const uint32_t f2 = e4m3x2_to_f16x2(h);
      k[d] = __half2float(__ushort_as_half((unsigned short)f2)) * c.ks[r.srow * (D / 64) + d / 64];
    } else {
      k[d] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(c.k)[r.row * D + d] << 16);
    }
  }
  float sum = 0.f;
  for (int i = 0; i < ql; ++i) {
    if (!sees(a, ql, kl, b, i, j)) continue;
    for (int g = 0; g < a.G; ++g) {
      const int h = hk * a.G + g;
      const int64_t tok = qrow + i;
      const uint16_t* q = a.q + tok * a.q_stride + (int64_t)h * D;
      float s = 0.f;
      for (int d = 0; d < D; ++d) s += k[d] * __uint_as_float((uint32_t)q[d] << 16);
      const float lse = a.lse[a.cu_seqlens_q ? tok * a.QN + h
                                             : ((int64_t)b * a.QN + h) * a.S_q + i];
      sum += expf(s * a.scale - lse);
    }
  }
  const int64_t at = ((int64_t)b * a.KVN + hk) * a.stride + j;
  a.w_out[at] = (a.w_in ? a.w_in[at] : 0.f) + sum;
}

}  // namespace

cudaError_t launch_key_weights(const WeightsArgs& a, const fia_kv_cache& cache, cudaStream_t s) {
  const CacheView c = cache_view(cache);
  const dim3 grid((a.S_kv + 127) / 128, a.KVN, a.B);
  if (a.S_kv == 0) return cudaSuccess;
  if (a.D == 64) key_weights_kernel<64><<<grid, 128, 0, s>>>(a, c);
  else key_weights_kernel<128><<<grid, 128, 0, s>>>(a, c);
  return cudaGetLastError();
}

}  // namespace fia
