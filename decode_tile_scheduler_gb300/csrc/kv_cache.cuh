// kv_cache.cuh -- a KV cache as the calls that write to it see it: where the
// row of a key lies in either page layout or a contiguous cache, and the
// checks of the public struct they share (kv_append.cu, kv_evict.cu).
#pragma once

#include <cstring>

#include "../../include/fia.h"
#include "common.cuh"
#include "internal.h"

namespace fia {

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* bt;      // null: contiguous
  int64_t num_blocks;
  int B, KVN, D, cap;
  int max_blocks, bs;
  int head_major, fp8;
  uint32_t magic;         // j / bs == (j * magic) >> shift for 0 <= j < 2^31
  int shift;
};

struct RowAt {
  int64_t row;    // K and V: element row * D of the pool
  int64_t srow;   // FP8 scales: element srow * (D / 64)
  bool ok;        // the page lies inside the pool
};

// Page of key j of a paged cache, and the row of a key in it whose table entry is blk.
__device__ __forceinline__ int cache_page(const CacheView& c, int j) {
  return (int)(((uint64_t)(uint32_t)j * c.magic) >> c.shift);
}
__device__ __forceinline__ RowAt page_row(const CacheView& c, int hk, int j, int pg, int64_t blk) {
  RowAt r;
  const int jp = j - pg * c.bs;
  r.ok = blk >= 0 && blk < c.num_blocks;
  r.srow = (blk * c.KVN + hk) * c.bs + jp;
  r.row = c.head_major ? r.srow : (blk * c.bs + jp) * c.KVN + hk;
  return r;
}

// Row of key j (0 <= j < cap) of sequence b, KV head hk.
__device__ __forceinline__ RowAt cache_row(const CacheView& c, int b, int hk, int j) {
  if (!c.bt) {
    RowAt r;
    r.row = ((int64_t)b * c.cap + j) * c.KVN + hk;
    r.srow = ((int64_t)b * c.KVN + hk) * c.cap + j;
    r.ok = true;
    return r;
  }
  const int pg = cache_page(c, j);
  return page_row(c, hk, j, pg, __ldg(c.bt + (int64_t)b * c.max_blocks + pg));
}

inline int64_t cache_capacity(const fia_kv_cache& c) {
  return c.block_table ? (int64_t)c.max_blocks_per_seq * c.block_size : c.max_seqlen_kv;
}

inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// The limits of fia_params' cache (fia.h), without its query.
inline fia_status check_cache(const fia_kv_cache& c) {
  if (c.batch < 1 || c.batch > 65536) return FIA_ERR_BAD_SHAPE;
  if (c.num_kv_heads < 1 || c.num_kv_heads > 256) return FIA_ERR_BAD_SHAPE;
  if (c.head_dim < 1 || c.head_dim > 512) return FIA_ERR_BAD_SHAPE;
  if (c.kv_dtype != FIA_KV_BF16 && c.kv_dtype != FIA_KV_FP8_E4M3) return FIA_ERR_BAD_DTYPE;
  if (c.kv_layout != FIA_KV_LAYOUT_BNBSH && c.kv_layout != FIA_KV_LAYOUT_BNNBSD)
    return FIA_ERR_BAD_SHAPE;
  if (c.kv_layout == FIA_KV_LAYOUT_BNNBSD && !c.block_table) return FIA_ERR_BAD_SHAPE;
  if (!c.k_cache || !c.v_cache) return FIA_ERR_NULL_ARG;
  if (!aligned_to(c.k_cache, 16) || !aligned_to(c.v_cache, 16)) return FIA_ERR_BAD_SHAPE;
  const bool fp8 = c.kv_dtype == FIA_KV_FP8_E4M3;
  if (fp8) {
    if (!c.k_scale || !c.v_scale) return FIA_ERR_NULL_ARG;
    if (c.quant_tile != 64 || c.head_dim % 64) return FIA_ERR_BAD_SHAPE;
    if (!aligned_to(c.k_scale, 16) || !aligned_to(c.v_scale, 16)) return FIA_ERR_BAD_SHAPE;
    if (!c.block_table && (c.max_seqlen_kv & 1)) return FIA_ERR_BAD_SHAPE;
  }
  if (c.block_table) {
    if (c.block_size <= 0 || c.block_size % 16 || c.block_size > 1024) return FIA_ERR_BAD_SHAPE;
    if (fp8 && (c.block_size % 32 || c.block_size > 512)) return FIA_ERR_BAD_SHAPE;
    if (c.num_blocks <= 0 || c.max_blocks_per_seq <= 0) return FIA_ERR_BAD_SHAPE;
    if ((int64_t)c.num_blocks * c.block_size *
            (c.kv_layout == FIA_KV_LAYOUT_BNNBSD ? c.num_kv_heads : 1) > INT32_MAX)
      return FIA_ERR_BAD_SHAPE;
    if ((int64_t)c.max_blocks_per_seq * c.block_size > 20971520) return FIA_ERR_BAD_SHAPE;
  } else {
    if (c.max_seqlen_kv < 0 || c.max_seqlen_kv > 20971520) return FIA_ERR_BAD_SHAPE;
    if ((int64_t)c.batch * c.max_seqlen_kv > INT32_MAX) return FIA_ERR_BAD_SHAPE;
  }
  if (c.head_dim != 64 && c.head_dim != 128) return FIA_ERR_UNSUPPORTED;
  if (fp8 && c.head_dim != 128) return FIA_ERR_UNSUPPORTED;
  return FIA_OK;
}

// Multiplier and shift of j / d for 0 <= j < 2^31 (1 <= d <= 2^20): with
// l = ceil(log2 d), floor(2^(31+l) / d) + 1 and 31 + l.
inline CacheView cache_view(const fia_kv_cache& c) {
  CacheView w;
  memset(&w, 0, sizeof w);
  w.k = static_cast<uint8_t*>(c.k_cache);
  w.v = static_cast<uint8_t*>(c.v_cache);
  w.ks = c.k_scale;
  w.vs = c.v_scale;
  w.bt = c.block_table;
  w.num_blocks = c.num_blocks;
  w.B = c.batch;
  w.KVN = c.num_kv_heads;
  w.D = c.head_dim;
  w.cap = (int)cache_capacity(c);
  w.max_blocks = c.max_blocks_per_seq;
  w.bs = c.block_table ? c.block_size : 1;
  w.head_major = c.block_table && c.kv_layout == FIA_KV_LAYOUT_BNNBSD;
  w.fp8 = c.kv_dtype == FIA_KV_FP8_E4M3;
  int l = 0;
  while ((1 << l) < w.bs) ++l;
  w.magic = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint64_t)w.bs + 1);
  w.shift = 31 + l;
  return w;
}

}  // namespace fia
