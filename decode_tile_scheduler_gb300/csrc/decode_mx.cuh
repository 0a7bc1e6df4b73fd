// decode_mx.cuh -- the decode kernel over an MXFP4 cache (part of decode.cu: the same
// plan, queue, units and combine).
//
// A key is 68 bytes of K and of V where FP8 has 136, for the same number of elements to
// widen, so the kernel is bound by the instructions of an element, not by memory.  What
// it does about that:
//  - Three CTAs to an SM, each with one producer warp and four consumer warps, so that a
//    chunk's set-up and waits run beside the others' products.
//  - Units of 16 columns (NG = 2) where a KV head has more than 8 widen the codes once for
//    both halves: 32 sequences of 512 to 4096 keys, 16 columns 51.6 us for 58.6, 128 query
//    heads 49.2 for 58.3; 16 sequences of 2 to 16 k keys with 1 to 4 rows of 4 heads 63.6
//    for 71.7 (when it was chosen; the columns' own factors and the windows of V scales
//    have cost these units 3 to 5 % since).  Window calls keep 8: of few tiles a unit, many
//    of them edges, 64 sequences, window 1024, 1 to 4 rows 54.4 us where 16 columns took
//    66.1; long windows lose by it (window 4096, four rows: 49.6 where 16 took 45.1).
//  - S^T = K Q^T: a warp has 32 of a tile's rows.  O^T = V^T P^T: it has 32 of the 128
//    elements, the ones under one scale, and all rows; P goes through shared memory, twice
//    (one barrier a tile).  So O is 8 registers a lane and needs no merge behind a chunk
//    (560 cycles where adding up four warps' O took 4500), and P meets one scale a key.
//  - Codes go from shared memory to mma fragments by ldmatrix.  K: 32 bits of a row are
//    eight elements of one scale group, two k-steps of m16n8k16 (the order of a
//    contraction is free).  V: to the transposing ldmatrix four elements of a key are
//    one 16-bit unit, so a lane gets two keys' units in a register; masks and shifts
//    pair the keys' codes in bytes, and cvt makes an fp16 pair of a byte.
//  - E2M1 codes are fp16 values as they are.  K scales multiply the partial scores of
//    their 32 elements in fp32; V scales multiply P, already in fp16 and transposed, as
//    fp16 pairs, where a chunk's scales of a group lie within 16 binades.  A group whose
//    scales do not has its P times scale made of the scores, as two terms in bf16, whose
//    exponents reach (kFar): a key of little weight, or none, takes no bit from the
//    others however large its V is.  (A batch whose every group is far 139 us for 35.)
//  - Each column's query is multiplied by a power of two of its own, so that no head or row
//    meets another's size.
//
// Measured (one GB300; the call with plan and combine): 4 sequences of 32 to 128 k keys,
// 64 / 8 heads (364 MB) 86.0 us, of which this kernel 79; its loads alone 65.6, its work
// alone 76.8.  32 sequences of 512 to 4096 keys 34.8 us.  A warp issues 518 instructions
// for 32 rows (139 of them conversions of 2 clocks, of which 128 of a byte of codes), in 950
// clocks of its scheduler: the ALU pipe is 50 % and mma 26 % busy, and these two do not run
// wholly side by side (4 cvt 8.1 clocks, 1 mma 8.1, both together 10.8; with 2 lop3 14.8
// where 12 were due).  So more warps do not help: four CTAs to an SM took 87.6 us, stages
// 2 to 4 the same, five CTAs (72 registers) 105; nor do finer chunks (the end times of
// CTAs draw together, the mean moves up).
#pragma once

namespace fia {
namespace {

template <bool MR, int NG>
struct MxCfg {
  static constexpr int D = 128, kRowBytes = D / 2;
  static constexpr int kWarps = 4, kRows = kKvTile / kWarps;  // consumers, rows of a tile each
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kCtas = 3;                             // to an SM
  static constexpr int kTileBytes = kKvTile * kRowBytes;      // K, or V
  static constexpr int kScaleBytes = kKvTile * 4;
  static constexpr int kOffScale = 2 * kTileBytes, kOffMask = kOffScale + 2 * kScaleBytes;
  static constexpr int kStageBytes = kOffMask + (MR ? kDecodeMaxRows * kKvTile : 0);
  static constexpr int kStages = NG == 2 ? 2 : 3;
  static constexpr int kQBytes = 8 * NG * D * 2;
  static constexpr int kOffQ = kStages * kStageBytes;
  // P^T of a tile for everyone, twice: the B fragments of a warp's rows, 16 bytes a lane and
  // half of the columns
  static constexpr int kOffQs = kOffQ + kQBytes;  // NG 2: the fragments of Q, in fp16
  static constexpr int kOffP = kOffQs + (NG == 2 ? kQBytes : 0);
  // a tile's scales as the products take them: K's of a row as four floats; V's, a copy of
  // 128 rows for each warp and its group, as fp16 pairs
  static constexpr int kOffKs = kOffP + 2 * NG * kWarps * 32 * 16;
  static constexpr int kOffVs = kOffKs + kKvTile * 16;
  // the warps' largest scores and sums of the columns
  static constexpr int kOffRed = kOffVs + kWarps * kKvTile * 2;
  static constexpr int kOffBar = kOffRed + 2 * kWarps * 8 * NG * 4;
  static constexpr int kOffMsg = (kOffBar + 8 * (2 * kStages + 2) + 15) / 16 * 16;
  static constexpr int kOffMisc = kOffMsg + 128;
  static constexpr int kOffGroups = kOffMisc + 16;            // the far groups' references, twice
  static constexpr int kOffFactors = kOffGroups + 8 * kWarps;  // NG 2: the columns' score factors
  static constexpr int kSmem = kOffFactors + (NG == 2 ? 64 : 0) + 512;  // + alignment slack (a swizzle's 512 bytes)
  static_assert(kStageBytes % 512 == 0, "alignment");
  static_assert(kCtas * (kSmem + 1024) <= 233472, "shared memory");
};

// Byte offset of 16-byte chunk `chunk` (0..3) of row `row` in a tile of 64-byte rows
// written by TMA with 64-byte swizzling.
__device__ __forceinline__ uint32_t sw64(uint32_t row, uint32_t chunk) {
  return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}
// Four E8M0 bytes as two bf16 pairs (exact; 255 is NaN, 0 is 2^-127), as four floats.
__device__ __forceinline__ void e8m0x4_to_bf16x2x2(uint32_t w, __nv_bfloat162 (&v)[2]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\tcvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  v[0] = *reinterpret_cast<const __nv_bfloat162*>(&lo);
  v[1] = *reinterpret_cast<const __nv_bfloat162*>(&hi);
}
__device__ __forceinline__ void bf16x2x2_to_f32x4(__nv_bfloat162 a, __nv_bfloat162 b, float (&f)[4]) {
  const uint32_t x = *reinterpret_cast<const uint32_t*>(&a), y = *reinterpret_cast<const uint32_t*>(&b);
  f[0] = __uint_as_float(x << 16);
  f[1] = __uint_as_float(x & 0xffff0000u);
  f[2] = __uint_as_float(y << 16);
  f[3] = __uint_as_float(y & 0xffff0000u);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 c = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&c);
}
__device__ __forceinline__ void e8m0x4_to_f32x4(uint32_t w, float (&f)[4]) {
  __nv_bfloat162 v[2];
  e8m0x4_to_bf16x2x2(w, v);
  bf16x2x2_to_f32x4(v[0], v[1], f);
}
// Where a window of V scales starts: its inner codes, 2^-7 to 1, are those of 32 values whose
// largest is 2^-6 to 6 (at 0 a chunk's first tile took its way to a window always: 32
// sequences of 512 to 4096 keys 35.7 us for 35.3, two of 300 and 777 9.5 for 9.0).
constexpr uint32_t kMxWindow = 131;
// A column's sum l as l * 2^-k below 2^-7, k returned and its exponent moved by it: O, moved
// as far, is then a 128th of an average of V, and 128 such do not leave fp32 together.
__device__ __forceinline__ int mx_lower(float& m, float& l) {
  const int k = l > 0.f ? (int)(__float_as_uint(l) >> 23) - 119 : 0;
  m += (float)k;
  l *= pow2_of(-k);
  return k;
}
// Keys of a block of 16.  The transposing ldmatrix gives a lane keys a, b of its first
// matrix and c, d of its second, whose codes pair as (a, c) and (b, d); movmatrix gives it
// neighbours of the score fragment.  With (a, b, c, d) = (q, 4 + q, 12 + q, 8 + q) every
// one of these sets of eight rows differs modulo 8, so no ldmatrix meets a bank twice.
__device__ __forceinline__ int mx_v_key(int lane) {  // whose address a lane gives: V
  const int q = (lane & 7) >> 1, kind = (lane & 1) | ((lane >> 2) & 2);
  return q + (kind == 0 ? 0 : kind == 1 ? 4 : kind == 2 ? 12 : 8);
}
__device__ __forceinline__ int mx_k_key(int row) {  // the key in row 0..15 of a score fragment
  const int q = (row & 7) >> 1, kind = (row & 1) | ((row >> 2) & 2);
  return q + (kind == 0 ? 0 : kind == 1 ? 12 : kind == 2 ? 4 : 8);
}
// The fragments of a group's two m-tiles.  A lane has four elements d = 4g .. +3 of the
// group of its four keys; m-tile h holds the elements 2h in its fragment rows 0-7, 2h + 1
// in rows 8-15.
__device__ __forceinline__ void mx_v_fragments(uint32_t lo, uint32_t hi, uint32_t (&va)[2][4]) {
  // bytes of two keys' codes of one element: 0, 2 (keys a, c), 0, 2 (b, d)
  const uint32_t ev = (lo & 0x0f0f0f0fu) | ((hi << 4) & 0xf0f0f0f0u);
  const uint32_t od = ((lo >> 4) & 0x0f0f0f0fu) | (hi & 0xf0f0f0f0u);  // and 1, 3
  e2m1x8_to_f16x2x4(ev, va[0][0], va[1][0], va[0][2], va[1][2]);
  e2m1x8_to_f16x2x4(od, va[0][1], va[1][1], va[0][3], va[1][3]);
}

// NG: halves of 8 columns; MR, X: as decode_kernel's.
template <int NG, bool MR, bool X>
__global__ void __launch_bounds__(MxCfg<MR, NG>::kThreads, MxCfg<MR, NG>::kCtas)
    decode_mx_kernel(const DecodeArgs a, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv) {
  using Cfg = MxCfg<MR, NG>;
  constexpr int D = Cfg::D, S = Cfg::kStages, W = Cfg::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) &
                                             ~uintptr_t(511));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBar);
  uint64_t* empty = full + S;
  uint64_t* qfull = empty + S;
  uint64_t* qempty = qfull + 1;
  int* misc = reinterpret_cast<int*>(smem + Cfg::kOffMisc);
  UnitMsg& msg = *reinterpret_cast<UnitMsg*>(smem + Cfg::kOffMsg);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], W);
    }
    mbar_init(qfull, 1);  // a chunk's message and query vectors
    mbar_init(qempty, W);
    misc[0] = 0;  // abort flag
    fence_barrier_init();
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  __syncthreads();
  pdl_wait();  // the plan (and anything else before us on the stream) is complete

  if (warp == W) {
    // ======================= producer =======================
    // Lanes 0-15 issue the K boxes (and the explicit-mask slices), 16-31 the V boxes, each
    // with its scales beside it; page ids as in decode_kernel, one per lane.
    const int isv = lane >> 4, rb = lane & 15;
    const int nrb = kKvTile / a.box_rows;
    int it = 0, ucount = 0;
    bool aborted = false;
    const bool once = a.HG == 1;
    const uint64_t pol = l2_evict_first_policy();
    const int4 ent0 = a.queue[blockIdx.x];
    int64_t hd[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) hd[k] = a.sched[k];
    const int64_t pmark = *a.prefill_mark;
    const bool plan_ok = (hd[5] == kDecodePlanMark) & (hd[6] == a.B) & (hd[7] == a.num_ctas) &
                         (hd[0] >= 1) & (hd[1] >= 1) & (hd[2] >= 0) & (hd[2] <= a.max_chunks) &
                         (pmark != kPrefillPlanMark);
    if (!plan_ok && lane == 0 && blockIdx.x == 0) atomicExch(a.err, 2);
    const int64_t C = plan_ok ? hd[0] : 1, c2 = plan_ok ? hd[1] : 1;
    const int64_t N = plan_ok ? hd[2] : 0;
    const int UPB = a.KVN * a.HG;
    int64_t g = plan_ok ? (int64_t)blockIdx.x : N;
    int4 ent = g < N ? ent0 : make_int4(0, 0, 0, 0);
    while (g < N) {
      int gn_l = 0;  // the next claim, read behind this chunk's first tile
      if (lane == 0) gn_l = (int)gridDim.x + atomicAdd(a.claim, 1);
      int64_t gn = N;
      int4 ent_n = make_int4(0, 0, 0, 0);
      bool fetched = false;
      const int b = ent.x & 0xffff, ql = (int)((uint32_t)ent.x >> 16);
      const int ci = (int)((uint32_t)ent.y >> 16), w = ent.y & 0xffff;
      bool ent_ok = b < a.B && ql >= 1 && ql <= a.S_max && w < UPB && ent.z >= 0 &&
                    ent.z <= a.S_kv && ent.w >= 0 && (int64_t)ent.w + ql <= a.q_rows;
      const UnitInfo r = unit_from(a, b, w, ent.w, ql, ent.z);
      const int ha = active_groups(a, r.q_len);
      ent_ok = ent_ok && r.hg < ha && r.ncols > 0;  // an active unit of the batch
      if (!ent_ok && lane == 0) atomicExch(a.err, 2);
      const int64_t cost = max(1, r.ntiles);
      const ChunkGeom gm = chunk_geom(cost, C, c2);
      int t_begin, t_end;
      if (ci < gm.n1) {
        t_begin = (int)(ci * C);
        t_end = (int)(t_begin + C);
      } else {
        t_begin = (int)(gm.n1 * C + (ci - gm.n1) * c2);
        t_end = (int)min(cost, t_begin + c2);
      }
      if (!ent_ok || ci >= gm.nch) t_begin = t_end = 0;  // nothing of a bad entry runs
      const int i_first = MR ? r.c0 / a.G : 0;
      const int i_last = MR ? (r.c0 + max(r.ncols, 1) - 1) / a.G : 0;
      // the chunk's page ids: the window's tiles, then the first tokens'
      int pg0 = 0, fg0 = 0, npg = 0, nfg = 0, mypage = 0;
      if (a.block_table && r.ntiles > 0 && t_begin < t_end) {
        const int we = X ? min(t_end, r.nwin) : t_end;
        if (t_begin < we) {
          pg0 = (int)page_index(a, (int64_t)(r.tile0 + t_begin) * kKvTile);
          npg = (int)page_index(a, min((int64_t)(r.tile0 + we) * kKvTile, (int64_t)r.kv_len) - 1) - pg0 + 1;
        }
        if (X && t_end > r.nwin) {
          fg0 = (int)page_index(a, (int64_t)max(t_begin - r.nwin, 0) * kKvTile);
          nfg = (int)page_index(a, min((int64_t)(t_end - r.nwin) * kKvTile, (int64_t)r.kv_len) - 1) - fg0 + 1;
        }
        if (npg + nfg <= 32 && lane < npg + nfg)
          mypage = a.block_table[(int64_t)r.b * a.max_blocks +
                                 (lane < npg ? pg0 + lane : fg0 + lane - npg)];
      }
      if (ent_ok && ci < gm.nch) {  // chunk description + the columns' query vectors
        const int64_t slot0 = a.sched[kSchedHeader + b];  // (in flight with the page ids)
        // (the consumers take both before the chunk's first tile)
        wait_or_abort(qempty, (ucount & 1) ^ 1, a.err, misc);
        if (lane == 0) {
          UnitMsg& m = msg;
          m.r = r;
          m.slot = slot0 + (int64_t)ci * (a.KVN * ha) + r.hk * ha + r.hg;
          m.ci = ci;
          m.nch = gm.nch;
          m.t_begin = t_begin;
          m.t_end = t_end;
          m.done = 0;
          mbar_arrive_expect_tx(qfull, (uint32_t)(r.ncols * D * 2));
        }
        __syncwarp();
        for (int i = i_first + lane; i <= i_last; i += 32) {
          const int cb = max(r.c0, i * a.G), ce = min(r.c0 + r.ncols, (i + 1) * a.G);
          bulk_load(smem + Cfg::kOffQ + (cb - r.c0) * D * 2,
                    a.q + ((int64_t)r.qrow0 + i) * a.q_stride +
                        ((int64_t)r.hk * a.G + cb - i * a.G) * D,
                    (uint32_t)((ce - cb) * D * 2), qfull);
        }
        ++ucount;
      }
      for (int t = t_begin; r.ntiles > 0 && t < t_end; ++t) {
        const int s = it % S;
        const int j0 = tile_at<X>(r, t) * kKvTile;
        const int jb = j0 + rb * a.box_rows;
        const bool mine = rb < nrb && jb < r.kv_len;
        int blk = 0, jp = 0;
        if (a.block_table) {
          const int pj = mine ? (int)page_index(a, jb) : 0;
          jp = jb - pj * a.block_size;
          if (npg + nfg <= 32)
            blk = pool_page(a, __shfl_sync(0xffffffffu, mypage, !X || t < r.nwin ? pj - pg0 : npg + pj - fg0));
          else if (mine)
            blk = pool_page(a, a.block_table[(int64_t)r.b * a.max_blocks + pj]);
        }
        if (a.debug && mine && a.block_table && blk == a.num_blocks) atomicExch(a.err, 3);
        const int prow = mine ? (int)pool_row(a, r.b, r.hk, blk, jb, jp) : 0;
        // the scales of a piece are contiguous, on 16-byte boundaries in 16-byte units:
        // pages are multiples of 32 rows, lengths of contiguous caches of 4
        const float* ssrc = zero_scales;  // (a page outside the pool: zeros)
        if (mine && (!a.block_table || blk < a.num_blocks))
          ssrc = (isv ? a.v_scale : a.k_scale) + scale_row_in(a, r.b, r.hk, blk, jb, jp);
        const int srows = a.block_table ? a.box_rows : min(a.box_rows, a.S_kv - jb);
        const int nvalid = min(nrb, (r.kv_len - j0 + a.box_rows - 1) / a.box_rows);
        const uint32_t bytes = 2u * (uint32_t)(nvalid * a.box_rows * Cfg::kRowBytes +
                                               (a.block_table ? nvalid * a.box_rows
                                                              : min(a.box_rows, a.S_kv - j0)) * 4);
        const bool with_mask = MR && a.mask;
        const int mrow_bytes = with_mask ? min(kKvTile, (r.kv_len - j0 + 15) & ~15) : 0;
        const int nmrows = with_mask ? i_last - i_first + 1 : 0;
        wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.err, misc);
        if (*reinterpret_cast<volatile int*>(misc)) {  // issue nothing after a time-out
          aborted = true;
          break;
        }
        uint8_t* st = smem + s * Cfg::kStageBytes;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes + (uint32_t)(nmrows * mrow_bytes));
        __syncwarp();
        if (with_mask && lane < nmrows)
          bulk_load(st + Cfg::kOffMask + lane * kKvTile,
                    a.mask + (int64_t)r.b * a.mask_bstride + (int64_t)(i_first + lane) * a.mask_rstride + j0,
                    (uint32_t)mrow_bytes, &full[s]);
        if (mine) {
          uint8_t* dst = st + isv * Cfg::kTileBytes + rb * a.box_rows * Cfg::kRowBytes;
          const int col = a.kv_layout == 1 ? 0 : r.hk * Cfg::kRowBytes;
          if (once) tma_load_2d_hint(dst, isv ? &tv : &tk, &full[s], col, prow, pol);
          else tma_load_2d(dst, isv ? &tv : &tk, &full[s], col, prow);
          bulk_load(st + Cfg::kOffScale + isv * Cfg::kScaleBytes + rb * a.box_rows * 4, ssrc,
                    (uint32_t)(srows * 4), &full[s]);
        }
        ++it;
        if (!fetched) {
          gn = __shfl_sync(0xffffffffu, (int64_t)gn_l, 0);
          if (gn < N) ent_n = a.queue[gn];
          fetched = true;
        }
      }
      if (aborted || *reinterpret_cast<volatile int*>(misc)) {
        aborted = true;
        break;
      }
      if (!fetched) {
        gn = __shfl_sync(0xffffffffu, (int64_t)gn_l, 0);
        if (gn < N) ent_n = a.queue[gn];
      }
      g = gn;
      ent = ent_n;
    }
    if (aborted) {
      // issue nothing more, and give the copies in flight a bounded time to land
      for (int k = max(0, it - S); k < it; ++k) mbar_wait(&full[k % S], (k / S) & 1, a.err);
      return;
    }
    pdl_trigger();  // this CTA loads nothing more: the combine kernel may launch
    if (lane == 0 && plan_ok) {  // the last CTA out resets the queue for the next execute
      __threadfence();
      if (atomicAdd(a.claim + 1, 1) == a.num_ctas - 1) {
        a.claim[0] = 0;
        a.claim[1] = 0;
      }
    }
    wait_or_abort(qempty, (ucount & 1) ^ 1, a.err, misc);  // the end: an empty message
    if (lane == 0) {
      msg.done = 1;
      mbar_arrive(qfull);
    }
    return;
  }

  // ======================= consumers =======================
  const int g = lane >> 2, q4 = lane & 3;
  const int R0 = warp * Cfg::kRows;
  const uint32_t smem_base = smem_u32(smem);
  constexpr int KS = D / 16;           // k-steps of the scores
  constexpr int NB = Cfg::kRows / 16;  // blocks of 16 rows, side by side
  // This lane's row in the ldmatrix of groups 0, 1 and of groups 2, 3 of a block of 16
  // rows: matrices (fragment rows 0-7, even group), (8-15, even), (0-7, odd), (8-15, odd);
  // and in the transposing one of two blocks of V, this warp's group.
  const int krow = R0 + mx_k_key(lane & 15);
  const uint32_t off[2] = {sw64(krow, lane >> 4), sw64(krow, 2 + (lane >> 4))};
  const uint32_t voff = Cfg::kTileBytes + sw64(16 * (lane >> 4) + mx_v_key(lane), warp);
  const int key[2] = {mx_k_key(g), mx_k_key(g + 8)};  // of this lane's two score rows
  float* red = reinterpret_cast<float*>(smem + Cfg::kOffRed);
  // V scales: this lane makes the pairs of keys (q, 12 + q), (4 + q, 8 + q) of block lane / 4
  const int vrow = 16 * g + q4;
  uint8_t* vs_mine = smem + Cfg::kOffVs + warp * (2 * kKvTile) + ((g >> 1) * 4 + q4) * 16 + (g & 1) * 8;
  const uint4* vs = reinterpret_cast<const uint4*>(smem + Cfg::kOffVs + warp * (2 * kKvTile)) + q4;

  int it = 0, ucount = 0;
  while (true) {
    wait_or_abort(qfull, ucount & 1, a.err, misc);
    // (the warps leave together: the merge meets at a named barrier)
    if (named_bar_or(1, 32 * W, msg.done || *reinterpret_cast<volatile int*>(misc))) break;
    const UnitInfo r = msg.r;
    const int kvl = r.kv_len;
    const int64_t slot0 = msg.slot;
    const int t_begin = msg.t_begin, t_end = msg.t_end;
    const bool split = msg.nch > 1;
    const bool two = NG == 2 && r.ncols > 8;  // (columns in the second half)
    // Q^T fragments in fp16, each column times a power of two that puts its largest element
    // at exponent 15 (decode_kernel tells why); k-step kk = 2*group + j covers
    // d = 32*group + 8*q + 4*j + {0..3}
    uint32_t qb[NG][KS][2];
    // the score factors of columns 2q, 2q + 1 (NG 2: in shared memory, for their registers)
    float slc[2];
    float* factors = reinterpret_cast<float*>(smem + Cfg::kOffFactors);
    {
      const uint16_t* qsm = reinterpret_cast<const uint16_t*>(smem + Cfg::kOffQ) + g * D + 8 * q4;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        uint32_t top = 0;  // (bf16 magnitudes order as integers)
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          uint2 v = make_uint2(0u, 0u);
          if (8 * n + g < r.ncols)
            v = *reinterpret_cast<const uint2*>(qsm + 8 * n * D + (kk >> 1) * 32 + 4 * (kk & 1));
          qb[n][kk][0] = v.x;
          qb[n][kk][1] = v.y;
          top = __vmaxu2(top, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu));
        }
        const int sh = column_shift(max(top >> 16, top & 0xffffu) >> 7);
        // (the score factor is positive, its sign in the queries: hidden scores stay -inf)
        const float up = copysignf(__int_as_float((127 + sh) << 23), a.scale_log2);
        const float down = fmaxf(fabsf(a.scale_log2) * __int_as_float((127 - sh) << 23), 1e-36f);
        if constexpr (NG == 2) {
          if (warp == 0 && q4 == 0) factors[8 * n + g] = down;
        } else {
          slc[0] = __shfl_sync(0xffffffffu, down, 8 * q4);
          slc[1] = __shfl_sync(0xffffffffu, down, 8 * q4 + 4);
        }
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t v = qb[n][kk][k];
            qb[n][kk][k] = pack_f16(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
          }
      }
      if constexpr (NG == 2) {  // (the four warps' fragments are the same: each keeps a quarter)
        uint4* qs = reinterpret_cast<uint4*>(smem + Cfg::kOffQs) + lane;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int j = 0; j < KS / 2; ++j)
            if (j == warp)
              qs[32 * (n * (KS / 2) + j)] =
                  make_uint4(qb[n][2 * j][0], qb[n][2 * j][1], qb[n][2 * j + 1][0], qb[n][2 * j + 1][1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty);
      ++ucount;
      if constexpr (NG == 2) named_bar_sync(1, 32 * W);
    }
    // O^T of this warp's group of 32 elements (mx_v_fragments)
    float acc[NG][2][4];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
    // Softmax references m_r, the warps' own copies of one (-inf: none yet; mu is 0 then),
    // lazy: a score may pass its column's by kOver.  They are kept kLift below the scores that
    // set them, so that P, at most 2^kOver, has fp16's bits down to 2^-(14 + kLift) of the
    // largest.
    constexpr float kLift = 8.f, kOver = 14.f;
    float m_r[NG][2], mu[NG][2], l_r[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_r[n][e] = -INFINITY;
        mu[n][e] = l_r[n][e] = 0.f;
      }
    // The window of this warp's V scales: codes win - 15 .. win, over whose 2^(win - 128) O is
    // kept; P meets factors of 2^-14 to 2.  So no product of a key within 2^-8 of its
    // column's largest weight falls below fp16's normal numbers, and what smaller ones lose
    // is below 2^-18 of O's terms.  It stays where it is unless a scale of the chunk's first
    // tile lies outside its inner eight codes.  A later code outside it, NaN (255) and 0
    // (values below bf16's normal numbers) apart, makes the group far for the rest of the
    // chunk: O is then over 2^(win - 127 - kFar), win the largest code so far.  Both halves
    // of `win` hold the code; far: the upper one 0xffff.
    uint32_t win = kMxWindow * 0x10001u;
    // The far groups' references, 0 where a group is not far: a copy for a tile and one for the
    // next, whose warps may write theirs while others still go by this tile's.
    if (lane < 2) reinterpret_cast<int*>(smem + Cfg::kOffGroups)[W * lane + warp] = 0;
    // Keys that count as zeros in O whatever they hold: past kv_len, and between a band's
    // first tokens and its window.  (Codes are numbers all: a scale of 0 is enough.)
    const auto gone = [&](int j) {
      return j >= kvl || (X && ((j < r.lo && j >= a.first_tokens) || j > r.hi));
    };

    const int ntile_here = r.ntiles == 0 ? 0 : (t_end - t_begin);
    for (int tt = 0; tt < ntile_here; ++tt, ++it) {
      const int s = it % S;
      wait_or_abort(&full[s], (it / S) & 1, a.err, misc);
      const uint32_t st = smem_base + s * Cfg::kStageBytes;
      const uint8_t* stp = smem + s * Cfg::kStageBytes;
      const int jt = tile_at<X>(r, t_begin + tt) * kKvTile;
      const int jw = jt + R0;  // first KV row of this warp
      const bool edge = (jw < r.lo_last) || (jw + Cfg::kRows - 1 > r.hi_first) || (MR && a.mask != nullptr);
      // ---------------- scales ----------------
      {
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(stp + Cfg::kOffScale) + R0 + lane;
        float kf[4];  // (K: a lane takes a row; NaN: the row's scores are NaN)
        e8m0x4_to_f32x4(sc[0], kf);
        *reinterpret_cast<float4*>(smem + Cfg::kOffKs + (R0 + lane) * 16) = make_float4(kf[0], kf[1], kf[2], kf[3]);
        const uint8_t* sv = stp + Cfg::kOffScale + Cfg::kScaleBytes + vrow * 4 + warp;
        uint32_t c[4] = {sv[0], sv[48], sv[16], sv[32]};  // keys q, 12 + q, 4 + q, 8 + q
        const bool some_gone = jt + kKvTile > kvl || (X && jt + kKvTile > a.first_tokens);
        const auto key_gone = [&](int k) { return gone(jt + vrow + (k == 0 ? 0 : k == 1 ? 12 : 4 * k - 4)); };
        if (some_gone)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (key_gone(k)) c[k] = (win - 4u) & 0xffffu;
        // factor 2^(1 - d) of a code d below the window's top: fp16 exponent 16 - d
        const uint32_t c01 = c[0] | c[1] << 16, c23 = c[2] | c[3] << 16;
        const uint32_t high = tt == 0 ? win - 0x40004u : win, out = tt == 0 ? 0xfff8fff8u : 0xfff0fff0u;
        uint2 f = make_uint2((c01 + 0x100010u - win) << 10, (c23 + 0x100010u - win) << 10);
        if (__any_sync(0xffffffffu, (((high - c01) | (high - c23)) & out) != 0u)) {
          uint32_t most = 0u, least = 255u;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c[k] != 0u && c[k] != 255u && !(some_gone && key_gone(k))) {
              most = max(most, c[k]);
              least = min(least, c[k]);
            }
          most = __reduce_max_sync(0xffffffffu, most);
          least = __reduce_min_sync(0xffffffffu, least);
          const uint32_t top = tt == 0 ? scale_window(least, most, kMxWindow) : win & 0xffffu;
          const bool was = win >> 31, far = was || most > top || least + 15 < top;
          const uint32_t now = far ? max(top, most) : top;
          if (far) {
            const int e = (int)(top - now) - (was ? kFar : 1) + kFar;  // O moves by 2^e
            const float f0 = pow2_of(e / 2), f1 = pow2_of(e - e / 2);
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[n][i][k] = acc[n][i][k] * f0 * f1;
            if (lane == 0) reinterpret_cast<int*>(smem + Cfg::kOffGroups)[W * (it & 1) + warp] = (int)now;
          }
          win = now | (far ? 0xffffu : now) << 16;
          uint32_t h[4];  // (far: O's products are made apart)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            h[k] = far ? 0u : c[k] == 255u ? 0x7e00u : (uint32_t)max((int)(c[k] + 16u - now), 0) << 10;
          f = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        }
        *reinterpret_cast<uint2*>(vs_mine) = f;
        __syncwarp();
      }
      // ---------------- S^T = K Q^T ----------------
      const float4* ks = reinterpret_cast<const float4*>(smem + Cfg::kOffKs) + R0;
      float x[NG][NB][4];  // keys key[0], key[0], key[1], key[1]; columns 2q, 2q + 1, ...
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float4 f0 = ks[16 * b + key[0]], f1 = ks[16 * b + key[1]];
        const float fa[4] = {f0.x, f0.y, f0.z, f0.w}, fb[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int n = 0; n < NG; ++n) x[n][b][0] = x[n][b][1] = x[n][b][2] = x[n][b][3] = 0.f;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {  // groups 2*jj, 2*jj + 1
          uint32_t w[4];  // (group 2*jj: both rows), (group 2*jj + 1: both), d = 8*q .. +7 of each
          ldsm_x4(st + off[jj] + 1024 * b, w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = 2 * jj + k;
            uint32_t ka[2][4];
            e2m1x8_to_f16x2x4(w[2 * k], ka[0][0], ka[0][2], ka[1][0], ka[1][2]);
            e2m1x8_to_f16x2x4(w[2 * k + 1], ka[0][1], ka[0][3], ka[1][1], ka[1][3]);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              if (n && !two) break;
              float s4[4] = {0.f, 0.f, 0.f, 0.f};
              if constexpr (NG == 2) {
                const uint4 qv = reinterpret_cast<const uint4*>(smem + Cfg::kOffQs)[32 * (n * (KS / 2) + j) + lane];
                mma_f16(s4, ka[0], qv.x, qv.y);
                mma_f16(s4, ka[1], qv.z, qv.w);
              } else {
                mma_f16(s4, ka[0], qb[n][2 * j][0], qb[n][2 * j][1]);
                mma_f16(s4, ka[1], qb[n][2 * j + 1][0], qb[n][2 * j + 1][1]);
              }
              x[n][b][0] += s4[0] * fa[j];
              x[n][b][1] += s4[1] * fa[j];
              x[n][b][2] += s4[2] * fb[j];
              x[n][b][3] += s4[3] * fb[j];
            }
          }
        }
      }
      // (rounded here, once: with the factor in the exponent's fma, the largest score and its
      // reference would differ by the product's rounding, thousands for scores of 2^40)
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float f[2] = {slc[0], slc[1]};
        if constexpr (NG == 2) {
          f[0] = factors[8 * n + 2 * q4];
          f[1] = factors[8 * n + 2 * q4 + 1];
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[n][b][k] *= f[k & 1];
      }
      // ---------------- mask ----------------
      if (edge) {
        const uint8_t* mk = stp + Cfg::kOffMask + R0;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // column 2q + e of the half
            int lo = r.lo, hi = r.hi, mrow = 0;  // the keys it sees, its mask row
            if constexpr (MR) {
              const int i = (r.c0 + min(8 * n + 2 * q4 + e, max(r.ncols, 1) - 1)) / a.G;
              row_bounds(a, r.q_len, kvl, i, &lo, &hi);
              mrow = (i - r.c0 / a.G) * kKvTile;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int k = e; k < 4; k += 2) {
                const int row = 16 * b + key[k >> 1], j = jw + row;
                bool ok = j >= lo;
                if (X) ok = ok || j < a.first_tokens;
                ok = ok && j <= hi;
                if (MR && a.mask) ok = ok && mk[mrow + row] == 0;
                if (!ok) x[n][b][k] = -INFINITY;
              }
          }
      }
      if (X && a.scores) {  // (decode_kernel: key weights)
        const int64_t base = ((int64_t)r.b * a.KVN + r.hk) * a.S_kv;
        const int end = min(kvl, a.S_kv);
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const int j = jw + 16 * b + key[k >> 1], c = 8 * n + 2 * q4;
              if (c < r.ncols && j < end)
                *reinterpret_cast<float2*>(a.scores + (base + j) * a.score_cols + r.c0 + c) =
                    make_float2(x[n][b][k], x[n][b][k + 1]);
            }
      }
      // ---------------- online softmax per column ----------------
      float top[NG][2];
      bool over = false;
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[n][0][e], x[n][0][2 + e]);
#pragma unroll
          for (int b = 1; b < NB; ++b) mx = fmaxf(mx, fmaxf(x[n][b][e], x[n][b][2 + e]));
          top[n][e] = mx;
          over |= mx > m_r[n][e] + kOver;
        }
      // P^T in fp16, transposed (keys q, 12 + q and 4 + q, 8 + q of column g), to everyone
      uint4* pm = reinterpret_cast<uint4*>(smem + Cfg::kOffP) + (it & 1) * (NG * 32 * W);
      float sum[NG][2];
      const auto store_p = [&]() {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          sum[n][0] = sum[n][1] = 0.f;
          if (n && !two) break;
          uint32_t pt[NB][2];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float pr[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              pr[k] = fast_exp2(x[n][b][k] - mu[n][k & 1]);
              sum[n][k & 1] += pr[k];
            }
            pt[b][0] = movmatrix_t(pack_f16(pr[0], pr[1]));
            pt[b][1] = movmatrix_t(pack_f16(pr[2], pr[3]));
          }
          pm[32 * (W * n + warp) + lane] = make_uint4(pt[0][0], pt[0][1], pt[1][0], pt[1][1]);
        }
      };
      static_assert(NB == 2, "P's words");
      store_p();
      bool any_far = false;
      // (the other copy of P has been read by all when they are here)
      if (named_bar_or(1, 32 * W, over || win >> 31)) {  // new references, and P again; far groups
        const int4 far = reinterpret_cast<const int4*>(smem + Cfg::kOffGroups)[it & 1];
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = top[n][e];
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (g == 0) red[(warp * NG + n) * 8 + 2 * q4 + e] = mx;
          }
        named_bar_sync(1, 32 * W);
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = red[n * 8 + 2 * q4 + e];
#pragma unroll
            for (int w2 = 1; w2 < W; ++w2) mx = fmaxf(mx, red[(w2 * NG + n) * 8 + 2 * q4 + e]);
            const float mold = m_r[n][e];
            if (mx > mold + kOver) {
              m_r[n][e] = mu[n][e] = mx - kLift;
              const float f = mold == -INFINITY ? 0.f : fast_exp2(mold - mu[n][e]);
              l_r[n][e] *= f;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                acc[n][i][e] *= f;
                acc[n][i][2 + e] *= f;
              }
            }
          }
        store_p();
        named_bar_sync(1, 32 * W);
        any_far = (far.x | far.y | far.z | far.w) != 0;
        if (any_far) {  // the scores in the place of this warp's K rows
          float4* xs = reinterpret_cast<float4*>(smem + s * Cfg::kStageBytes + R0 * Cfg::kRowBytes) + lane;
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int b = 0; b < NB; ++b)
              xs[32 * (n * NB + b)] = make_float4(x[n][b][0], x[n][b][1], x[n][b][2], x[n][b][3]);
        }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) l_r[n][e] += sum[n][e];
      // ---------------- O^T += V^T P^T, this warp's group, every row of the tile ----------------
#pragma unroll
      for (int b2 = 0; b2 < W; ++b2) {  // two blocks of 16
        const uint4 sv = vs[4 * b2];
        uint32_t w[4];  // (keys a, b), (c, d) of the first block, of the second
        ldsm_x4_t(st + voff + 2048 * b2, w[0], w[1], w[2], w[3]);
        uint32_t va[2][2][4];
        mx_v_fragments(w[0], w[1], va[0]);
        mx_v_fragments(w[2], w[3], va[1]);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          if (n && !two) break;
          const uint4 pv = pm[32 * (W * n + b2) + lane];
          uint32_t b0 = mul_f16x2(pv.x, sv.x), b1 = mul_f16x2(pv.y, sv.y);
          mma_f16(acc[n][0], va[0][0], b0, b1);
          mma_f16(acc[n][1], va[0][1], b0, b1);
          b0 = mul_f16x2(pv.z, sv.z);
          b1 = mul_f16x2(pv.w, sv.w);
          mma_f16(acc[n][0], va[1][0], b0, b1);
          mma_f16(acc[n][1], va[1][1], b0, b1);
        }
      }
      if (any_far) {
        // A far group's P times its scale over 2^(its reference - kFar), as two terms in bf16
        // one after the other, goes through the other copy of P, which nobody reads now.
        const float4* xs = reinterpret_cast<const float4*>(stp + R0 * Cfg::kRowBytes) + lane;
        uint4* pf = reinterpret_cast<uint4*>(smem + Cfg::kOffP) + (~it & 1) * (NG * 32 * W);
#pragma unroll 1
        for (int term = 0; term < 2 * W; ++term) {
          const int j = term >> 1;
          const int ref = reinterpret_cast<const int*>(smem + Cfg::kOffGroups)[W * (it & 1) + j];
          if (ref == 0) continue;
          const uint8_t* sv = stp + Cfg::kOffScale + Cfg::kScaleBytes + R0 * 4 + j;
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            if (n && !two) break;
            uint32_t pt[NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const float4 v = xs[32 * (n * NB + b)];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int row = 16 * b + key[h], c = gone(jw + row) ? 0 : sv[4 * row];
                const float e = c == 255 ? __int_as_float(0x7fffffff) : (float)(c + kFar - ref);
                pt[b][h] = movmatrix_t(bf16_term(fast_exp2((h ? v.z : v.x) - mu[n][0] + e),
                                                 fast_exp2((h ? v.w : v.y) - mu[n][1] + e), term & 1));
              }
            }
            pf[32 * (W * n + warp) + lane] = make_uint4(pt[0][0], pt[0][1], pt[1][0], pt[1][1]);
          }
          named_bar_sync(1, 32 * W);
          if (warp == j) {
#pragma unroll 1
            for (int b2 = 0; b2 < W; ++b2) {
              uint32_t w[4];
              ldsm_x4_t(st + voff + 2048 * b2, w[0], w[1], w[2], w[3]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t va[2][4];
                mx_v_fragments(w[2 * h], w[2 * h + 1], va);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int k = 0; k < 4; ++k) va[i][k] = f16x2_to_bf16x2(va[i][k]);
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                  if (n && !two) break;
                  const uint4 pv = pf[32 * (W * n + b2) + lane];
                  mma_bf16(acc[n][0], va[0], h ? pv.z : pv.x, h ? pv.w : pv.y);
                  mma_bf16(acc[n][1], va[1], h ? pv.z : pv.x, h ? pv.w : pv.y);
                }
              }
            }
          }
          named_bar_sync(1, 32 * W);
        }
        fence_proxy_async_smem();  // (before the copy that overwrites the scores)
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ---------------- the columns' sums over the warps ----------------
    float L[NG][2];
    float* red_l = red + W * NG * 8;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_r[n][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) red_l[(warp * NG + n) * 8 + 2 * q4 + e] = l;
      }
    named_bar_sync(1, 32 * W);
    const int back = (int)(win & 0xffffu) - (win >> 31 ? 127 + kFar : 128);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        L[n][e] = 0.f;
#pragma unroll
        for (int w2 = 0; w2 < W; ++w2) L[n][e] += red_l[(w2 * NG + n) * 8 + 2 * q4 + e];
        m_r[n][e] = number_of(m_r[n][e], L[n][e]);
        const int by = back - mx_lower(m_r[n][e], L[n][e]);
        const float f0 = pow2_of(by / 2), f1 = pow2_of(by - by / 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[n][i][e] = acc[n][i][e] * f0 * f1;
          acc[n][i][2 + e] = acc[n][i][2 + e] * f0 * f1;
        }
      }
    }
    const int64_t slot = min(max(slot0, (int64_t)0), a.max_chunks - 1);
    const int d = 32 * warp + 4 * g;
#pragma unroll
    for (int k = 0; k < 2 * NG; ++k) {
      const int n = k >> 1, e = k & 1, hh = 8 * n + 2 * q4 + e;  // the unit's column
      if (hh >= r.ncols) continue;
      const float4 o = make_float4(acc[n][0][e], acc[n][0][2 + e], acc[n][1][e], acc[n][1][2 + e]);
      if (!split) {
        const int c = r.c0 + hh;
        const int i = c / a.G, h = r.hk * a.G + (c - i * a.G);
        const int64_t tok = (int64_t)r.qrow0 + i;
        float scl, lse;
        finish_head(a, h, m_r[n][e], L[n][e], &scl, &lse);
        *reinterpret_cast<uint2*>(a.out + tok * a.out_stride + (int64_t)h * D + d) =
            make_uint2(pack_bf16(o.x * scl, o.y * scl), pack_bf16(o.z * scl, o.w * scl));
        if (a.lse && warp == 0 && g == 0)
          a.lse[a.layout == 1 ? tok * a.QN + h : ((int64_t)r.b * a.QN + h) * a.S_q + i] = lse;
      } else {
        // (the slot is clamped, as in decode_kernel; rows of D + 2 floats: 8-byte stores)
        float* col = a.partials + slot * (int64_t)a.GH * (D + 2) + (int64_t)hh * (D + 2);
        *reinterpret_cast<float2*>(col + d) = make_float2(o.x, o.y);
        *reinterpret_cast<float2*>(col + d + 2) = make_float2(o.z, o.w);
        if (warp == 0 && g == 0) *reinterpret_cast<float2*>(col + D) = make_float2(m_r[n][e], L[n][e]);
      }
    }
  }
}

template <int NG, bool MR, bool X>
cudaError_t launch_mx_t(const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  using Cfg = MxCfg<MR, NG>;
  auto kern = decode_mx_kernel<NG, MR, X>;
  static std::atomic<uint64_t> done_mask[4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask[(dev >> 6) & 3].load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    done_mask[(dev >> 6) & 3].fetch_or(bit);
  }
  return launch_pdl(kern, dim3(a.num_ctas), dim3(Cfg::kThreads), Cfg::kSmem, s, a, tk, tv);
}

template <int NG>
cudaError_t launch_mx(const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  const bool mr = a.S_max > 1 || a.mask != nullptr;
  if (a.first_tokens > 0 || a.scores)
    return mr ? launch_mx_t<NG, true, true>(a, tk, tv, s) : launch_mx_t<NG, false, true>(a, tk, tv, s);
  return mr ? launch_mx_t<NG, true, false>(a, tk, tv, s) : launch_mx_t<NG, false, false>(a, tk, tv, s);
}

}  // namespace

int decode_mx_ctas() { return MxCfg<false, 1>::kCtas; }

static cudaError_t launch_decode_mx(const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                                    cudaStream_t s) {
  return a.GH == 16 ? launch_mx<2>(a, tk, tv, s) : launch_mx<1>(a, tk, tv, s);
}

}  // namespace fia
