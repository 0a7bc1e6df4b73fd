// key_weights.cu -- how much attention weight each cached key received from a
// prompt: for key j of KV head g, w_j = sum over the query rows i and the heads
// h of g's group that see it of exp(scale * q_ih . k_j - lse_ih), added to what
// the key had.  It runs behind the prefill kernel, whose lse it takes (the
// probabilities need the finished lse, so the products Q K^T are formed again).
// The decode kernel's calls keep their scores instead (decode.cu).
//
// The products are formed transposed, S^T = K Q^T: 128 keys are the M rows of a
// tcgen05.mma (TMEM lanes), 128 query rows of one head its N columns.  A key's
// weight is then a sum along a lane: one thread adds up its key over all rows
// and heads in a register, with no reduction across threads and no atomics.
//
// Work: a unit is (sequence, KV head, 256 keys), its steps the (query tile,
// head) pairs that see some of its keys, cut into parts of at most `chunk`
// steps so that short calls still fill the GPU.  A part keeps its two K tiles in
// shared memory and streams the Q tiles past them; each K tile belongs to one
// epilogue warpgroup, so a Q tile in shared memory serves 2 x 128 keys (with one
// K tile per part the Q reads from L2 alone would be 32 KB per 1024 cycles of
// exponentials, on 152 SMs about the L2's rate).  A part's sums go to its own
// row of the workspace, and key_weights_fold_kernel adds the parts of a key in
// order, so the result does not depend on which CTA ran what.
//
// FP8 keys: E4M3 codes are bf16 values as they are, so the K tiles are widened
// to bf16 without their scales, the two 64-element halves of D accumulate apart,
// and a key's two scales multiply the two sums of its lane: no rounding of K.
//
// Bound: one ex2 per (key, row, head) on the MUFU, 16 a clock per SM, i.e. 1024
// cycles per 128 x 128 tile, against 512 on the tensor core (D = 128).
#include <algorithm>
#include <atomic>

#include "kv_cache.cuh"
#include "tcgen05.cuh"

namespace fia {

namespace {

constexpr int kWThreads = 384;
constexpr int kUnitKeys = 2 * kKvTile;

template <int D, bool FP8>
struct WeightsCfg {
  static constexpr int kNsub = D / 64;
  static constexpr int kTile = kNsub * 128 * 128;           // a 128-row bf16 tile
  static constexpr int kQStages = D == 128 ? 3 : 4;
  // bf16: two units' K tiles; FP8: one unit's, and two of codes
  static constexpr int kKStages = FP8 ? 1 : 2;
  static constexpr int kCodeStages = FP8 ? 2 : 0;
  static constexpr int kCodeTile = 128 * 128;
  static constexpr int kSBuf = FP8 ? 1 : 2;                 // S buffers per warpgroup
  static constexpr int kOffK = 0;
  static constexpr int kOffCode = kOffK + 2 * kKStages * kTile;
  static constexpr int kOffQ = kOffCode + 2 * kCodeStages * kCodeTile;
  static constexpr int kOffLse = kOffQ + kQStages * kTile;
  static constexpr int kLseStages = 3;
  static constexpr int kOffBar = kOffLse + kLseStages * 128 * 4;
  // mfull[2] mempty[2] kfull[2] kempty[2] kconv qfull[QS] qempty[QS] lfull[LS]
  // lempty[LS] sfull[2][2] sempty[2][2] drain
  static constexpr int kBars = 9 + 2 * kQStages + 2 * kLseStages + 8 + 1;
  static constexpr int kOffMsg = kOffBar + 8 * kBars;
  static constexpr int kOffMisc = kOffMsg + 2 * 64;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

struct WMsg {
  int b, hk, j0, kl, ql, qt0, s0, s1;  // steps s0 .. s1 - 1 of the unit
  int part, done;
  int64_t qrow;                        // first token row of the sequence
};
static_assert(sizeof(WMsg) <= 64, "message slot");

// First token row, query length and KV length of sequence b.
__device__ __forceinline__ void w_lengths(const WeightsArgs& a, int b, int64_t* qrow, int* ql,
                                          int* kl) {
  if (a.cu_seqlens_q) {
    // (lengths past the declared bounds are cut: the partial sums have no room)
    *qrow = max(a.cu_seqlens_q[b], 0);
    *ql = (int)max(min(min((int64_t)a.cu_seqlens_q[b + 1], a.q_rows) - *qrow, (int64_t)a.S_q),
                   (int64_t)0);
  } else {
    *qrow = (int64_t)b * a.S_q;
    *ql = a.S_q;
  }
  *kl = min(max(a.seqused_kv ? a.seqused_kv[b] : a.S_kv, 0), a.S_kv);
}

// Query rows [*lo, *hi] of a sequence that see key j (hi < lo: none).  An
// explicit mask hides single pairs of them.
__device__ __forceinline__ void rows_of_key(const WeightsArgs& a, int ql, int kl, int j, int* lo,
                                            int* hi) {
  int64_t l = 0, h = (int64_t)ql - 1;
  const int64_t off = (int64_t)kl - ql;  // row i sits at position off + i
  if (a.mask_mode == 2) {
    l = j;
  } else if (a.mask_mode == 3) {
    l = j - off;
  } else if (a.mask_mode == 4) {
    l = (int64_t)j - a.next_tokens - off;
    if (j >= a.first_tokens) h = min(h, (int64_t)j + a.pre_tokens - off);
  }
  l = max(l, (int64_t)0);
  if (j >= kl) l = ql;
  *lo = (int)min(l, (int64_t)ql);
  *hi = (int)max(h, (int64_t)-1);
}

// Steps of the unit at key j0: query tiles *qt0 .. *qt0 + n - 1 times G heads.
__device__ __forceinline__ int unit_steps(const WeightsArgs& a, int ql, int kl, int j0, int* qt0) {
  *qt0 = 0;
  if (j0 >= kl || ql <= 0) return 0;
  int lo, hi, lo1, hi1;
  rows_of_key(a, ql, kl, j0, &lo, &hi);
  rows_of_key(a, ql, kl, min(j0 + kUnitKeys, kl) - 1, &lo1, &hi1);
  if (hi1 < hi) hi1 = hi;  // (a first token is seen by every later row)
  if (hi1 < lo) return 0;
  *qt0 = lo / kQTile;
  return (hi1 / kQTile - lo / kQTile + 1) * a.G;
}
__device__ __forceinline__ int unit_parts(const WeightsArgs& a, int steps) {
  return (steps + a.chunk - 1) / a.chunk;
}

__device__ __forceinline__ bool plan_ok(const WeightsArgs& a) {
  return a.plan[0] == kPrefillPlanMark && a.plan[1] == a.B && a.plan[2] == a.num_ctas;
}

__device__ __forceinline__ float2 w_ffma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float w_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kWThreads, 1)
    key_weights_kernel(const WeightsArgs a, const CacheView c,
                       const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk) {
  using Cfg = WeightsCfg<D, FP8>;
  constexpr int QS = Cfg::kQStages, LS = Cfg::kLseStages, NSUB = Cfg::kNsub;
  constexpr int KS = FP8 ? Cfg::kCodeStages : Cfg::kKStages;  // stages the producer fills
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* mfull = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBar);
  uint64_t* mempty = mfull + 2;
  uint64_t* kfull = mempty + 2;
  uint64_t* kempty = kfull + 2;
  uint64_t* kconv = kempty + 2;
  uint64_t* qfull = kconv + 1;
  uint64_t* qempty = qfull + QS;
  uint64_t* lfull = qempty + QS;
  uint64_t* lempty = lfull + LS;
  uint64_t* sfull = lempty + LS;   // [warpgroup][buffer]
  uint64_t* sempty = sfull + 4;
  uint64_t* drain = sempty + 4;
  WMsg* msg = reinterpret_cast<WMsg*>(smem + Cfg::kOffMsg);
  int* misc = reinterpret_cast<int*>(smem + Cfg::kOffMisc);  // [0] abort, [1] tmem base
  float* lse_s = reinterpret_cast<float*>(smem + Cfg::kOffLse);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&mfull[s], 1);
      mbar_init(&mempty[s], 4);        // MMA thread, lse warp, two warpgroups
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], FP8 ? 2 : 1);  // codes: the warpgroups; bf16: the MMA's commit
    }
    mbar_init(kconv, 2);
    for (int s = 0; s < QS; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qempty[s], 1);
    }
    for (int s = 0; s < LS; ++s) {
      mbar_init(&lfull[s], 1);
      mbar_init(&lempty[s], 8);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], 4);
    }
    mbar_init(drain, 1);
    misc[0] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
  }
  if (warp == 1) {
    tmem_alloc(reinterpret_cast<uint32_t*>(&misc[1]), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[1]);
  pdl_wait();  // the attention is done: its lse, and the plan before it
  const bool ok = plan_ok(a);
  volatile int* abort_flag = misc;
  // (the same answer for a whole warp)
  auto stopped = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };

  if (warp == 0) {
    // ============================ producer ============================
    // Items in order: sequence, then 256 keys, then KV head, then part (each
    // unit of a sequence with as many parts as its longest has; those past a
    // unit's own are skipped).  A CTA's claims only grow, so the sequence of an
    // item is found by walking on from the last one's, 32 lengths at a time.
    int ucnt = 0, qn = 0;
    int win = 0;                 // first sequence of the lanes' window
    int64_t base = 0;            // items before it
    int64_t qrow = 0, items = 0, before = 0, total = 0;
    int ql = 0, kl = 0, parts = 0;
    auto load_window = [&]() {
      const int b = win + lane;
      ql = kl = parts = 0;
      items = 0;
      if (ok && b < a.B) {
        w_lengths(a, b, &qrow, &ql, &kl);
        parts = unit_parts(a, (ql + kQTile - 1) / kQTile * a.G);
        items = (int64_t)((kl + kUnitKeys - 1) / kUnitKeys) * a.KVN * parts;
      }
      int64_t x = items;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      before = x - items;
      total = __shfl_sync(0xffffffffu, x, 31);
    };
    load_window();
    int claim = 0;
    if (lane == 0 && ok) claim = atomicAdd(a.claim, 1);
    while (true) {
      const int64_t idx = __shfl_sync(0xffffffffu, claim, 0);
      while (ok && win < a.B && base + total <= idx) {
        base += total;
        win += 32;
        load_window();
      }
      const bool done = stopped() || !ok || win >= a.B;
      if (!done && lane == 0) claim = atomicAdd(a.claim, 1);  // the next one, ahead
      WMsg m;
      int nsteps = 0;
      if (!done) {
        const int64_t r = idx - base;
        const uint32_t at = __ballot_sync(0xffffffffu, items > 0 && before <= r && r < before + items);
        const int src = __ffs(at) - 1;
        m.b = win + src;
        m.ql = __shfl_sync(0xffffffffu, ql, src);
        m.kl = __shfl_sync(0xffffffffu, kl, src);
        m.qrow = __shfl_sync(0xffffffffu, qrow, src);
        const int np = __shfl_sync(0xffffffffu, parts, src);
        const int64_t local = r - __shfl_sync(0xffffffffu, before, src);
        m.part = (int)(local % np);
        const int64_t u = local / np;
        m.hk = (int)(u % a.KVN);
        m.j0 = (int)(u / a.KVN) * kUnitKeys;
        const int steps = unit_steps(a, m.ql, m.kl, m.j0, &m.qt0);
        m.s0 = m.part * a.chunk;
        m.s1 = min(steps, m.s0 + a.chunk);
        nsteps = m.s1 - m.s0;
        m.done = 0;
        if (nsteps <= 0) continue;  // past the unit's parts
      }
      const int ms = ucnt & 1;
      wait_or_abort(&mempty[ms], ((ucnt >> 1) & 1) ^ 1, a.err, misc);
      if (done) {
        if (lane == 0) {
          if (ok) {
            // the last CTA out re-arms the counter for the next execute
            __threadfence();
            if (atomicAdd(a.claim + 1, 1) == (int)gridDim.x - 1) {
              a.claim[0] = 0;
              a.claim[1] = 0;
            }
          }
          msg[ms].done = 1;
          mbar_arrive(&mfull[ms]);
        }
        break;
      }
      if (lane == 0) {
        msg[ms] = m;
        mbar_arrive(&mfull[ms]);
      }
      // the unit's K tiles
      const int ks = ucnt % KS;
      const int nrb = kUnitKeys / a.box_rows;        // boxes of a 128-byte column slice
      const int nslice = FP8 ? 1 : NSUB;
      uint32_t bytes = 0;
      for (int q = 0; q < nrb; ++q)
        if (m.j0 + q * a.box_rows < m.kl) bytes += (uint32_t)(nslice * a.box_rows * 128);
      wait_or_abort(&kempty[ks], ((ucnt / KS) & 1) ^ 1, a.err, misc);
      if (!stopped()) {
        if (lane == 0) mbar_arrive_expect_tx(&kfull[ks], bytes);
        __syncwarp();
        uint8_t* kdst = FP8 ? smem + Cfg::kOffCode + ks * 2 * Cfg::kCodeTile
                            : smem + Cfg::kOffK + ks * 2 * Cfg::kTile;
        for (int x = lane; x < nrb * nslice; x += 32) {
          const int rb = x / nslice, sub = x % nslice;
          const int j = m.j0 + rb * a.box_rows;
          if (j < m.kl) {
            int64_t row;
            if (c.bt) {
              const int pg = (int)(((uint64_t)(uint32_t)j * c.magic) >> c.shift);
              const int64_t blk = __ldg(c.bt + (int64_t)m.b * c.max_blocks + pg);
              row = (c.head_major ? blk * c.KVN + m.hk : blk) * c.bs + (j - pg * c.bs);
            } else {
              row = (int64_t)m.b * c.cap + j;
            }
            const int r = rb * a.box_rows;  // row of the unit
            uint8_t* dst = kdst + (r >> 7) * (FP8 ? Cfg::kCodeTile : Cfg::kTile) + sub * 16384 +
                           (r & 127) * 128;
            tma_load_2d(dst, &tk, &kfull[ks], (c.head_major ? 0 : m.hk * D) + sub * 64, (int)row);
          }
        }
      }
      ++ucnt;
      for (int s = m.s0; s < m.s1; ++s, ++qn) {
        const int qs = qn % QS;
        wait_or_abort(&qempty[qs], ((qn / QS) & 1) ^ 1, a.err, misc);
        if (stopped()) break;
        if (lane == 0) mbar_arrive_expect_tx(&qfull[qs], (uint32_t)Cfg::kTile);
        __syncwarp();
        const int h = m.hk * a.G + s % a.G;
        const int64_t row = m.qrow + (int64_t)(m.qt0 + s / a.G) * kQTile;
        if (lane < NSUB)
          tma_load_2d(smem + Cfg::kOffQ + qs * Cfg::kTile + lane * 16384, &tq, &qfull[qs],
                      h * D + lane * 64, (int)row);
      }
    }
    // after a time-out: the copies in flight land before the CTA ends
    if (stopped()) {
      for (int k = max(0, qn - QS); k < qn; ++k) mbar_wait(&qfull[k % QS], (k / QS) & 1, a.err);
      for (int k = max(0, ucnt - KS); k < ucnt; ++k) mbar_wait(&kfull[k % KS], (k / KS) & 1, a.err);
    }
  } else if (warp == 1) {
    // ============================ MMA issuer ============================
    if (lane == 0) {
      constexpr uint32_t kId = idesc_bf16(128, 128, false);
      const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + Cfg::kOffK), 16, 1024);
      const uint64_t qd0 = smem_desc_sw128(smem_u32(smem + Cfg::kOffQ), 16, 1024);
      constexpr uint64_t kUnits = Cfg::kTile >> 4;
      int ucnt = 0, n = 0;
      int sn[2] = {0, 0};  // S buffers filled per warpgroup
      while (true) {
        const int ms = ucnt & 1;
        wait_or_abort(&mfull[ms], (ucnt >> 1) & 1, a.err, misc);
        const WMsg m = msg[ms];
        mbar_arrive(&mempty[ms]);
        if (*abort_flag || m.done) break;
        const int ks = FP8 ? 0 : ucnt % Cfg::kKStages;
        if constexpr (FP8) wait_or_abort(kconv, ucnt & 1, a.err, misc);
        else wait_or_abort(&kfull[ks], (ucnt / Cfg::kKStages) & 1, a.err, misc);
        const int nwg = m.j0 + kKvTile < m.kl ? 2 : 1;
        for (int s = m.s0; s < m.s1; ++s, ++n) {
          const int qs = n % QS;
          wait_or_abort(&qfull[qs], (n / QS) & 1, a.err, misc);
          for (int w = 0; w < nwg; ++w) {
            const int sb = sn[w] % Cfg::kSBuf;
            wait_or_abort(&sempty[2 * w + sb], ((sn[w] / Cfg::kSBuf) & 1) ^ 1, a.err, misc);
            if (*abort_flag) break;
            tc_fence_after();
            const uint64_t kd = kd0 + (uint64_t)(2 * ks + w) * kUnits;
            const uint64_t qd = qd0 + (uint64_t)qs * kUnits;
            const uint32_t tS = tmem + 256 * w + 128 * sb;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              if constexpr (FP8)  // the halves of D apart
                mma_ss(tS + 128 * (kk >> 2), kd + off, qd + off, kId, (kk & 3) > 0);
              else
                mma_ss(tS, kd + off, qd + off, kId, kk > 0);
            }
            tc_commit(&sfull[2 * w + sb]);
            ++sn[w];
          }
          if (*abort_flag) break;
          tc_commit(&qempty[qs]);
        }
        if (*abort_flag) break;
        if constexpr (!FP8) tc_commit(&kempty[ks]);
        ++ucnt;
      }
      tc_commit(drain);
      mbar_wait(drain, 0, a.err);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ============================ lse rows ============================
    // -lse * log2(e) of a step's 128 query rows (rows past the sequence: -inf)
    int ucnt = 0, n = 0;
    while (true) {
      const int ms = ucnt & 1;
      wait_or_abort(&mfull[ms], (ucnt >> 1) & 1, a.err, misc);
      const WMsg m = msg[ms];
      __syncwarp();
      if (lane == 0) mbar_arrive(&mempty[ms]);
      ++ucnt;
      if (stopped() || m.done) break;
      for (int s = m.s0; s < m.s1; ++s, ++n) {
        const int ls = n % LS;
        const int h = m.hk * a.G + s % a.G;
        const int i0 = (m.qt0 + s / a.G) * kQTile;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + lane + 32 * k;
          v[k] = -INFINITY;
          if (i < m.ql)
            v[k] = -1.4426950408889634f *
                   __ldcg(a.lse + (a.cu_seqlens_q ? (m.qrow + i) * a.QN + h
                                                  : ((int64_t)m.b * a.QN + h) * a.S_q + i));
        }
        wait_or_abort(&lempty[ls], ((n / LS) & 1) ^ 1, a.err, misc);
        if (stopped()) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) lse_s[ls * 128 + lane + 32 * k] = v[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(&lfull[ls]);
      }
    }
  } else if (warp >= 4) {
    // ============================ epilogue ============================
    const int w = (warp - 4) >> 2;          // warpgroup: K tile of the unit
    const int row = tid - 128 - 128 * w;    // key of the tile = TMEM lane
    const uint32_t tS0 = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256 * w;
    const float sl = a.scale_log2;
    int ucnt = 0, n = 0, sn = 0;
    while (true) {
      const int ms = ucnt & 1;
      wait_or_abort(&mfull[ms], (ucnt >> 1) & 1, a.err, misc);
      const WMsg m = msg[ms];
      // (every warp of the warpgroup leaves together: the message's end, or the
      // abort flag, ORed over its threads)
      if (named_bar_or(2 + w, 128, m.done || *abort_flag)) break;
      if (row == 0) mbar_arrive(&mempty[ms]);
      const int j = m.j0 + kKvTile * w + row;
      const bool active = m.j0 + kKvTile * w < m.kl;
      float f0 = sl, f1 = sl;  // score factors of the key (FP8: of its two halves)
      if constexpr (FP8) {
        const int ks = ucnt % KS;
        wait_or_abort(&kfull[ks], (ucnt / KS) & 1, a.err, misc);
        // (the previous unit's products are done: its last S was awaited below)
        if (active) {
          const RowAt r = j < m.kl ? cache_row(c, m.b, m.hk, j) : RowAt{0, 0, false};
          const float2 sc = r.ok ? __ldg(reinterpret_cast<const float2*>(c.ks) + r.srow)
                                 : make_float2(0.f, 0.f);
          f0 = sl * sc.x;
          f1 = sl * sc.y;
          const uint8_t* src = smem + Cfg::kOffCode + (ks * 2 + w) * Cfg::kCodeTile;
          uint8_t* dst = smem + Cfg::kOffK + w * Cfg::kTile;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int ch = (q + row) & 7;  // a warp's rows start at different chunks
            const uint4 v = *reinterpret_cast<const uint4*>(src + sw128(row, ch));
            const uint32_t cw[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t lo, hi;
              e4m3x4_to_f16x2x2(cw[k], lo, hi);
              const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&lo));
              const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              o[2 * k] = pack_bf16(fl.x, fl.y);
              o[2 * k + 1] = pack_bf16(fh.x, fh.y);
            }
            // elements 16 ch .. 16 ch + 15: slice ch / 4, chunks 2 (ch % 4) and + 1
            uint8_t* d = dst + (ch >> 2) * 16384;
            *reinterpret_cast<uint4*>(d + sw128(row, 2 * (ch & 3))) =
                make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(d + sw128(row, 2 * (ch & 3) + 1)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async_smem();
        }
        named_bar_sync(2 + w, 128);
        if (row == 0) {
          mbar_arrive(&kempty[ks]);
          mbar_arrive(kconv);
        }
      }
      int lo, hi;
      rows_of_key(a, m.ql, m.kl, j, &lo, &hi);
      const uint8_t* mrow = a.mask ? a.mask + (int64_t)m.b * a.mask_bstride + j : nullptr;
      float sum = 0.f;
      for (int s = m.s0; s < m.s1; ++s, ++n) {
        const int ls = n % LS;
        wait_or_abort(&lfull[ls], (n / LS) & 1, a.err, misc);
        if (active) {
          const int sb = sn % Cfg::kSBuf;
          wait_or_abort(&sfull[2 * w + sb], (sn / Cfg::kSBuf) & 1, a.err, misc);
          ++sn;
          tc_fence_after();
          const int i0 = (m.qt0 + s / a.G) * kQTile;
          const int c0 = lo - i0, c1 = hi - i0;  // columns c0 .. c1 are seen
          const bool full = __all_sync(0xffffffffu, c0 <= 0 && c1 >= 127) && !a.mask;
          const bool none = __all_sync(0xffffffffu, c1 < c0 || c1 < 0 || c0 > 127);
          const float* ls4 = lse_s + ls * 128;
          const uint32_t tS = tS0 + 128 * sb;
          float2 acc[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
          if (!none) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t v[64], u[FP8 ? 64 : 1];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                tmem_ld32(tS + 64 * half + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * k]));
                if constexpr (FP8)
                  tmem_ld32(tS + 128 + 64 * half + 32 * k,
                            *reinterpret_cast<uint32_t(*)[32]>(&u[32 * k]));
              }
              tmem_wait_ld();
              const float2 f0v = make_float2(f0, f0), f1v = make_float2(f1, f1);
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                const float4 nl = *reinterpret_cast<const float4*>(ls4 + 64 * half + e);
                float2 x[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float2 t = k ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y);
                  if constexpr (FP8)
                    t = w_ffma2(make_float2(__uint_as_float(u[e + 2 * k]),
                                            __uint_as_float(u[e + 2 * k + 1])), f1v, t);
                  t = w_ffma2(make_float2(__uint_as_float(v[e + 2 * k]),
                                          __uint_as_float(v[e + 2 * k + 1])), f0v, t);
                  x[k] = make_float2(w_ex2(t.x), w_ex2(t.y));
                }
                if (!full) {
                  float p[4] = {x[0].x, x[0].y, x[1].x, x[1].y};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const int col = 64 * half + e + k;
                    bool see = col >= c0 && col <= c1;
                    if (see && mrow) see = __ldg(mrow + (int64_t)(i0 + col) * a.mask_rstride) == 0;
                    if (!see) p[k] = 0.f;
                  }
                  x[0] = make_float2(p[0], p[1]);
                  x[1] = make_float2(p[2], p[3]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float2& s2 = acc[(e / 2 + k) & 3];
                  s2.x += x[k].x;
                  s2.y += x[k].y;
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[2 * w + sb]);
          sum += ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) +
                 ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&lempty[ls]);
      }
      ++ucnt;
      if (active && j < m.kl && !*abort_flag)
        a.partials[((int64_t)m.part * a.B * a.KVN + (int64_t)m.b * a.KVN + m.hk) * a.S_kv + j] = sum;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// w_out = w_in + the parts of each key, in order.
__global__ void __launch_bounds__(256) key_weights_fold_kernel(const WeightsArgs a, int per_pair) {
  pdl_wait();
  if (a.plan && !plan_ok(a)) return;
  const int pair = blockIdx.x / per_pair, b = pair / a.KVN;
  int64_t qrow;
  int ql, kl;
  w_lengths(a, b, &qrow, &ql, &kl);
  const int64_t stride = (int64_t)a.B * a.KVN * a.S_kv;
  for (int j = (blockIdx.x % per_pair) * 256 + threadIdx.x; j < kl; j += per_pair * 256) {
    int qt0;
    const int parts = a.plan ? unit_parts(a, unit_steps(a, ql, kl, j / kUnitKeys * kUnitKeys, &qt0)) : 0;
    const int64_t at = (int64_t)pair * a.stride + j;
    float w = 0.f;
    const float* p = a.partials + (int64_t)pair * a.S_kv + j;
    for (int k = 0; k < parts; ++k) w += __ldcg(p + k * stride);
    a.w_out[at] = (a.w_in ? a.w_in[at] : 0.f) + w;
  }
}

template <int D, bool FP8>
cudaError_t launch_t(const WeightsArgs& a, const CacheView& c, const CUtensorMap& tq,
                     const CUtensorMap& tk, cudaStream_t s) {
  using Cfg = WeightsCfg<D, FP8>;
  auto kern = key_weights_kernel<D, FP8>;
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
  return launch_pdl(kern, dim3(a.num_ctas), dim3(kWThreads), Cfg::kSmem, s, a, c, tq, tk);
}

}  // namespace

// Steps per part: at least 8 (a part loads 64 KB of K; a step takes about 1 us),
// and few enough parts that the partial sums stay below 16 times the weights.
int weights_chunk(int G, int64_t max_q, int* parts) {
  const int64_t steps = (max_q + kQTile - 1) / kQTile * G;
  const int chunk = (int)std::max<int64_t>(8, (steps + 15) / 16);
  *parts = (int)std::max<int64_t>(1, (steps + chunk - 1) / chunk);
  return chunk;
}

cudaError_t launch_key_weights_fold(const WeightsArgs& a, cudaStream_t s) {
  const int pairs = a.B * a.KVN;
  if (a.S_kv == 0) return cudaSuccess;
  const int per_pair = (int)std::max<int64_t>(
      1, std::min<int64_t>((a.S_kv + 255) / 256, (int64_t)a.num_ctas * 8 / pairs));
  return launch_pdl(key_weights_fold_kernel, dim3(pairs * per_pair), dim3(256), 0, s, a, per_pair);
}

cudaError_t launch_key_weights(const WeightsArgs& a, const fia_kv_cache& cache,
                               const CUtensorMap& tq, const CUtensorMap& tk, cudaStream_t s) {
  const CacheView c = cache_view(cache);
  cudaError_t e;
  if (c.fp8) e = launch_t<128, true>(a, c, tq, tk, s);
  else if (a.D == 64) e = launch_t<64, false>(a, c, tq, tk, s);
  else e = launch_t<128, false>(a, c, tq, tk, s);
  return e == cudaSuccess ? launch_key_weights_fold(a, s) : e;
}

}  // namespace fia
