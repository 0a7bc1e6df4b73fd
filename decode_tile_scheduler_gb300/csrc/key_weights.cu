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
// head) pairs that see some of its keys.  All steps of the call form one list, of
// which every CTA takes an equal range; a unit that ranges cut has several parts.
// (With units cut in parts of 4 or 8 steps that CTAs claimed one by one, each CTA
// held one or two claims ahead for its loads, and on four prompts of up to 2048
// rows the slowest had 20 steps where the mean was 16.)  A unit's two K tiles stay
// in shared memory while the Q tiles stream past them; each K tile belongs to one
// epilogue warpgroup, so a Q tile in shared memory serves 2 x 128 keys (with one K
// tile the reads of Q from L2 alone would be 32 KB per 512 cycles of products, on
// 152 SMs above the L2's rate).  The sums of a unit's parts go to rows of the
// workspace, and key_weights_fold_kernel adds them in order: no atomics, the same
// bits every time.
//
// FP8 keys: E4M3 codes are bf16 values as they are, so the K tiles are widened
// to bf16 without their scales, the two 64-element halves of D accumulate apart,
// and a key's two scales multiply the two sums of its lane: no rounding of K.
//
// Bound: a step of 256 keys x 128 rows is 1024 cycles on the tensor core (D = 128)
// and as many on the MUFU (an ex2 per key, row and head), and takes 1.2 to 1.4 us,
// 2300 to 2700 cycles: one prompt of 8192 rows with 32 heads 312 us for 222 steps
// a CTA, 44 % of the tensor core's and of the MUFU's cycles.  The issue of a step's
// products alone then takes 0.88 us, where they run in 0.53 us by themselves:
// products and reads of their results share TMEM and shared memory.  Not kept, of
// the same time or slower (312 us here): both K tiles to each of two warpgroups,
// 64 rows each, so that an lse is read once for two keys (309 us; FP8 433 -> 478);
// four warpgroups of a tile and 64 rows each (360 us), or of both tiles and 32
// rows each (323 us).
#include <algorithm>
#include <atomic>

#include "kv_cache.cuh"
#include "tcgen05.cuh"

namespace fia {

namespace {

constexpr int kWThreads = 384;
constexpr int kUnitKeys = 2 * kKvTile;
constexpr int kMaxParts = 16;  // parts of a unit, at most

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
  // mfull[2] mempty[2] kfull[2] kempty[2] kconv[2] qfull[QS] qempty[QS] lfull[LS]
  // lempty[LS] sfull[2][2] sempty[2][2] drain
  static constexpr int kBars = 10 + 2 * kQStages + 2 * kLseStages + 8 + 1;
  static constexpr int kOffMsg = kOffBar + 8 * kBars;
  static constexpr int kOffMisc = kOffMsg + 2 * 64;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

struct WMsg {
  int b, hk, j0, kl, ql, qt0, s0, s1;  // steps s0 .. s1 - 1 of the unit
  int part, parts, done;               // this part of the unit, parts of the unit
  int64_t qrow;                        // first token row of the sequence
};
static_assert(sizeof(WMsg) <= 64, "message slot");

// Sequences whose steps are summed at a time, and how many such windows there
// can be (fia.h: at most 65536 sequences).
constexpr int kSeqWindow = 4096, kSeqWindows = 16;

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
__device__ __forceinline__ float2 w_fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float w_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// n / d for n >= 0, d > 0, in 32 bits where they allow (a 64-bit division takes
// ten times as long, and a CTA's first loads wait for some).
__device__ __forceinline__ int64_t div_int(int64_t n, int64_t d) {
  return ((uint64_t)(n | d) >> 32) == 0 ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}
__device__ __forceinline__ int64_t div_up(int64_t n, int64_t d) { return div_int(n + d - 1, d); }

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
  uint64_t* qfull = kconv + 2;
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
    // (a barrier per warpgroup, and only units with keys of its own count: a
    // warpgroup without keys runs ahead of the other)
    mbar_init(&kconv[0], 1);
    mbar_init(&kconv[1], 1);
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
  // the attention is done: its lse, and the plan before it.  (Waiting for the lse alone,
  // with the attention letting this kernel start on SMs that have finished, made four
  // prompts slower, 103 -> 105 us a call.)
  pdl_wait();
  const bool ok = plan_ok(a);
  volatile int* abort_flag = misc;

  // Every CTA takes an equal range of the list of all steps (sequence, 256 keys,
  // KV head, step).  The sums over a sequence, for finding a range's start, are
  // formed by all CTAs alike, a warp per sequence and a lane per 256 keys.
  int64_t* win_sum = reinterpret_cast<int64_t*>(smem + Cfg::kOffQ);
  int64_t* seq_sum = win_sum + kSeqWindows;
  const int nwin = (a.B + kSeqWindow - 1) / kSeqWindow;
  auto sum_window = [&](int w0) {
    const int nb = min(kSeqWindow, a.B - w0 * kSeqWindow);
    for (int i = warp; i < nb; i += kWThreads / 32) {
      int64_t qrow, n = 0;
      int ql, kl, t0;
      w_lengths(a, w0 * kSeqWindow + i, &qrow, &ql, &kl);
      for (int j0 = lane * kUnitKeys; j0 < kl; j0 += 32 * kUnitKeys)
        n += unit_steps(a, ql, kl, j0, &t0);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane == 0) seq_sum[i] = n * a.KVN;
    }
    __syncthreads();
    if (warp == 0) {
      int64_t n = 0;
      for (int i = lane; i < nb; i += 32) n += seq_sum[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane == 0) win_sum[w0] = n;
    }
    __syncthreads();
  };
  int64_t all_steps = 0, range = 1;
  if (ok) {
    for (int w0 = 0; w0 < nwin; ++w0) {
      sum_window(w0);
      all_steps += win_sum[w0];
    }
    // no shorter than a.chunk (a part has its K tiles to load, and a unit's
    // longest has to fit kMaxParts parts)
    range = max((int64_t)a.chunk, div_up(all_steps, gridDim.x));
    if (nwin > 1) {  // back to the window of this CTA's start
      int64_t before = 0;
      int w0 = 0;
      while (w0 < nwin - 1 && before + win_sum[w0] <= range * (int64_t)blockIdx.x)
        before += win_sum[w0++];
      sum_window(w0);
    }
  }
  // (the same answer for a whole warp)
  auto stopped = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };

  // (the other warps only meet the producer: it reads the sums, then fills the
  // Q stages they lie in)
  if (warp != 0) named_bar_sync(4, kWThreads);

  if (warp == 0) {
    // ============================ producer ============================
    // The CTA's range of the list of all steps, unit by unit.
    int ucnt = 0, qn = 0;
    int b = 0, kt = 0, hk = 0, ql = 0, kl = 0, nkt = 0, steps = 0, qt0 = 0;
    int64_t qrow = 0, at = range * (int64_t)blockIdx.x, s = 0;  // place in the list, in the unit
    const int64_t end = min(at + range, all_steps);
    // the first unit with steps at or behind tile pair `from` of the sequence
    auto next_kt = [&](int from) {
      for (int base = from; base < nkt; base += 32) {
        int t0 = 0;
        const int n = base + lane < nkt ? unit_steps(a, ql, kl, (base + lane) * kUnitKeys, &t0) : 0;
        const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
        if (some) {
          const int src = __ffs(some) - 1;
          kt = base + src;
          steps = __shfl_sync(0xffffffffu, n, src);
          qt0 = __shfl_sync(0xffffffffu, t0, src);
          return true;
        }
      }
      return false;
    };
    // the first sequence with steps at or behind `from`
    auto next_seq = [&](int from) {
      for (int base = from; base < a.B; base += 32) {
        int l = 0, k = 0;
        int64_t r = 0;
        if (base + lane < a.B) w_lengths(a, base + lane, &r, &l, &k);
        uint32_t some = __ballot_sync(0xffffffffu, l > 0 && k > 0);
        while (some) {
          const int src = __ffs(some) - 1;
          some &= some - 1;
          b = base + src;
          ql = __shfl_sync(0xffffffffu, l, src);
          kl = __shfl_sync(0xffffffffu, k, src);
          qrow = __shfl_sync(0xffffffffu, r, src);
          nkt = (kl + kUnitKeys - 1) / kUnitKeys;
          if (next_kt(0)) return true;
        }
      }
      return false;
    };
    bool more = at < end;
    if (more) {
      // sequence of the range's first step: window, then the prefix inside it
      int64_t before = 0;
      int w0 = 0;
      while (w0 < nwin - 1 && before + win_sum[w0] <= at) before += win_sum[w0++];
      const int nb = min(kSeqWindow, a.B - w0 * kSeqWindow);
      for (int base = 0; base < nb; base += 32) {
        const int64_t n = base + lane < nb ? seq_sum[base + lane] : 0;
        int64_t x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, before + x > at);
        if (here) {
          const int src = __ffs(here) - 1;
          b = w0 * kSeqWindow + base + src;
          before += __shfl_sync(0xffffffffu, x - n, src);
          break;
        }
        before += __shfl_sync(0xffffffffu, x, 31);
      }
      more = next_seq(b);
      // then its unit: a lane per 256 keys, 32 units at a time
      for (int base = 0; more; base += 32) {
        int t0 = 0;
        const int n = base + lane < nkt ? unit_steps(a, ql, kl, (base + lane) * kUnitKeys, &t0) : 0;
        int64_t x = (int64_t)n * a.KVN;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, before + x > at);
        if (here) {
          const int src = __ffs(here) - 1;
          kt = base + src;
          steps = __shfl_sync(0xffffffffu, n, src);
          qt0 = __shfl_sync(0xffffffffu, t0, src);
          before += __shfl_sync(0xffffffffu, x, src) - (int64_t)steps * a.KVN;
          hk = (int)div_int(at - before, steps);
          s = at - before - (int64_t)hk * steps;
          break;
        }
        before += __shfl_sync(0xffffffffu, x, 31);
        more = base + 32 < nkt;
      }
    }
    named_bar_sync(4, kWThreads);  // the sums, in the Q stages' place, have been read
    fence_proxy_async_smem();      // (before the copies that overwrite them)
    while (true) {
      const bool done = stopped() || !more || at >= end;
      WMsg m;
      const int ms = ucnt & 1;
      wait_or_abort(&mempty[ms], ((ucnt >> 1) & 1) ^ 1, a.err, misc);
      if (done) {
        if (lane == 0) {
          msg[ms].done = 1;
          mbar_arrive(&mfull[ms]);
        }
        break;
      }
      m.b = b;
      m.hk = hk;
      m.j0 = kt * kUnitKeys;
      m.kl = kl;
      m.ql = ql;
      m.qt0 = qt0;
      m.qrow = qrow;
      m.s0 = (int)s;
      m.s1 = (int)min((int64_t)steps, s + (end - at));
      const int64_t first = div_int(at - s, range);  // the CTA of the unit's first part
      m.part = (int)(blockIdx.x - first);
      m.parts = (int)(div_int(at - s + steps - 1, range) - first + 1);
      m.done = 0;
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
              // (a page outside the pool: a box before the map's rows, zeros)
              row = blk < 0 || blk >= c.num_blocks
                        ? -kKvTile
                        : (c.head_major ? blk * c.KVN + m.hk : blk) * c.bs + (j - pg * c.bs);
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
      for (int st = m.s0; st < m.s1; ++st, ++qn) {
        const int qs = qn % QS;
        wait_or_abort(&qempty[qs], ((qn / QS) & 1) ^ 1, a.err, misc);
        if (stopped()) break;
        if (lane == 0) mbar_arrive_expect_tx(&qfull[qs], (uint32_t)Cfg::kTile);
        __syncwarp();
        const int h = m.hk * a.G + st % a.G;
        const int64_t row = m.qrow + (int64_t)(m.qt0 + st / a.G) * kQTile;
        if (lane < NSUB)
          tma_load_2d(smem + Cfg::kOffQ + qs * Cfg::kTile + lane * 16384, &tq, &qfull[qs],
                      h * D + lane * 64, (int)row);
      }
      // on to the next unit: the next KV head, 256 keys, sequence
      at += m.s1 - m.s0;
      s = 0;
      if (at < end && ++hk == a.KVN) {
        hk = 0;
        more = next_kt(kt + 1) || next_seq(b + 1);
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
      int kc[2] = {0, 0};  // (FP8) K tiles taken per warpgroup
      while (true) {
        const int ms = ucnt & 1;
        wait_or_abort(&mfull[ms], (ucnt >> 1) & 1, a.err, misc);
        const WMsg m = msg[ms];
        mbar_arrive(&mempty[ms]);
        if (*abort_flag || m.done) break;
        const int ks = FP8 ? 0 : ucnt % Cfg::kKStages;
        const int nwg = m.j0 + kKvTile < m.kl ? 2 : 1;
        if constexpr (FP8) {
          for (int w = 0; w < nwg; ++w) {
            wait_or_abort(&kconv[w], kc[w] & 1, a.err, misc);
            ++kc[w];
          }
        } else {
          wait_or_abort(&kfull[ks], (ucnt / Cfg::kKStages) & 1, a.err, misc);
        }
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
      auto fetch = [&](int s, float (&v)[4]) {
        const int h = m.hk * a.G + s % a.G;
        const int i0 = (m.qt0 + s / a.G) * kQTile;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + lane + 32 * k;
          v[k] = INFINITY;
          if (s < m.s1 && i < m.ql)
            v[k] = __ldcg(a.lse + (a.cu_seqlens_q ? (m.qrow + i) * a.QN + h
                                                  : ((int64_t)m.b * a.QN + h) * a.S_q + i));
        }
      };
      float v[4], next[4];
      fetch(m.s0, v);
      for (int s = m.s0; s < m.s1; ++s, ++n) {
        const int ls = n % LS;
        fetch(s + 1, next);  // in flight while this step's values are stored
        wait_or_abort(&lempty[ls], ((n / LS) & 1) ^ 1, a.err, misc);
        if (stopped()) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          lse_s[ls * 128 + lane + 32 * k] = -1.4426950408889634f * v[k];
          v[k] = next[k];
        }
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
          if (active) mbar_arrive(&kconv[w]);
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
          const float* ls4 = lse_s + ls * 128;
          const uint32_t tS = tS0 + 128 * sb;
          float2 acc[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
          const float2 f0v = make_float2(f0, f0), f1v = make_float2(f1, f1);
          auto release = [&]() {  // the S buffer, once its values are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sempty[2 * w + sb]);
          };
          const bool full = __all_sync(0xffffffffu, c0 <= 0 && c1 >= 127) && !a.mask;
          if (!FP8 && full) {
            // every pair is seen: the row's 128 scores in registers with one
            // wait, the buffer free for the next product at once
            uint32_t v[128];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              tmem_ld32(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * q]));
            tmem_wait_ld();
            release();
#pragma unroll
            for (int e = 0; e < 128; e += 4) {
              const float4 nl = *reinterpret_cast<const float4*>(ls4 + e);
              const float2 t0 = w_ffma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                        f0v, make_float2(nl.x, nl.y));
              const float2 t1 = w_ffma2(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                        f0v, make_float2(nl.z, nl.w));
              acc[(e >> 1) & 3] = w_fadd2(acc[(e >> 1) & 3], make_float2(w_ex2(t0.x), w_ex2(t0.y)));
              acc[((e >> 1) + 1) & 3] =
                  w_fadd2(acc[((e >> 1) + 1) & 3], make_float2(w_ex2(t1.x), w_ex2(t1.y)));
            }
          } else {
            // 32 columns at a time (a rolled loop: unrolled over all 128, the
            // instructions no longer fit their cache)
            const uint32_t span = (uint32_t)(c1 - c0);
            const bool any = c1 >= c0;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              // on a diagonal most of a warp's 32 x 32 squares are seen whole or
              // not at all
              if (!__any_sync(0xffffffffu, any && c0 <= 32 * q + 31 && c1 >= 32 * q)) continue;
              const bool whole = __all_sync(0xffffffffu, c0 <= 32 * q && c1 >= 32 * q + 31) && !a.mask;
              uint32_t v[32], u[FP8 ? 32 : 1];
              tmem_ld32(tS + 32 * q, v);
              if constexpr (FP8) tmem_ld32(tS + 128 + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&u));
              tmem_wait_ld();
              const float4* nl4 = reinterpret_cast<const float4*>(ls4 + 32 * q);
              float x[32];  // exponents, log2 units
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 nl = nl4[e / 4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float2 t = k ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y);
                  if constexpr (FP8)
                    t = w_ffma2(make_float2(__uint_as_float(u[e + 2 * k]),
                                            __uint_as_float(u[e + 2 * k + 1])), f1v, t);
                  t = w_ffma2(make_float2(__uint_as_float(v[e + 2 * k]),
                                          __uint_as_float(v[e + 2 * k + 1])), f0v, t);
                  x[e + 2 * k] = t.x;
                  x[e + 2 * k + 1] = t.y;
                }
              }
              if (!whole) {  // pairs outside the row interval, or hidden by the mask
                uint32_t hid = 0;
                if (a.mask) {
#pragma unroll 4
                  for (int e = 0; e < 32; ++e) {
                    const int col = 32 * q + e;
                    if (any && (uint32_t)(col - c0) <= span &&
                        __ldg(mrow + (int64_t)(i0 + col) * a.mask_rstride) != 0)
                      hid |= 1u << e;
                  }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!any || (uint32_t)(32 * q + e - c0) > span || ((hid >> e) & 1u))
                    x[e] = -INFINITY;
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float2& s2 = acc[(e / 2) & 3];
                s2 = w_fadd2(s2, make_float2(w_ex2(x[e]), w_ex2(x[e + 1])));
              }
            }
            release();
          }
          sum += ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) +
                 ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&lempty[ls]);
      }
      ++ucnt;
      if (active && j < m.kl && !*abort_flag) {
        const int64_t pair = (int64_t)m.b * a.KVN + m.hk;
        if (m.parts == 1) {  // the whole unit: nothing to fold
          const int64_t o = pair * a.stride + j;
          a.w_out[o] = (a.w_in ? a.w_in[o] : 0.f) + sum;
        } else {
          a.partials[((int64_t)m.part * a.B * a.KVN + pair) * a.S_kv + j] = sum;
        }
        if (m.part == 0 && w == 0 && row == 0)
          a.nparts[pair * a.units_max + m.j0 / kUnitKeys] = m.parts;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// w_out = w_in + the parts of each key, in order, where a unit had several; and
// w_in where no row sees any of a unit's keys.
__global__ void __launch_bounds__(256) key_weights_fold_kernel(const WeightsArgs a, int per_pair) {
  pdl_wait();
  if (a.plan && !plan_ok(a)) return;
  const int pair = blockIdx.x / per_pair, b = pair / a.KVN;
  int64_t qrow;
  int ql, kl;
  w_lengths(a, b, &qrow, &ql, &kl);
  const int64_t stride = (int64_t)a.B * a.KVN * a.S_kv;
  for (int j = (blockIdx.x % per_pair) * 256 + threadIdx.x; j < kl; j += per_pair * 256) {
    int qt0, parts = 0;
    if (a.plan && unit_steps(a, ql, kl, j / kUnitKeys * kUnitKeys, &qt0) > 0)
      parts = min(__ldcg(a.nparts + (int64_t)pair * a.units_max + j / kUnitKeys), kMaxParts);
    if (parts == 1) continue;  // written by its part
    const int64_t at = (int64_t)pair * a.stride + j;
    float w = 0.f, x[kMaxParts];
    const float* p = a.partials + (int64_t)pair * a.S_kv + j;
#pragma unroll
    for (int k = 0; k < kMaxParts; ++k) x[k] = k < parts ? __ldcg(p + k * stride) : 0.f;
#pragma unroll
    for (int k = 0; k < kMaxParts; ++k) w += x[k];
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

// The fewest steps per part: 2 (a part loads 64 KB of K, and a step takes about
// 1.2 us: one prompt of 34 rows over 6 keys 30.5 us with 4, 28.1 us with 2), and enough
// that a unit of queries of max_q rows, cut anywhere, has at most kMaxParts parts.
int weights_chunk(int G, int64_t max_q) {
  const int64_t steps = (max_q + kQTile - 1) / kQTile * G;
  return (int)std::max<int64_t>(2, (steps + kMaxParts - 2) / (kMaxParts - 1));
}
int64_t weights_units(int64_t capacity) { return (capacity + kUnitKeys - 1) / kUnitKeys; }
int weights_parts() { return kMaxParts; }

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
