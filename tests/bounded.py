"""The bounded cache's operators in 64 bits, straight from their definitions, and
the tolerances their outputs are held to."""
import math

import numpy as np
import torch

import fia_inputs as fi

HALF_BF16, HALF_FP16, HALF_FP32 = (torch.finfo(t).eps / 2
                                   for t in (torch.bfloat16, torch.float16, torch.float32))


def cache_values(pool, scale, table, b, n, block, head_major):
    """Keys 0 .. n-1 of sequence b in 64 bits, [n, KVN, D]."""
    j = torch.arange(n)
    if table is None:
        x = pool[b, :n]
        sc = None if scale is None else scale[b, :, :n].permute(1, 0, 2)
    else:
        page, row = table[b, j // block].long(), j % block
        x = pool[page, :, row] if head_major else pool[page, row]
        sc = None if scale is None else scale[page, :, row]
    if scale is None:
        return x.double()
    v = x.view(torch.float8_e4m3fn).float().double()
    return (v.unflatten(-1, (-1, 64)) * sc.double()[..., None]).flatten(-2)


def visible(p, b, ql, kl):
    """[ql, kl] whether row i sees key j."""
    i, j = torch.arange(ql)[:, None], torch.arange(kl)[None]
    pos = i + (0 if p.mask_mode == fi.MASK_LEFT_UP_CAUSAL else kl - ql)
    if p.mask_mode in (fi.MASK_LEFT_UP_CAUSAL, fi.MASK_RIGHT_DOWN_CAUSAL):
        return j <= pos
    if p.mask_mode == fi.MASK_BAND:
        return (j <= pos + p.next_tokens) & ((j >= pos - p.pre_tokens) | (j < p.first_tokens))
    if p.atten_mask is not None:
        return p.atten_mask[min(b, p.atten_mask.shape[0] - 1), :ql, :kl] == 0
    return torch.ones(ql, kl, dtype=torch.bool)


def attention(prob):
    """Per sequence: out [ql, QN, D], lse [ql, QN], key weights [KVN, kl], and the
    sizes the tolerances go by: sum_j w_j |v_j| for each output, the largest sum
    of |q_d k_d scale| over the visible pairs."""
    p = prob.to("cpu")
    got, t0, G = [], 0, p.QN // p.KVN
    for b in range(p.B):
        ql, kl = p.q_lens[b], p.kv_lens[b]
        q = (p.q[t0:t0 + ql] if p.layout == fi.LAYOUT_TND else p.q[b]).double()
        t0 += ql
        k, v = (cache_values(c, s, p.block_table, b, kl, p.block_size, p.kv_layout == 1)
                for c, s in ((p.k_cache, p.k_scale), (p.v_cache, p.v_scale)))
        see = visible(p, b, ql, kl)
        some = see.any(1) if kl else torch.zeros(ql, dtype=torch.bool)
        used = see.any(0)
        k, v = torch.where(used[:, None, None], k, 0), torch.where(used[:, None, None], v, 0)
        out = torch.zeros(ql, p.QN, p.D, dtype=torch.float64)
        mag = torch.zeros_like(out)
        lse = torch.full((ql, p.QN), math.inf, dtype=torch.float64)
        w = torch.zeros(p.KVN, kl, dtype=torch.float64)
        A = 0.0
        for h in range(p.QN if kl and ql else 0):
            x = (q[:, h] @ k[:, h // G].T * p.scale).masked_fill(~see, -math.inf)
            A = max(A, float(((q[:, h].abs() @ k[:, h // G].abs().T) * abs(p.scale))[see].max())
                    if see.any() else 0.0)
            if p.sinks is not None:
                x = torch.cat([x, p.sinks[h].double().expand(ql, 1)], 1)
            l = torch.logsumexp(x, 1)
            pr = torch.exp(x - torch.where(some, l, 0)[:, None])[:, :kl]
            pr[~some] = 0
            out[:, h], mag[:, h] = pr @ v[:, h // G], pr @ v[:, h // G].abs()
            lse[some, h] = l[some]
            w[h // G] += pr.sum(0)
        got.append((out, lse, w, mag, A))
    return got


def lse_tolerance(prob, A, n):
    """How far a score minus its row's lse may be off: the products' sums take
    D/16 steps in fp32, each off by at most a truncation (twice the half step)
    of a partial sum below A; the exponent's argument and the lse are rounded a
    few times (|x| <= 1.45 A, up to four half steps, and the exponential's own
    2^-22); the sum of n terms is off by at most a half step each.  Prompts over
    an FP8 cache run on K rounded to fp16."""
    t = prob.D / 16 * 2 * HALF_FP32 * A + 4 * HALF_FP32 * (1.45 * A + math.log(n + 1) + 2) \
        + 2 ** -22 + n * HALF_FP32
    if prob.kv_dtype == fi.KV_FP8_E4M3 and max(prob.q_lens) > 16:
        t += HALF_FP16 * A
    return t


def check_attention(prob, out, lse, weights=None, weights_in=None):
    """The call's outputs against attention(prob)."""
    ref, t0, worst = attention(prob), 0, 0.0
    out, lse = out.cpu().double(), lse.cpu().double()
    for b, (o, l, w, mag, A) in enumerate(ref):
        ql, kl = prob.q_lens[b], prob.kv_lens[b]
        if prob.layout == fi.LAYOUT_TND:
            go, gl = out[t0:t0 + ql], lse[t0:t0 + ql, :, 0]
        else:
            go, gl = out[b], lse[b, :, :, 0].T
        t0 += ql
        tl = lse_tolerance(prob, A, kl)
        # P is rounded to 16 bits before P V (half a step of bf16, each on a term
        # of mag), a split's weights and the output's rounding on top
        to = 1.01 * HALF_BF16 * (mag + o.abs()) + 2 * tl * mag + 1e-30
        if prob.kv_dtype == fi.KV_FP8_E4M3:  # V (prompts) or P times its scale in fp16
            to = to + 2 * HALF_FP16 * mag
        none = torch.isinf(l)
        assert torch.equal(torch.isinf(gl) & (gl > 0), none), f"sequence {b}: rows without keys"
        assert torch.all(go[none] == 0), f"sequence {b}: a row without keys is not 0"
        assert torch.isfinite(go).all()
        assert torch.all((go - o).abs() <= to), \
            f"sequence {b}: out off by {float(((go - o).abs() / to).max()):.3g} of its tolerance"
        assert torch.all((gl - l)[~none].abs() <= tl), \
            f"sequence {b}: lse off by {float((gl - l)[~none].abs().max()):.3g} of {tl:.3g}"
        if weights is not None:
            gw = weights[b, :, :kl].cpu().double()
            w0 = torch.zeros_like(w) if weights_in is None else weights_in[b, :, :kl].cpu().double()
            rows = max(1, ql * prob.QN // prob.KVN)
            # (the sum over rows and heads and the addition round half a step each)
            tw = w * (2 * tl + rows * HALF_FP32) + 2 * HALF_FP32 * (w + w0.abs()) + 1e-30
            assert torch.all((gw - (w0 + w)).abs() <= tw), \
                f"sequence {b}: weights off by {float(((gw - w0 - w).abs() / tw).max()):.3g}"


def keep_of(weights, positions, n, budget, first, recent, seen):
    """Which of a head's n slots stay: protected positions, then larger weights
    (NaN below every number), then lower slots."""
    w = np.asarray(weights, np.float64)[:n]
    pos = np.arange(n) if positions is None else np.asarray(positions)[:n]
    safe = (pos < first) | (pos >= seen - recent)
    nan = np.isnan(w)
    best = np.lexsort((np.arange(n), np.where(safe | nan, 0.0, -w), ~safe & nan, ~safe))
    kept = np.zeros(n, bool)
    kept[best[:budget]] = True
    return kept


def evicted(weights, positions, lens, budget, first, recent, seen):
    """For every (sequence, head): (new length, holes, tails)."""
    got = []
    for b, n in enumerate(lens):
        m = min(n, budget)
        for h in range(weights.shape[1]):
            kept = keep_of(weights[b, h], None if positions is None else positions[b, h], n, budget,
                           first, recent, n if seen is None else seen[b])
            got.append((b, h, m, np.nonzero(~kept[:m])[0], m + np.nonzero(kept[m:])[0]))
    return got


def e4m3(x):
    """fp32 values (x / scale as fp32 rounds it) to E4M3 codes, nearest even,
    saturated; from the format's definition."""
    x = np.asarray(x, np.float32).astype(np.float64)
    a = np.where(np.isnan(x), 0.0, np.minimum(np.abs(x), 448.0))
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    e = np.maximum(e, -6)
    m = np.rint(a / 2.0 ** (e - 3))
    e, m = np.where(m >= 16, e + 1, e), np.where(m >= 16, 8, m)
    code = np.where(m < 8, m, (e + 7) * 8 + (m - 8)).astype(np.uint8)
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | (np.signbit(x).astype(np.uint8) << 7)).astype(np.uint8)


def quantised(x):
    """bf16 [..., D] as codes and scales: scale = amax / 448 (1 for zeros), NaN
    left out of amax, infinities as the largest bf16 value; fp32 divisions."""
    t = x.float().unflatten(-1, (-1, 64)).numpy()
    big = np.float32(torch.finfo(torch.bfloat16).max)
    amax = np.minimum(np.where(np.isnan(t), 0, np.abs(t)).max(-1), big)
    scale = np.where(amax > 0, amax / np.float32(448), np.float32(1)).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        y = (t / scale[..., None]).astype(np.float32)
    return e4m3(y).reshape(x.shape), scale
