"""The operators of a bounded KV cache, as cases to measure and to check.

A serving program that keeps a paged KV cache within a budget makes four
calls: it appends the keys and values of new tokens, attends through a sliding
window whose first few tokens stay visible, attends while adding up how much
weight every cached key received, and evicts the keys that received least.
Each case is one such call.  With `own` false, run() computes it in elementary
torch operations in 32 bits; with `own` true, through this package's calls.

Shapes: the cache is a pool of pages, K and V [pages, rows, KV heads, D] (or
head-major [pages, KV heads, rows, D]) in bf16, or E4M3 codes with one fp32
scale per 64 elements, head-major in its page; block_table[b, j // rows] names
the page of key j of sequence b.  Accumulated weights and original positions
are [B, KV heads, capacity].
"""
import math
from types import SimpleNamespace

import numpy as np
import torch

own = False

TILE = 64          # elements of D that share one FP8 scale
FP8_MAX = 448.0    # largest E4M3 value
SPARE_PAGES = 8    # pages of the pool that no sequence owns


def _case(name, op, **kw):
    c = dict(name=name, op=op, B=1, QN=32, KVN=8, D=128, q_min=1, q_max=1, kv_min=1, kv_max=1,
             fresh=False, tnd=False, rows=128, fp8=False, head_major=False, window=0, first=0,
             sinks=False, budget=0, recent=0, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # one chat at its first tokens past the window: the latency of a single step
        _case("window_decode_one", "window", kv_min=1500, kv_max=1500, window=1024, first=4),
        # a full decode batch of long chats
        _case("window_decode_batch", "window", B=32, kv_min=8192, kv_max=32768, window=4096,
              first=4, lens=2),
        # multi-token decode (drafted tokens, ragged) over an FP8 cache, sinks in the softmax too
        _case("window_decode_rows_fp8", "window", B=16, QN=64, q_min=1, q_max=4, tnd=True,
              kv_min=2000, kv_max=16384, fp8=True, window=2048, first=64, sinks=True, lens=3),
        # prompts of mixed lengths in one call
        _case("window_prefill_varlen", "window", B=8, q_min=256, q_max=4096, tnd=True, fresh=True,
              window=1024, first=4, lens=4),
        # two short contexts: the latency of a step that also counts weights
        _case("weights_decode_small", "weights", B=2, kv_min=300, kv_max=777, lens=5),
        # the ordinary decode batch, counting weights
        _case("weights_decode_batch", "weights", B=32, kv_min=512, kv_max=4096, lens=6),
        # few long contexts in FP8, eight query heads per KV head
        _case("weights_decode_fp8_long", "weights", B=4, QN=64, kv_min=16384, kv_max=65536,
              fp8=True, lens=7),
        # prompts whose keys get their first weights
        _case("weights_prefill", "weights", B=4, q_min=256, q_max=2048, tnd=True, fresh=True,
              lens=8),
        # steady state: a page of new tokens past the budget, every sequence
        _case("evict_step", "evict", B=32, kv_min=2049, kv_max=2176, budget=2048, first=4,
              recent=256, lens=9),
        # long prompts cut down to the budget once
        _case("evict_prompt_fp8", "evict", B=4, kv_min=8192, kv_max=32768, fp8=True, budget=2048,
              first=4, recent=512, lens=10),
        # one new token for each sequence of a batch, quantised into the cache
        _case("append_token_fp8", "append", B=64, kv_min=17, kv_max=4096, fp8=True, lens=11),
        # prompts of mixed lengths written to their pages
        _case("append_prompt", "append", B=8, q_min=256, q_max=4096, tnd=True, fresh=True, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kvn = rng.choice([1, 2, 4, 8])
    fp8 = rng.random() < 0.4
    c = dict(KVN=kvn, QN=kvn * rng.choice([1, 2, 3, 4, 7, 8]), fp8=fp8,
             D=128 if fp8 else rng.choice([64, 128, 128]), rows=rng.choice([32, 64, 96, 128, 256]),
             head_major=rng.random() < 0.3, sinks=rng.random() < 0.3, tnd=rng.random() < 0.5,
             lens=rng.randrange(1 << 20))
    op = rng.choice(["window_decode", "window_prefill", "weights_decode", "weights_prefill",
                     "evict", "append"])
    if op.endswith("decode"):
        hi = _log(rng, 1, 24000)
        c.update(B=_log(rng, 1, 32), q_max=rng.choice([1, 1, 1, 2, 3, 4]),
                 kv_min=max(1, hi // rng.choice([1, 2, 9])), kv_max=hi)
        if op == "weights_decode":
            c.update(B=min(c["B"], max(1, 65536 // hi)))
    elif op.endswith("prefill"):
        hi = _log(rng, 17, 2000)
        c.update(B=_log(rng, 1, 8), q_min=max(1, hi // rng.choice([1, 3, 11])), q_max=hi,
                 tnd=True, fresh=rng.random() < 0.6, QN=min(c["QN"], 32),
                 # (prompts over an FP8 cache run on its values rounded to fp16, and
                 # their 32-bit outputs hold that format's bound, not fp32's)
                 fp8=False)
        if not c["fresh"]:
            c.update(kv_min=1, kv_max=_log(rng, 1, 2000))
    if op.startswith("window"):
        c.update(window=_log(rng, 1, 4096), first=rng.choice([0, 1, 4, 4, 64, 130, 300]))
    elif op == "evict":
        hi = _log(rng, 2, 32768)
        first, recent = rng.choice([0, 4, 32]), rng.choice([0, 1, 100, 500])
        c.update(B=_log(rng, 1, max(1, min(32, 131072 // hi))), kv_min=max(1, hi // 2), kv_max=hi,
                 first=first, recent=recent, budget=max(first + recent, _log(rng, 1, hi)))
    elif op == "append":
        hi = _log(rng, 1, 4000)
        c.update(B=_log(rng, 1, 16), q_min=max(1, hi // rng.choice([1, 2, 50])), q_max=hi,
                 tnd=True, fresh=rng.random() < 0.5, kv_min=0, kv_max=_log(rng, 1, 4000))
    if not c["tnd"] and "q_max" in c:
        c["q_min"] = c["q_max"]
    got = _case("", op.split("_")[0], **c)
    del got["name"]
    return got


# ----------------------------------------------------------------------------
# lengths, tables, inputs
# ----------------------------------------------------------------------------

def _lengths(c):
    """New rows and keys (the new ones among them) of each sequence."""
    r = np.random.RandomState(c["lens"])
    q = r.randint(c["q_min"], c["q_max"] + 1, c["B"])
    if not c["tnd"]:
        q[:] = c["q_max"]
    kv = q.copy() if c["fresh"] else r.randint(c["kv_min"], c["kv_max"] + 1, c["B"])
    if c["op"] == "append" and not c["fresh"]:
        kv = kv + q
    elif not c["fresh"] and c["q_max"] > 16:
        kv = kv + q  # a chunk of a prompt behind what the cache already holds
    else:
        kv = np.maximum(kv, 1)
    return q, kv


def _dev():
    return torch.device("cuda")


def _quantise(x):
    t = x.float().unflatten(-1, (-1, TILE))
    amax = t.abs().amax(-1)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    codes = (t / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return codes.flatten(-2).view(torch.uint8), scale


def prepare(case, seed):
    c, dev = case, _dev()
    g = torch.Generator(device=dev).manual_seed(seed)
    q_lens, kv_lens = _lengths(c)
    B, KVN, QN, D, rows = c["B"], c["KVN"], c["QN"], c["D"], c["rows"]
    pages = [-(-int(n) // rows) for n in kv_lens]
    width = max(max(pages), 1)
    if c["op"] == "evict":
        width = max(width, -(-c["budget"] // rows))
    nb = sum(pages) + SPARE_PAGES
    perm = np.random.RandomState(seed % (1 << 31)).permutation(nb)
    table = np.full((B, width), perm[-1], np.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    cap = width * rows

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)

    s = SimpleNamespace(op=c["op"], B=B, QN=QN, KVN=KVN, D=D, window=c["window"], first=c["first"],
                        budget=c["budget"], recent=c["recent"], cap=cap,
                        layout=1 if c["tnd"] else 0, S_q=int(q_lens.max()), T=int(q_lens.sum()),
                        kv_dtype=1 if c["fp8"] else 0, block_size=rows, num_blocks=nb, S_kv=cap,
                        kv_layout=1 if c["head_major"] else 0, scale=1.0 / math.sqrt(D),
                        kv_max=int(kv_lens.max()), atten_mask=None, next_tokens=0,
                        mask_mode=4 if c["op"] == "window" else 3,
                        pre_tokens=c["window"] - 1 if c["op"] == "window" else 0,
                        first_tokens=c["first"] if c["op"] == "window" else 0)
    s.block_table = torch.from_numpy(table).to(dev)
    s.seqused_kv = torch.from_numpy(kv_lens.astype(np.int32)).to(dev)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    s.cu = torch.from_numpy(cu).to(dev)
    s.cu_seqlens_q = s.cu if c["tnd"] else None
    s.k_scale = s.v_scale = s.sinks = None
    for name in "kv":
        x = normal(nb, rows, KVN, D)
        if c["op"] == "append":
            x.zero_()
        if c["fp8"]:
            x, sc = _quantise(x)
            setattr(s, name + "_scale", sc.permute(0, 2, 1, 3).contiguous())
        setattr(s, name + "_cache", x.permute(0, 2, 1, 3).contiguous() if c["head_major"] else x)
    if c["op"] in ("window", "weights"):
        s.q = normal(s.T, QN, D) if c["tnd"] else normal(B, s.S_q, QN, D)
        if c["sinks"]:
            s.sinks = torch.randn(QN, generator=g, device=dev)
    if c["op"] == "weights":
        # what a key got so far is of the size of what this call adds
        s.weights = torch.rand(B, KVN, cap, generator=g, device=dev)
        s.weights *= 2 * QN // KVN * s.S_q / s.seqused_kv.float()[:, None, None]
        s.weights_out = torch.zeros_like(s.weights)
    if c["op"] == "evict":
        # weights fall off steeply; the newest keys have had no query yet
        s.weights = torch.randn(B, KVN, cap, generator=g, device=dev).mul_(2).exp_()
        s.weights[torch.rand(B, KVN, cap, generator=g, device=dev) < 0.05] = 0.0
        # slots after earlier evictions: the first `budget` hold older tokens in
        # any order, each KV head its own, the rest the newest ones in theirs
        s.tokens_seen = s.seqused_kv + torch.randint(0, 5000, (B,), generator=g, device=dev,
                                                     dtype=torch.int32)
        old = torch.rand(B, KVN, cap, generator=g, device=dev).argsort(-1).argsort(-1)
        slot = torch.arange(cap, device=dev)
        old_n = torch.minimum(s.seqused_kv, torch.full_like(s.seqused_kv, c["budget"]))[:, None, None]
        inside = torch.where(slot < old_n, torch.where(slot < old_n, old, cap).argsort(-1).argsort(-1),
                             slot)
        shift = (s.tokens_seen - s.seqused_kv)[:, None, None]
        s.positions = torch.where(inside < c["first"], inside, inside + shift).to(torch.int32)
        s.weights_out, s.positions_out = torch.zeros_like(s.weights), torch.zeros_like(s.positions)
        s.seqused_out = torch.zeros_like(s.seqused_kv)
    if c["op"] == "append":
        shape = (s.T, KVN, D) if c["tnd"] else (B, s.S_q, KVN, D)
        s.k_new, s.v_new = normal(*shape), normal(*shape)
        s.tokens_seen = s.seqused_kv + 100
        s.weights = torch.rand(B, KVN, cap, generator=g, device=dev)
        s.positions = torch.zeros(B, KVN, cap, dtype=torch.int32, device=dev)
    if own:  # the call object that a program keeps for its buffers
        s.call = _make_call(s)
    return s


# ----------------------------------------------------------------------------
# the package's calls
# ----------------------------------------------------------------------------

def _make_call(s):
    import decode_tile_scheduler_gb300 as fia
    if s.op == "window":
        return fia.FiaCall(s)
    if s.op == "weights":
        return fia.KeyWeightsCall(s, weights=s.weights, weights_out=s.weights_out)
    cache = fia.KvCache(s.k_cache, s.v_cache, s.block_table, k_scale=s.k_scale, v_scale=s.v_scale,
                        kv_layout=s.kv_layout)
    if s.op == "append":
        return fia.KvAppendCall(cache, s.k_new, s.v_new, s.seqused_kv, cu_seqlens_q=s.cu_seqlens_q,
                                weights=s.weights, positions=s.positions,
                                tokens_seen=s.tokens_seen)
    return fia.KvEvictCall(cache, s.seqused_kv, s.weights, budget=s.budget, first_tokens=s.first,
                           recent_tokens=s.recent, positions=s.positions,
                           tokens_seen=s.tokens_seen, weights_out=s.weights_out,
                           positions_out=s.positions_out, seqused_out=s.seqused_out)


def _cache_values(s):
    """K and V of the cache as they stand (E4M3 codes as the values they are)."""
    if s.kv_dtype == 0:
        return {"k": s.k_cache, "v": s.v_cache}
    e4m3 = torch.float8_e4m3fn
    return {"k": s.k_cache.view(e4m3), "v": s.v_cache.view(e4m3), "k_scale": s.k_scale,
            "v_scale": s.v_scale}


def run(s):
    if own:
        r = s.call.run()
        if s.op == "window":
            return {"out": r[0], "lse": r[1]}
        if s.op == "weights":
            return {"out": r[0], "lse": r[1], "weights": r[2]}
    elif s.op in ("window", "weights"):
        return _plain_attention(s)
    elif s.op == "append":
        _plain_append(s)
    else:
        _plain_evict(s)
    if s.op == "append":
        return {**_cache_values(s), "weights": s.weights, "positions": s.positions}
    return {**_cache_values(s), "weights": s.weights_out, "positions": s.positions_out,
            "lens": s.seqused_out}


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _by_token(pool, s):
    """The pool with (page, row) first, whichever its layout."""
    return pool.permute(0, 2, 1, 3) if s.kv_layout else pool


def _gathered(s, j):
    """K and V of the keys j [B, N] of each sequence, in 32 bits, [B, KVN, N, D]."""
    page = s.block_table.gather(1, j // s.block_size).long()
    row = j % s.block_size
    got = []
    for pool, scale in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)):
        x = _by_token(pool, s)[page, row]
        if scale is None:
            x = x.float()
        else:
            sc = scale.permute(0, 2, 1, 3)[page, row]
            x = x.view(torch.float8_e4m3fn).float() * sc.repeat_interleave(TILE, -1)
        got.append(x.permute(0, 2, 1, 3))
    return got


def _plain_attention(s):
    dev = s.q.device
    kv = s.seqused_kv.long()[:, None]
    if s.layout:
        q_len = (s.cu[1:] - s.cu[:-1]).long()[:, None]
        i = torch.arange(s.S_q, device=dev)[None]
        token = torch.where(i < q_len, s.cu[:-1].long()[:, None] + i, 0)
        q = s.q[token]                                    # [B, S, QN, D]
    else:
        q_len = torch.full((s.B, 1), s.S_q, device=dev)
        i = torch.arange(s.S_q, device=dev)[None]
        q = s.q
    p = kv - q_len + i                                    # [B, S] positions of the rows
    n = torch.arange(s.kv_max, device=dev)[None]
    ok = n < kv
    j = torch.where(ok, n, 0)
    if s.op == "window" and s.S_q <= 16 and s.first + s.window + s.S_q < s.kv_max:
        # only the keys that some row of the sequence may see
        n = torch.arange(s.first + s.window + s.S_q, device=dev)[None]
        late = kv - q_len - s.pre_tokens + n - s.first
        j = torch.where(n < s.first, n, late)
        ok = (j < kv) & ((n < s.first) | (j >= s.first))
        j = torch.where(ok, j, 0)
    k, v = _gathered(s, j)
    G = s.QN // s.KVN
    qg = q.float().reshape(s.B, s.S_q, s.KVN, G, s.D).permute(0, 2, 1, 3, 4)
    x = qg.reshape(s.B, s.KVN, s.S_q * G, s.D) @ k.transpose(2, 3) * s.scale
    see = ok[:, None, :] & (j[:, None, :] <= p[:, :, None]) & (i < q_len)[:, :, None]
    if s.op == "window":
        see = see & ((j[:, None, :] >= p[:, :, None] - s.pre_tokens) | (j[:, None, :] < s.first))
    x = x.reshape(s.B, s.KVN, s.S_q, G, -1).masked_fill_(~see[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    if s.sinks is not None:
        sink = s.sinks.reshape(1, s.KVN, 1, G, 1)
        m = torch.maximum(m, sink)
    seen = see.any(-1)[:, None, :, None, None]
    m = torch.where(seen, m, 0.0)
    e = (x - m).exp_()
    z = e.sum(-1, keepdim=True)
    if s.sinks is not None:
        z = z + (sink - m).exp()
    w = e.div_(torch.where(seen, z, 1.0))
    o = (w.flatten(2, 3) @ v).unflatten(2, (s.S_q, G))
    lse = torch.where(seen, m + z.log(), math.inf)[..., 0]    # [B, KVN, S, G]
    o = o.permute(0, 2, 1, 3, 4).reshape(s.B, s.S_q, s.QN, s.D).to(torch.bfloat16)
    if s.layout:
        keep = i < q_len
        got = {"out": o[keep], "lse": lse.permute(0, 2, 1, 3).reshape(s.B, s.S_q, s.QN)[keep][..., None]}
    else:
        got = {"out": o, "lse": lse.permute(0, 1, 3, 2).reshape(s.B, s.QN, s.S_q)[..., None]}
    if s.op == "weights":
        total = w.sum((2, 3))
        s.weights_out[:, :, :s.kv_max] = torch.where(
            ok[:, None, :], s.weights[:, :, :s.kv_max] + total, s.weights_out[:, :, :s.kv_max])
        got["weights"] = s.weights_out
    return got


def _plain_append(s):
    dev = s.k_new.device
    t = torch.arange(s.T if s.layout else s.B * s.S_q, device=dev)
    if s.layout:
        b = torch.searchsorted(s.cu[1:].long(), t, right=True)
        q_len = (s.cu[1:] - s.cu[:-1]).long()[b]
        i = t - s.cu.long()[b]
    else:
        b, i, q_len = t // s.S_q, t % s.S_q, s.S_q
    back = i - q_len
    slot = s.seqused_kv.long()[b] + back
    page, row = s.block_table[b, slot // s.block_size].long(), slot % s.block_size
    for new, pool, scale in ((s.k_new, s.k_cache, s.k_scale), (s.v_new, s.v_cache, s.v_scale)):
        x = new.reshape(-1, s.KVN, s.D)
        if scale is not None:
            x, sc = _quantise(x)
            scale.permute(0, 2, 1, 3)[page, row] = sc
        _by_token(pool, s)[page, row] = x
    s.weights[b, :, slot] = 0.0
    s.positions[b, :, slot] = (s.tokens_seen.long()[b] + back).to(torch.int32)[:, None]


def _plain_evict(s):
    slot = torch.arange(s.cap, device=s.weights.device)
    n = s.seqused_kv[:, None, None]
    inside = slot < n
    safe = (s.positions < s.first) | (s.positions >= s.tokens_seen[:, None, None] - s.recent)
    score = torch.where(inside, torch.where(safe, math.inf, s.weights.double()), -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    keep = inside & (rank < s.budget)
    new_n = s.seqused_kv.clamp(max=s.budget)
    hole = ((slot < new_n[:, None, None]) & ~keep).nonzero(as_tuple=True)
    tail = (keep & (slot >= s.budget)).nonzero(as_tuple=True)
    stays = slot < new_n[:, None, None]
    for a, out in ((s.weights, s.weights_out), (s.positions, s.positions_out)):
        out.copy_(torch.where(stays, a, out))
        out[hole] = a[tail]
    b, h = hole[0], hole[1]
    to = s.block_table[b, hole[2] // s.block_size].long(), hole[2] % s.block_size
    of = s.block_table[b, tail[2] // s.block_size].long(), tail[2] % s.block_size
    for pool, scale in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)):
        x = _by_token(pool, s)
        x[to[0], to[1], h] = x[of[0], of[1], h]
        if scale is not None:
            scale[to[0], h, to[1]] = scale[of[0], h, of[1]]
    s.seqused_out.copy_(new_n)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def _seen(c, ql, kl):
    """(row, key) pairs that the mask leaves, and keys that some row sees."""
    p = kl - ql + np.arange(ql, dtype=np.int64)
    p = p[p >= 0]
    if not len(p):
        return 0, 0
    if c["op"] == "weights":
        return int((p + 1).sum()), int(p[-1] + 1)
    lo = np.maximum(p - c["window"] + 1, 0)
    pairs = int((p + 1 - lo + np.minimum(lo, c["first"])).sum())
    return pairs, int(p[-1] + 1 - lo[0] + min(lo[0], c["first"]))


def work(case):
    c = case
    q_lens, kv_lens = _lengths(c)
    KVN, QN, D = c["KVN"], c["QN"], c["D"]
    row = 2 * (D + 4 * D // TILE if c["fp8"] else 2 * D)  # K and V of one key, one head
    T = int(q_lens.sum())
    if c["op"] in ("window", "weights"):
        pairs, keys = (sum(x) for x in zip(*(_seen(c, int(a), int(b)) for a, b in zip(q_lens, kv_lens))))
        nbytes = T * QN * (4 * D + 4) + keys * KVN * row
        if c["op"] == "weights":
            nbytes += 8 * KVN * int(kv_lens.sum())
        return {"bytes": nbytes, "flops": 4 * D * QN * pairs}
    if c["op"] == "append":
        return {"bytes": T * KVN * (4 * D + row + 8), "flops": 0}
    over = kv_lens[kv_lens > c["budget"]]
    new = np.minimum(kv_lens, c["budget"])
    # at least the protected newest keys move, where they stand past the budget
    moved = int(np.minimum(over - c["budget"], max(c["recent"], 1)).sum()) if len(over) else 0
    return {"bytes": KVN * (8 * int(kv_lens.sum()) + 8 * int(new.sum()) + 2 * row * moved), "flops": 0}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _exact_cache(s, pool, scale, b, n):
    """Keys 0..n-1 of sequence b in 64 bits, [n, KVN, D]."""
    j = np.arange(n)
    table = s.block_table[b].cpu().numpy()
    page = torch.from_numpy(table[j // s.block_size].astype(np.int64)).to(pool.device)
    row = torch.from_numpy(j % s.block_size).to(pool.device)
    x = pool[page, :, row] if s.kv_layout else pool[page, row]
    if scale is None:
        return x.double()
    v = x.view(torch.float8_e4m3fn).float().double()
    sc = scale[page, :, row].double()
    return (v.reshape(n, s.KVN, -1, TILE) * sc[..., None]).reshape(n, s.KVN, s.D)


def _exact_attention(c, s):
    q_lens, kv_lens = _lengths(c)
    outs, lses, G = [], [], s.QN // s.KVN
    weights = torch.zeros(s.weights_out.shape, dtype=torch.float64, device=s.q.device) \
        if c["op"] == "weights" else None
    t0 = 0
    for b in range(s.B):
        ql, kl = int(q_lens[b]), int(kv_lens[b])
        q = (s.q[t0:t0 + ql] if s.layout else s.q[b]).double()
        t0 += ql
        j = torch.arange(kl, device=s.q.device)
        p = kl - ql + torch.arange(ql, device=s.q.device)[:, None]
        see = j <= p
        cols = j
        if c["op"] == "window":
            see = see & ((j > p - c["window"]) | (j < c["first"]))
            cols = see.any(0).nonzero()[:, 0]
            see = see[:, cols]
        k = _exact_cache(s, s.k_cache, s.k_scale, b, kl)[cols]
        v = _exact_cache(s, s.v_cache, s.v_scale, b, kl)[cols]
        o = torch.zeros(ql, s.QN, s.D, dtype=torch.float64, device=s.q.device)
        z = torch.full((ql, s.QN), math.inf, dtype=torch.float64, device=s.q.device)
        some = see.any(1)
        for h in range(s.QN):
            x = (q[:, h] @ k[:, h // G].T * s.scale).masked_fill(~see, -math.inf)
            if s.sinks is not None:
                x = torch.cat([x, s.sinks[h].double().expand(ql, 1)], 1)
            l = torch.logsumexp(x, 1)
            w = torch.exp(x - torch.where(some, l, 0)[:, None])[:, :len(cols)]
            w[~some] = 0
            o[:, h] = w @ v[:, h // G]
            z[:, h] = torch.where(some, l, math.inf)
            if weights is not None:
                weights[b, h // G, :kl] += w.sum(0)
        if weights is not None:
            weights[b, :, :kl] += s.weights[b, :, :kl].double()
        outs.append(o)
        lses.append(z if s.layout else z.T)
    got = {"out": torch.cat(outs) if s.layout else torch.stack(outs),
           "lse": (torch.cat(lses) if s.layout else torch.stack(lses))[..., None]}
    if weights is not None:
        got["weights"] = weights
    return got


def _exact_e4m3(x):
    """x rounded to E4M3 in 64 bits: 4 significant bits, steps of 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20)))
    e = torch.where(2.0 ** e > x.abs(), e - 1, torch.where(2.0 ** (e + 1) <= x.abs(), e + 1, e))
    step = 2.0 ** (e.clamp_min(-6) - 3)
    return (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_append(c, s):
    q_lens, kv_lens = _lengths(c)
    got = {}
    new = {}
    for name in "kv":
        x = getattr(s, name + "_new").double().reshape(-1, s.KVN, s.D)
        if s.kv_dtype:
            t = x.reshape(-1, s.KVN, s.D // TILE, TILE)
            amax = t.abs().amax(-1)
            scale = torch.where(amax > 0, amax / 448, 1.0)
            new[name + "_scale"] = scale
            x = _exact_e4m3(t / scale[..., None]).reshape(x.shape)
        new[name] = x
        pool = getattr(s, name + "_cache")
        got[name] = (pool.view(torch.float8_e4m3fn).float() if s.kv_dtype else pool).double()
        if s.kv_dtype:
            got[name + "_scale"] = getattr(s, name + "_scale").double()
    got["weights"] = s.weights.double()
    positions = s.positions.clone()
    table = s.block_table.cpu().numpy()
    seen = s.tokens_seen.cpu().numpy()
    t0 = 0
    for b in range(s.B):
        ql, kl = int(q_lens[b]), int(kv_lens[b])
        j = np.arange(kl - ql, kl)
        page = torch.from_numpy(table[b, j // s.block_size].astype(np.int64)).to(s.weights.device)
        row = torch.from_numpy(j % s.block_size).to(page.device)
        for name in new:
            x = new[name][t0:t0 + ql]
            if s.kv_layout or name.endswith("scale"):
                got[name][page, :, row] = x
            else:
                got[name][page, row] = x
        got["weights"][b, :, kl - ql:kl] = 0
        positions[b, :, kl - ql:kl] = torch.arange(int(seen[b]) - ql, int(seen[b]),
                                                   device=page.device, dtype=torch.int32)
        t0 += ql
    got["positions"] = positions
    return got


def _exact_evict(c, s):
    _, kv_lens = _lengths(c)
    dev = s.weights.device
    w, pos = s.weights.double().cpu().numpy(), s.positions.cpu().numpy()
    wo, po = np.zeros_like(w), np.zeros_like(pos)
    seen, table = s.tokens_seen.cpu().numpy(), s.block_table.cpu().numpy()
    moves = []
    for b in range(s.B):
        n, m = int(kv_lens[b]), min(int(kv_lens[b]), c["budget"])
        for h in range(s.KVN):
            safe = (pos[b, h, :n] < c["first"]) | (pos[b, h, :n] >= seen[b] - c["recent"])
            # best first: protected keys, then larger weights, then lower slots
            best = np.lexsort((np.arange(n), np.where(safe, 0.0, -w[b, h, :n]), ~safe))[:m]
            kept = np.zeros(n, bool)
            kept[best] = True
            hole, tail = np.nonzero(~kept[:m])[0], m + np.nonzero(kept[m:])[0]
            for a, o in ((w, wo), (pos, po)):
                o[b, h, :m] = a[b, h, :m]
                o[b, h, hole] = a[b, h, tail]
            rows = s.block_size
            moves.append(np.stack([table[b, hole // rows], hole % rows, table[b, tail // rows],
                                   tail % rows, np.full(len(hole), h)]))
    tp, tr, fp, fr, h = torch.from_numpy(np.concatenate(moves, 1).astype(np.int64)).to(dev)
    got = {}
    for name, x in _cache_values(s).items():
        x = (x.float() if x.element_size() == 1 else x).double()
        if s.kv_layout or name.endswith("scale"):
            x[tp, h, tr] = x[fp, h, fr]
        else:
            x[tp, tr, h] = x[fp, fr, h]
        got[name] = x
    return {**got, "weights": torch.from_numpy(wo).to(dev), "positions": torch.from_numpy(po).to(dev),
            "lens": s.seqused_kv.clamp(max=c["budget"])}


def exact(case, seed):
    if case["op"] in ("window", "weights"):
        if work(case)["flops"] > 6e12:
            return None
        return _exact_attention(case, prepare(case, seed))
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_evict(case, s)
