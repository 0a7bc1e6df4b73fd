"""The operators around a KV cache held in 4 bits, as cases to measure and to check.

A serving step over a paged cache makes four calls: it assigns pages to the
sequences that grew (block table, free list, and the slot and position of every
new token), it norms the heads of the new queries and keys, rotates them to
their positions and writes K and V to their slots, or it appends K and V that
are ready, quantised to 4 bits, and it attends over the cache.  Each case is one
such call.  With `own` false, run() computes it in elementary torch operations
in 32 bits; with `own` true, through this package's calls.

Shapes: the cache is a pool of pages, K and V [pages, rows, KV heads, D] (or
head-major [pages, KV heads, rows, D]).  In 4 bits a byte holds two E2M1 codes
(the element of the lower index in its lower half), [..., D/2], with one E8M0
scale byte per 32 elements, head-major in its page, [pages, KV heads, rows,
D/32].  block_table[b, j // rows] names the page of key j of sequence b; the
slot of a key is page * rows + j % rows.
"""
import math
from types import SimpleNamespace

import numpy as np
import torch

own = False

MX_TILE = 32       # elements of D that share one E8M0 scale
FP8_TILE = 64      # elements of D that share one fp32 scale
FP8_MAX = 448.0
SPARE_PAGES = 8    # pages of the pool that no sequence owns
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _case(name, op, **kw):
    c = dict(name=name, op=op, B=1, QN=32, KVN=8, D=128, q_min=1, q_max=1, kv_min=1, kv_max=1,
             fresh=False, tnd=False, rows=128, kv="mx", head_major=False, mask=3, window=0, first=0,
             sinks=False, rot=128, pairs=False, norm=True, ended=0.0, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # a decode step of a batch: one new token each, now and then a new page
        _case("pages_step", "pages", B=64, kv_min=17, kv_max=4096, ended=0.05, lens=21),
        # a large mixed batch: chunks of prompts and single tokens, many requests ending
        _case("pages_mixed", "pages", B=1024, q_min=1, q_max=256, tnd=True, kv_min=0, kv_max=4096,
              rows=64, ended=0.2, lens=22),
        # the new tokens of a decode batch: latency
        _case("rope_token", "rope", B=32, kv_min=512, kv_max=4096, kv="bf16", lens=23),
        # prompts of mixed lengths
        _case("rope_prompt", "rope", B=8, q_min=256, q_max=4096, tnd=True, fresh=True, kv="bf16",
              lens=24),
        # prompts into an FP8 cache, a part of D rotated in neighbouring pairs
        _case("rope_prompt_fp8", "rope", B=4, QN=64, q_min=256, q_max=2048, tnd=True, fresh=True,
              kv="fp8", rot=64, pairs=True, lens=25),
        # one new token for each sequence of a batch, quantised into the cache
        _case("append_token", "append", B=64, kv_min=17, kv_max=4096, lens=26),
        # prompts of mixed lengths written to their pages
        _case("append_prompt", "append", B=8, q_min=256, q_max=4096, tnd=True, fresh=True, lens=27),
        # two short contexts: the latency of a step
        _case("attend_small", "attend", B=2, kv_min=300, kv_max=777, lens=28),
        # the ordinary decode batch
        _case("attend_batch", "attend", B=32, kv_min=512, kv_max=4096, lens=29),
        # few long contexts, eight query heads per KV head
        _case("attend_long", "attend", B=4, QN=64, kv_min=32768, kv_max=131072, lens=30),
        # drafted tokens, ragged, with sinks, through a window whose first tokens stay visible
        _case("attend_rows", "attend", B=16, q_min=1, q_max=4, tnd=True, kv_min=2000, kv_max=16384,
              mask=4, window=4096, first=4, sinks=True, lens=31),
        # prompts of mixed lengths in one call
        _case("attend_prompt", "attend", B=8, q_min=256, q_max=4096, tnd=True, fresh=True, lens=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kvn = rng.choice([1, 2, 4, 8])
    c = dict(KVN=kvn, QN=kvn * rng.choice([1, 2, 3, 4, 7, 8]), rows=rng.choice([32, 64, 96, 128, 256]),
             head_major=rng.random() < 0.3, sinks=rng.random() < 0.3, tnd=rng.random() < 0.5,
             lens=rng.randrange(1 << 20))
    op = rng.choice(["pages", "rope", "append", "decode", "prefill"])
    if op == "pages":
        c.update(B=_log(rng, 1, 2048), q_max=_log(rng, 1, 64), kv_min=0, kv_max=_log(rng, 1, 4096),
                 ended=rng.choice([0.0, 0.1, 0.5]))
        c.update(q_min=rng.choice([0, 1]) if c["tnd"] else c["q_max"])
    elif op in ("rope", "append"):
        hi = _log(rng, 1, 4000)
        c.update(B=_log(rng, 1, 16), q_min=max(1, hi // rng.choice([1, 2, 50])), q_max=hi,
                 tnd=True, fresh=rng.random() < 0.5, kv_min=0, kv_max=_log(rng, 1, 4000))
        if op == "rope":
            c.update(QN=min(c["QN"], 32), kv=rng.choice(["bf16", "bf16", "fp8"]),
                     pairs=rng.random() < 0.4, norm=rng.random() < 0.8)
            c.update(D=128 if c["kv"] == "fp8" else rng.choice([64, 128, 128]))
            c.update(rot=c["D"] * rng.choice([2, 4, 4, 4]) // 4)
    elif op == "decode":
        hi = _log(rng, 1, 60000)
        c.update(B=min(_log(rng, 1, 32), max(1, 200000 // hi)), q_max=rng.choice([1, 1, 1, 2, 4, 8]),
                 kv_min=max(1, hi // rng.choice([1, 2, 9])), kv_max=hi)
        c.update(q_min=1 if c["tnd"] else c["q_max"], mask=rng.choice([0, 3, 3, 4]))
    else:
        hi = _log(rng, 17, 2000)
        c.update(B=_log(rng, 1, 8), q_min=max(1, hi // rng.choice([1, 3, 11])), q_max=hi,
                 tnd=True, fresh=rng.random() < 0.6, QN=min(c["QN"], 32), mask=rng.choice([3, 3, 4]))
        if not c["fresh"]:
            c.update(kv_min=1, kv_max=_log(rng, 1, 2000))
    if c.get("mask") == 4:
        c.update(window=_log(rng, 1, 4096), first=rng.choice([0, 1, 4, 64, 300]))
    got = _case("", {"decode": "attend", "prefill": "attend"}.get(op, op), **c)
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
    if c["op"] == "pages" and c["tnd"]:
        q[r.rand(c["B"]) < 0.5] = min(1, c["q_max"])  # (half of a mixed batch decodes)
        q[_ended(c)] = 0
    if c["op"] == "attend" and (c["fresh"] or c["q_max"] <= 16):
        kv = np.maximum(kv, 1)
    elif not c["fresh"]:
        kv = kv + q
    return q, kv


def _ended(c):
    """Sequences whose request has ended: they hold pages and need none."""
    return np.random.RandomState(c["lens"] + 1).rand(c["B"]) < c["ended"]


def _dev():
    return torch.device("cuda")


def _e4m3(x):
    t = x.float().unflatten(-1, (-1, FP8_TILE))
    amax = t.abs().amax(-1)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    codes = (t / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return codes.flatten(-2).view(torch.uint8), scale


def _pow2(e):
    """2^e as a 32-bit value, -127 <= e <= 127."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _mx(x):
    """Two E2M1 codes to a byte, and E8M0 scales: the smallest power of two that
    leaves no magnitude over 6 (1 where all are 0), codes to nearest, ties to even."""
    t = x.float().unflatten(-1, (-1, MX_TILE))
    amax = t.abs().amax(-1)
    m, e = torch.frexp(amax)                      # amax = m 2^e, 0.5 <= m < 1
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(-127, 127)
    e = torch.where(amax > 0, e, 0)
    y = t / _pow2(e)[..., None]
    a = y.abs()
    code = sum((a > b) if k % 2 == 0 else (a >= b)
               for k, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    c, dev = case, _dev()
    g = torch.Generator(device=dev).manual_seed(seed)
    q_lens, kv_lens = _lengths(c)
    B, KVN, QN, D, rows = c["B"], c["KVN"], c["QN"], c["D"], c["rows"]
    S_q, T = int(q_lens.max()), int(q_lens.sum())
    pages = [-(-int(n) // rows) for n in kv_lens]
    width, nb = max(max(pages), 1), sum(pages) + SPARE_PAGES
    perm = np.random.RandomState(seed % (1 << 31)).permutation(nb)
    table = np.full((B, width), perm[-1], np.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    s = SimpleNamespace(op=c["op"], B=B, QN=QN, KVN=KVN, D=D, layout=1 if c["tnd"] else 0, S_q=S_q,
                        T=T, kv=c["kv"], block_size=rows, num_blocks=nb, S_kv=width * rows,
                        kv_layout=1 if c["head_major"] else 0, kv_max=int(kv_lens.max()))
    s.block_table = torch.from_numpy(table).to(dev)
    s.seqused_kv = torch.from_numpy(kv_lens.astype(np.int32)).to(dev)
    s.cu = torch.from_numpy(cu).to(dev)
    s.cu_seqlens_q = s.cu if c["tnd"] else None
    if c["op"] == "pages":
        return _prepare_pages(c, s, q_lens, kv_lens, pages, perm, at, dev)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)

    s.k_scale = s.v_scale = None
    for name in "kv":
        x = normal(nb, rows, KVN, D)
        if c["op"] != "attend":
            x.zero_()
        if c["kv"] != "bf16":
            x, sc = (_mx if c["kv"] == "mx" else _e4m3)(x)
            setattr(s, name + "_scale", sc.permute(0, 2, 1, 3).contiguous())
        setattr(s, name + "_cache", x.permute(0, 2, 1, 3).contiguous() if c["head_major"] else x)
    if c["op"] == "attend":
        s.q = normal(T, QN, D) if c["tnd"] else normal(B, S_q, QN, D)
        s.sinks = torch.randn(QN, generator=g, device=dev) if c["sinks"] else None
        s.kv_dtype, s.scale, s.atten_mask, s.next_tokens = 4, 1.0 / math.sqrt(D), None, 0
        s.mask_mode = c["mask"]
        s.pre_tokens, s.first_tokens = (c["window"] - 1, c["first"]) if c["mask"] == 4 else (0, 0)
    elif c["op"] == "append":
        shape = (T, KVN, D) if c["tnd"] else (B, S_q, KVN, D)
        s.k_new, s.v_new = normal(*shape), normal(*shape)
    else:  # one projection's output: the heads of q, then of k, then of v
        s.qkv = normal(T, QN + 2 * KVN, D)
        s.q, s.k_new, s.v_new = s.qkv.split((QN, KVN, KVN), 1)
        s.q_out = torch.zeros(T, QN, D, dtype=torch.bfloat16, device=dev)
        w = [(1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) for _ in "qk"]
        s.q_weight, s.k_weight = w if c["norm"] else (None, None)
        s.eps, s.rot, s.pairs = 1e-6, c["rot"], c["pairs"]
        b = np.repeat(np.arange(B), q_lens)
        j = kv_lens[b] - q_lens[b] + np.arange(T) - cu[b]
        s.positions = torch.from_numpy(j.astype(np.int32)).to(dev)
        s.slots = torch.from_numpy((table[b, j // rows].astype(np.int64) * rows + j % rows)
                                   .astype(np.int32)).to(dev)
        angle = torch.arange(s.kv_max, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (
            -torch.arange(0, s.rot, 2, dtype=torch.float64, device=dev) / s.rot)
        s.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    if own:  # the call object that a program keeps for its buffers
        s.call = _make_call(s)
    return s


def _prepare_pages(c, s, q_lens, kv_lens, pages, perm, at, dev):
    """The state before the step: the pages that the lengths without the new rows
    take are held (an ended request's all), the others are free."""
    old = np.maximum(kv_lens - q_lens, 0)
    ended = _ended(c)
    held = np.where(ended, pages, -(-old // c["rows"]))
    s.seqused_kv = torch.from_numpy(np.where(ended, 0, kv_lens).astype(np.int32)).to(dev)
    table = s.block_table.cpu().numpy()
    slot = np.arange(table.shape[1])[None]
    mine = slot < np.asarray(pages)[:, None]
    free = np.concatenate([perm[at:], table[mine & (slot >= held[:, None])]]).astype(np.int32)
    table = np.where(mine & (slot < held[:, None]), table, -1).astype(np.int32)
    stack = np.full(s.num_blocks, -1, np.int32)
    stack[:len(free)] = free[np.random.RandomState(s.T).permutation(len(free))]
    s.block_table, s.pages_held = torch.from_numpy(table).to(dev), torch.from_numpy(held.astype(np.int32)).to(dev)
    s.free_pages = torch.from_numpy(stack).to(dev)
    s.free_count = torch.tensor([len(free)], dtype=torch.int32, device=dev)
    s.held_out, s.count_out = torch.zeros_like(s.pages_held), torch.zeros_like(s.free_count)
    s.slots = torch.zeros(s.T, dtype=torch.int32, device=dev)
    s.positions = torch.zeros(s.T, dtype=torch.int32, device=dev)
    s.status = torch.zeros(1, dtype=torch.int32, device=dev)
    if own:
        s.call = _make_call(s)
    return s


# ----------------------------------------------------------------------------
# the package's calls
# ----------------------------------------------------------------------------

def _make_call(s):
    import decode_tile_scheduler_gb300 as fia
    if s.op == "pages":
        # (the counts after the call go to tensors of their own, so that a pass
        # finds what the one before it found)
        return fia.AssignPagesCall(s.block_table, s.pages_held, s.free_pages, s.free_count,
                                   s.seqused_kv, block_size=s.block_size,
                                   cu_seqlens_q=s.cu_seqlens_q, seqlen_q=s.S_q, slots=s.slots,
                                   positions=s.positions, pages_held_out=s.held_out,
                                   free_count_out=s.count_out, status=s.status)
    if s.op == "attend":
        return fia.FiaCall(s)
    cache = fia.KvCache(s.k_cache, s.v_cache, s.block_table, k_scale=s.k_scale, v_scale=s.v_scale,
                        kv_layout=s.kv_layout)
    if s.op == "append":
        return fia.KvAppendCall(cache, s.k_new, s.v_new, s.seqused_kv, cu_seqlens_q=s.cu_seqlens_q)
    return fia.NormRopeAppendCall(cache, s.q, s.k_new, s.v_new, s.slots, s.positions, s.cos_sin,
                                  q_weight=s.q_weight, k_weight=s.k_weight, eps=s.eps,
                                  interleaved=s.pairs, q_out=s.q_out)


def _cache_values(s):
    """K and V of the cache as they stand (E4M3 codes as the values they are; 4-bit
    codes and their scales as the whole numbers that the format defines exactly)."""
    if s.kv == "bf16":
        return {"k": s.k_cache, "v": s.v_cache}
    k, v = s.k_cache, s.v_cache
    if s.kv == "fp8":
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return {"k": k, "v": v, "k_scale": s.k_scale, "v_scale": s.v_scale}


def run(s):
    if own:
        r = s.call.run()
        if s.op == "attend":
            return {"out": r[0], "lse": r[1]}
    elif s.op == "attend":
        return _plain_attention(s)
    elif s.op == "pages":
        _plain_pages(s)
    elif s.op == "append":
        _plain_append(s)
    else:
        _plain_rope(s)
    if s.op == "pages":
        return {"table": s.block_table, "free": s.free_pages, "held": s.held_out,
                "count": s.count_out, "slots": s.slots, "positions": s.positions,
                "status": s.status}
    if s.op == "append":
        return _cache_values(s)
    return {"q": s.q_out, **_cache_values(s)}


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _rows_of(s, dev):
    """Sequence, row in it, and row count of every new token."""
    t = torch.arange(s.T, device=dev)
    if s.layout:
        b = torch.searchsorted(s.cu[1:].long(), t, right=True)
        return b, t - s.cu.long()[b], (s.cu[1:] - s.cu[:-1]).long()[b]
    return t // s.S_q, t % s.S_q, torch.full_like(t, s.S_q)


def _plain_pages(s):
    dev, rows = s.block_table.device, s.block_size
    width, nb = s.block_table.shape[1], s.num_blocks
    lens = s.seqused_kv.long()
    need = ((lens.clamp(min=0) + rows - 1) // rows).clamp(max=width)
    held = s.pages_held.long().clamp(0, width)
    count = s.free_count.long().clamp(0, nb)
    give, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    given, taken = give.cumsum(0), take.cumsum(0)
    k = torch.arange(width, device=dev)[None]
    # pages given back lie on the free list in the order of their sequences
    stack = torch.full((2 * nb + 1,), -1, dtype=torch.int32, device=dev)
    stack[:nb] = s.free_pages
    back = (k >= need[:, None]) & (k < held[:, None])
    at = count + (given - give)[:, None] + k - need[:, None]
    stack[torch.where(back, at, 2 * nb)] = torch.where(back, s.block_table, -1)
    # and the takers take from its end
    top = count + given[-1]
    at = top - 1 - ((taken - take)[:, None] + k - held[:, None])
    new = (k >= held[:, None]) & (k < need[:, None])
    s.block_table.copy_(torch.where(new, torch.where(at >= 0, stack[at.clamp(min=0)], -1), s.block_table))
    got = torch.minimum(take, (top - (taken - take)).clamp(min=0))
    left = (top - taken[-1]).clamp(min=0)
    s.free_pages.copy_(stack[:nb])
    s.held_out.copy_(torch.minimum(held, need) + got)
    s.count_out.copy_(left)
    b, i, q_len = _rows_of(s, dev)
    j = lens[b] - q_len + i
    page = s.block_table[b, (j.clamp(min=0) // rows).clamp(max=width - 1)]
    ok = (j >= 0) & (j < width * rows) & (page >= 0)
    s.slots.copy_(torch.where(ok, page * rows + j % rows, -1))
    s.positions.copy_(j.clamp(min=-1))
    s.status.copy_(torch.where((got < take).any() | ((j >= 0) & ~ok).any(), 3, s.status))


def _by_token(pool, s):
    """The pool with (page, row) first, whichever its layout."""
    return pool.permute(0, 2, 1, 3) if s.kv_layout else pool


def _mx_values(codes, scale):
    """E2M1 codes and E8M0 scales as 32-bit values."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return x * _pow2(scale.int() - 127).repeat_interleave(MX_TILE, -1)


def _gathered(s, j):
    """K and V of the keys j [B, N] of each sequence, in 32 bits, [B, KVN, N, D]."""
    page = s.block_table.gather(1, j // s.block_size).long()
    row = j % s.block_size
    got = []
    for pool, scale in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)):
        x = _mx_values(_by_token(pool, s)[page, row], scale.permute(0, 2, 1, 3)[page, row])
        got.append(x.permute(0, 2, 1, 3))
    return got


def _plain_attention(s):
    dev = s.q.device
    kv = s.seqused_kv.long()[:, None]
    i = torch.arange(s.S_q, device=dev)[None]
    if s.layout:
        q_len = (s.cu[1:] - s.cu[:-1]).long()[:, None]
        q = s.q[torch.where(i < q_len, s.cu[:-1].long()[:, None] + i, 0)]  # [B, S, QN, D]
    else:
        q_len = torch.full((s.B, 1), s.S_q, device=dev)
        q = s.q
    p = kv - q_len + i                                    # [B, S] positions of the rows
    n = torch.arange(s.kv_max, device=dev)[None]
    j = torch.where(n < kv, n, 0)
    see = (n < kv)[:, None, :] & (i < q_len)[:, :, None]
    if s.mask_mode:
        see = see & (n <= p[:, :, None])
    if s.mask_mode == 4:
        see = see & ((n >= p[:, :, None] - s.pre_tokens) | (n < s.first_tokens))
    k, v = _gathered(s, j)
    G = s.QN // s.KVN
    qg = q.float().reshape(s.B, s.S_q, s.KVN, G, s.D).permute(0, 2, 1, 3, 4)
    x = qg.reshape(s.B, s.KVN, s.S_q * G, s.D) @ k.transpose(2, 3) * s.scale
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
        return {"out": o[keep], "lse": lse.permute(0, 2, 1, 3).reshape(s.B, s.S_q, s.QN)[keep][..., None]}
    return {"out": o, "lse": lse.permute(0, 1, 3, 2).reshape(s.B, s.QN, s.S_q)[..., None]}


def _store(s, page, row, k, v):
    """K and V rows [T, KVN, D] to their places, in the cache's format."""
    for x, pool, scale in ((k, s.k_cache, s.k_scale), (v, s.v_cache, s.v_scale)):
        if scale is not None:
            x, sc = (_mx if s.kv == "mx" else _e4m3)(x)
            scale.permute(0, 2, 1, 3)[page, row] = sc
        _by_token(pool, s)[page, row] = x.to(pool.dtype)


def _plain_append(s):
    b, i, q_len = _rows_of(s, s.k_new.device)
    slot = s.seqused_kv.long()[b] - q_len + i
    _store(s, s.block_table[b, slot // s.block_size].long(), slot % s.block_size,
           s.k_new.reshape(-1, s.KVN, s.D), s.v_new.reshape(-1, s.KVN, s.D))


def _turned(s, x, weight):
    """The heads normed (where there is a weight) and rotated, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s.eps) * weight.float()
    cos, sin = s.cos_sin[s.positions.long()][:, None].chunk(2, -1)
    r, rest = x[..., :s.rot], x[..., s.rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if s.pairs else r.chunk(2, -1)
    turned = (a * cos - b * sin, b * cos + a * sin)
    r = torch.stack(turned, -1).flatten(-2) if s.pairs else torch.cat(turned, -1)
    return torch.cat([r, rest], -1)


def _plain_rope(s):
    s.q_out.copy_(_turned(s, s.q, s.q_weight))
    slot = s.slots.long()
    _store(s, slot // s.block_size, slot % s.block_size, _turned(s, s.k_new, s.k_weight), s.v_new)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def _seen(c, ql, kl):
    """(row, key) pairs that the mask leaves, and keys that some row sees."""
    if c["mask"] == 0:
        return ql * kl, kl if ql else 0
    p = kl - ql + np.arange(ql, dtype=np.int64)
    p = p[p >= 0]
    if not len(p):
        return 0, 0
    if c["mask"] == 3:
        return int((p + 1).sum()), int(p[-1] + 1)
    lo = np.maximum(p - c["window"] + 1, 0)
    pairs = int((p + 1 - lo + np.minimum(lo, c["first"])).sum())
    return pairs, int(p[-1] + 1 - lo[0] + min(lo[0], c["first"]))


def work(case):
    c = case
    q_lens, kv_lens = _lengths(c)
    KVN, QN, D, rows = c["KVN"], c["QN"], c["D"], c["rows"]
    T = int(q_lens.sum())
    # K and V of one key, one head
    row = 2 * {"bf16": 2 * D, "fp8": D + 4 * D // FP8_TILE, "mx": D // 2 + D // MX_TILE}[c["kv"]]
    if c["op"] == "pages":
        ended = _ended(c)
        need = np.where(ended, 0, -(-kv_lens // rows))
        held = np.where(ended, -(-kv_lens // rows), -(-np.maximum(kv_lens - q_lens, 0) // rows))
        # lengths and counts in and out, a page that moves read and written, the
        # tokens' slots and positions
        return {"bytes": 16 * c["B"] + 8 * int(np.abs(need - held).sum()) + 8 * T, "flops": 0}
    if c["op"] == "attend":
        pairs, keys = (sum(x) for x in zip(*(_seen(c, int(a), int(b)) for a, b in zip(q_lens, kv_lens))))
        return {"bytes": T * QN * (4 * D + 4) + keys * KVN * row, "flops": 4 * D * QN * pairs}
    if c["op"] == "append":
        return {"bytes": T * KVN * (4 * D + row), "flops": 0}
    return {"bytes": T * (QN * 4 * D + KVN * (4 * D + row) + 8)
            + 4 * c["rot"] * min(T, int(kv_lens.max())), "flops": 0}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _exact_cache(s, pool, scale, b, n):
    """Keys 0..n-1 of sequence b in 64 bits, [n, KVN, D], bit by bit of their codes."""
    j = np.arange(n)
    table = s.block_table[b].cpu().numpy()
    page = torch.from_numpy(table[j // s.block_size].astype(np.int64)).to(pool.device)
    row = torch.from_numpy(j % s.block_size).to(pool.device)
    x = (pool[page, :, row] if s.kv_layout else pool[page, row]).long()
    got = torch.empty(n, s.KVN, s.D, dtype=torch.float64, device=pool.device)
    for half in (0, 1):
        code = x >> (4 * half)
        e, m = (code >> 1) & 3, (code & 1).double()
        v = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e.double() - 1), m / 2)
        got[..., half::2] = torch.where(code & 8 > 0, -v, v)
    f = 2.0 ** (scale[page, :, row].double() - 127)
    return (got.reshape(n, s.KVN, -1, MX_TILE) * f[..., None]).reshape(n, s.KVN, s.D)


def _exact_attention(c, s):
    q_lens, kv_lens = _lengths(c)
    outs, lses, G = [], [], s.QN // s.KVN
    t0 = 0
    for b in range(s.B):
        ql, kl = int(q_lens[b]), int(kv_lens[b])
        q = (s.q[t0:t0 + ql] if s.layout else s.q[b]).double()
        t0 += ql
        j = torch.arange(kl, device=s.q.device)
        p = kl - ql + torch.arange(ql, device=s.q.device)[:, None]
        see = (j <= p) | (c["mask"] == 0)
        if c["mask"] == 4:
            see = see & ((j > p - c["window"]) | (j < c["first"]))
        k = _exact_cache(s, s.k_cache, s.k_scale, b, kl)
        v = _exact_cache(s, s.v_cache, s.v_scale, b, kl)
        o = torch.zeros(ql, s.QN, s.D, dtype=torch.float64, device=s.q.device)
        z = torch.full((ql, s.QN), math.inf, dtype=torch.float64, device=s.q.device)
        some = see.any(1)
        for h in range(s.QN):
            x = (q[:, h] @ k[:, h // G].T * s.scale).masked_fill(~see, -math.inf)
            if s.sinks is not None:
                x = torch.cat([x, s.sinks[h].double().expand(ql, 1)], 1)
            l = torch.logsumexp(x, 1)
            w = torch.exp(x - torch.where(some, l, 0)[:, None])[:, :kl]
            w[~some] = 0
            o[:, h] = w @ v[:, h // G]
            z[:, h] = torch.where(some, l, math.inf)
        outs.append(o)
        lses.append(z if s.layout else z.T)
    return {"out": torch.cat(outs) if s.layout else torch.stack(outs),
            "lse": (torch.cat(lses) if s.layout else torch.stack(lses))[..., None]}


def _rounded(x, digits, least, most):
    """x to `digits` significant bits, ties to even, steps of 2^least at the least."""
    e = torch.frexp(x)[1].double() - digits
    step = 2.0 ** torch.clamp(e, min=least)
    return (torch.round(x / step) * step).clamp(-most, most)


def _exact_rows(s, x):
    """Rows [T, KVN, D] in 64 bits as the cache holds them: values (4 bits: bytes), scales."""
    if s.kv == "bf16":
        return x, None
    tile = FP8_TILE if s.kv == "fp8" else MX_TILE
    t = x.reshape(*x.shape[:-1], -1, tile)
    amax = t.abs().amax(-1)
    if s.kv == "fp8":
        scale = torch.where(amax > 0, amax / FP8_MAX, 1.0)
        return _rounded(t / scale[..., None], 4, -9, FP8_MAX).reshape(x.shape), scale
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax / 6, 1.0)))
    e = torch.where(6 * 2.0 ** (e - 1) >= amax, e - 1, torch.where(6 * 2.0 ** e < amax, e + 1, e))
    e = torch.where(amax > 0, e, 0).clamp(-127, 127)
    v = _rounded(t / (2.0 ** e)[..., None], 2, -1, 6.0).reshape(x.shape)
    code = (v.abs()[..., None] > torch.tensor(E2M1, device=x.device)).sum(-1) + 8 * torch.signbit(x)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), (e + 127).to(torch.uint8)


def _exact_store(s, page, row, k, v):
    got = {}
    for name, x in (("k", k), ("v", v)):
        val, scale = _exact_rows(s, x)
        pool = getattr(s, name + "_cache")
        kept = pool.view(torch.float8_e4m3fn).float().double() if s.kv == "fp8" else \
            pool.double() if s.kv == "bf16" else pool.clone()
        if s.kv_layout:
            kept[page, :, row] = val
        else:
            kept[page, row] = val
        got[name] = kept
        if scale is not None:
            sc = getattr(s, name + "_scale")
            sc = sc.double() if s.kv == "fp8" else sc.clone()
            sc[page, :, row] = scale
            got[name + "_scale"] = sc
    return got


def _exact_append(c, s):
    q_lens, kv_lens = _lengths(c)
    table, rows = s.block_table.cpu().numpy(), s.block_size
    j = [np.arange(n - q, n) for q, n in zip(q_lens, kv_lens)]
    page = np.concatenate([table[b, x // rows] for b, x in enumerate(j)]).astype(np.int64)
    page, row = (torch.from_numpy(x).to(s.k_new.device) for x in (page, np.concatenate(j) % rows))
    return _exact_store(s, page, row, s.k_new.double().reshape(-1, s.KVN, s.D),
                        s.v_new.double().reshape(-1, s.KVN, s.D))


def _exact_rope(c, s):
    """Each rotated pair as one complex number times e^(i angle)."""
    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s.D + s.eps) * w.double()
        row = s.cos_sin.double()[s.positions.long()]
        turn = torch.complex(row[:, :s.rot // 2], row[:, s.rot // 2:])[:, None]
        i = torch.arange(s.rot // 2, device=x.device)
        first, second = (2 * i, 2 * i + 1) if s.pairs else (i, i + s.rot // 2)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    slot = s.slots.long()
    kept = _exact_store(s, slot // s.block_size, slot % s.block_size, turned(s.k_new, s.k_weight),
                        s.v_new.double())
    return {"q": turned(s.q, s.q_weight), **kept}


def exact(case, seed):
    if case["op"] == "pages":  # whole numbers alone
        return None
    if case["op"] == "attend":
        return None if work(case)["flops"] > 6e12 else _exact_attention(case, prepare(case, seed))
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_rope(case, s)
