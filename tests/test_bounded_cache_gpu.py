"""The bounded cache on the GPU: append, window attention with first tokens,
attention that counts key weights, eviction, and a run of them together, each
against its definition in 64 bits (bounded.py, which holds the tolerances)."""
import numpy as np
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import bounded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


# ----------------------------------------------------------------------------
# append
# ----------------------------------------------------------------------------

def _empty_cache(B, KVN, D, pages, block, fp8, kv_layout, paged=True, seed=0, fill=None):
    """A cache filled with marks, its tensors and table (pages shuffled)."""
    g = torch.Generator().manual_seed(seed)
    nb = B * pages + 3
    head_major = kv_layout == fia.KV_LAYOUT_BNNBSD
    shape = ((nb, KVN, block, D) if head_major else (nb, block, KVN, D)) if paged \
        else (B, pages * block, KVN, D)
    dt = torch.uint8 if fp8 else torch.bfloat16
    mk = (lambda: torch.randint(0, 100, shape, generator=g).to(dt))
    k, v = mk().to(DEV), mk().to(DEV)
    ks = vs = None
    if fp8:
        ss = (nb, KVN, block, D // 64) if paged else (B, KVN, pages * block, D // 64)
        ks, vs = (torch.rand(ss, generator=g).to(DEV) for _ in range(2))
    table = None
    if paged:
        table = torch.randperm(nb, generator=g)[:B * pages].reshape(B, pages).int().to(DEV)
    cache = fia.KvCache(k, v, table, k_scale=ks, v_scale=vs, kv_layout=kv_layout)
    return cache, [k, v, ks, vs, table]


def _place(tensors, name, b, h, j, block, kv_layout):
    """The tensor `name` (0 K, 1 V, 2 / 3 scales) and the index of key j."""
    table = tensors[4]
    if table is None:
        return (b, h, j) if name >= 2 else (b, j, h)
    page, row = int(table[b, j // block]), j % block
    return (page, h, row) if name >= 2 or kv_layout == fia.KV_LAYOUT_BNNBSD else (page, row, h)


APPEND = {
    "token": dict(B=3, q=[1, 1, 1], kv=[1, 33, 96], bsnd=True),
    "rows": dict(B=2, q=[4, 4], kv=[4, 70], bsnd=True),
    "ragged": dict(B=4, q=[5, 0, 37, 1], kv=[5, 0, 90, 64]),
    "one": dict(B=1, q=[1], kv=[1]),
    "full": dict(B=2, q=[96, 3], kv=[96, 96]),
}


@pytest.mark.parametrize("kv_layout", [0, 1, None])
@pytest.mark.parametrize("fp8,D", [(False, 128), (False, 64), (True, 128)])
@pytest.mark.parametrize("name", sorted(APPEND))
def test_append_writes_its_rows_and_nothing_else(name, fp8, D, kv_layout):
    c, KVN, block, pages = APPEND[name], 3, 32, 3
    cache, t = _empty_cache(c["B"], KVN, D, pages, block, fp8, kv_layout or 0,
                            paged=kv_layout is not None, seed=1)
    g = torch.Generator().manual_seed(2)
    T = sum(c["q"])
    x = [torch.randn(T, KVN, D, generator=g).to(torch.bfloat16) for _ in range(2)]
    if T > 2:
        x[0][1, 0, :64] = 0                       # an all-zero tile
        x[0][0, 1, 3], x[1][1, 1, D - 2] = float("nan"), float("inf")
        x[1][0, 2, :] = 9.2e-41                   # below the normal range
    cap = block * pages
    weights = torch.rand(c["B"], KVN, cap + 5, generator=g).to(DEV)
    positions = torch.full((c["B"], KVN, cap + 5), -7, dtype=torch.int32, device=DEV)
    seen = torch.tensor([n + 1000 * (b + 1) for b, n in enumerate(c["kv"])], dtype=torch.int32)
    want = [None if a is None else a.cpu().clone() for a in t]
    want_w, want_p = weights.cpu().clone(), positions.cpu().clone()
    i = 0
    for b in range(c["B"]):
        for r in range(c["q"][b]):
            j = c["kv"][b] - c["q"][b] + r
            for h in range(KVN):
                for kv in range(2):
                    row = x[kv][i, h]
                    if fp8:
                        code, scale = bounded.quantised(row)
                        want[2 + kv][_place(t, 2 + kv, b, h, j, block, kv_layout)] = \
                            torch.from_numpy(scale)
                        row = torch.from_numpy(code)
                    want[kv][_place(t, kv, b, h, j, block, kv_layout)] = row
                want_w[b, h, j] = 0
                want_p[b, h, j] = int(seen[b]) - c["q"][b] + r
            i += 1
    dev = [a.to(DEV) for a in x]
    cu = None
    if c.get("bsnd"):
        dev = [a.unflatten(0, (c["B"], -1)) for a in dev]
    else:
        cu = torch.tensor([0] + list(np.cumsum(c["q"])), dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    fia.kv_append(cache, *dev, torch.tensor(c["kv"], dtype=torch.int32, device=DEV),
                  cu_seqlens_q=cu, weights=weights, positions=positions, tokens_seen=seen.to(DEV),
                  status=status)
    for a, w in zip(t, want):
        if a is not None:
            a, w = a.cpu(), w
            if a.dtype == torch.bfloat16:
                a, w = a.view(torch.int16), w.view(torch.int16)
            assert torch.equal(a, w)
    assert torch.equal(weights.cpu(), want_w) and torch.equal(positions.cpu(), want_p)
    assert int(status) == 0


def test_append_takes_slices_of_a_fused_projection():
    B, KVN, D, S = 3, 2, 128, 5
    cache, t = _empty_cache(B, KVN, D, 2, 32, False, 0)
    cache2, t2 = _empty_cache(B, KVN, D, 2, 32, False, 0)
    qkv = torch.randn(B, S, 8 + 2 * KVN, D, device=DEV).to(torch.bfloat16)
    lens = torch.tensor([5, 20, 64], dtype=torch.int32, device=DEV)
    k, v = qkv[:, :, 8:8 + KVN], qkv[:, :, 8 + KVN:]
    fia.kv_append(cache, k, v, lens)
    fia.kv_append(cache2, k.contiguous(), v.contiguous(), lens)
    assert torch.equal(t[0], t2[0]) and torch.equal(t[1], t2[1])
    one = qkv[:, :1]  # one token per sequence: the batch stride is the token stride
    fia.kv_append(cache, one[:, :, 8:8 + KVN], one[:, :, 8 + KVN:], lens)
    fia.kv_append(cache2, one[:, :, 8:8 + KVN].contiguous(), one[:, :, 8 + KVN:].contiguous(), lens)
    assert torch.equal(t[0], t2[0]) and torch.equal(t[1], t2[1])


def test_append_leaves_out_rows_without_a_place():
    B, KVN, D, block = 4, 2, 64, 16
    cache, t = _empty_cache(B, KVN, D, 2, block, False, 0)
    t[4][2, 0] = 10_000_000  # a page outside the pool
    t[4][3, 1] = -1
    before = [t[0].clone(), t[1].clone()]
    new = torch.randn(B, 2, KVN, D, device=DEV).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    # rows before the start, past the capacity, and in those two pages
    lens = torch.tensor([1, 33, 2, 18], dtype=torch.int32, device=DEV)
    pos = torch.zeros(B, KVN, 32, dtype=torch.int32, device=DEV)
    fia.kv_append(cache, new, new, lens, status=status, positions=pos)
    assert int(status) == 3
    want = before[0].clone()
    for b, j, r in ((0, 0, 1), (1, 31, 0)):
        want[int(t[4][b, j // block]), j % block] = new[b, r]
    assert torch.equal(t[0], want)
    assert int((pos != 0).sum()) == KVN  # slot 31's; slot 0 is position 0


@pytest.mark.parametrize("fp8", [False, True])
def test_append_of_a_padded_batch_is_no_error(fp8):
    """Rows before the first sequence and behind the last are nobody's."""
    B, KVN, D, block = 2, 2, 128, 32
    cache, t = _empty_cache(B, KVN, D, 2, block, fp8, 0)
    clean, t2 = _empty_cache(B, KVN, D, 2, block, fp8, 0)
    new = torch.randn(40, KVN, D, device=DEV).to(torch.bfloat16)
    lens = torch.tensor([5, 40], dtype=torch.int32, device=DEV)
    cu = torch.tensor([2, 7, 11], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = torch.full((B, KVN, 64), 3.0, device=DEV)
    fia.kv_append(cache, new, new, lens, cu_seqlens_q=cu, status=status, weights=w)
    fia.kv_append(clean, new[2:11].contiguous(), new[2:11].contiguous(), lens, cu_seqlens_q=cu - 2)
    assert int(status) == 0
    for x, y in zip(t, t2):
        assert x is None or torch.equal(x, y)
    want = torch.full((B, KVN, 64), 3.0)
    want[0, :, :5], want[1, :, 36:40] = 0, 0
    assert torch.equal(w.cpu(), want)


# ----------------------------------------------------------------------------
# window attention with first tokens
# ----------------------------------------------------------------------------

def _hide_unseen(p, spare):
    """Point the table entries of pages that lie wholly in KV tiles no row sees
    at a poisoned page: they must never be read."""
    t = p.block_table
    for b in range(p.B):
        ql, kl = p.q_lens[b], p.kv_lens[b]
        lo = max(kl - ql - p.pre_tokens, 0) // 128
        nf = -(-min(p.first_tokens, kl) // 128)
        for page in range(-(-kl // p.block_size)):
            j0, j1 = page * p.block_size, (page + 1) * p.block_size - 1
            if j0 // 128 >= nf and j1 // 128 < lo:
                t[b, page] = spare
    return p


def _window(**kw):
    kw.setdefault("QN", 8)
    kw.setdefault("KVN", 2)
    kw.setdefault("D", 128)
    kw.setdefault("block_size", 32)
    kw.setdefault("next_tokens", 0)
    kw.setdefault("layout", fi.LAYOUT_TND)
    p = fi.make_fia(mask_mode=fi.MASK_BAND, device=DEV, **kw)
    if p.block_table is not None:
        used = set(p.block_table.flatten().tolist())
        spare = next(x for x in range(p.num_blocks) if x not in used) \
            if len(used) < p.num_blocks else None
        if spare is not None:
            _hide_unseen(p, spare)
    return p


# CTAs too few for a cluster: a call of few units that runs in one kernel
# otherwise takes the kernels of the larger ones
NO_CLUSTER = 7


def _check(p):
    for num_sms in (0, NO_CLUSTER):
        _check_on(p, num_sms)


def _check_on(p, num_sms):
    call = fia.FiaCall(p, num_sms=num_sms)
    out, lse = call.run()
    torch.cuda.synchronize()
    bounded.check_attention(p, out, lse)
    assert call.error_word() == 0
    first = (out.clone(), lse.clone())
    out, lse = call.run()  # the same bits again
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


WINDOW_DECODE = {
    "short": dict(kv_lens=[1, 2, 5, 130], pre_tokens=63, first_tokens=4),
    "gap": dict(kv_lens=[1500, 900, 513, 512], pre_tokens=255, first_tokens=4),
    "far": dict(kv_lens=[5000, 129, 4097, 2048], pre_tokens=1000, first_tokens=130),
    "first_only_window_of_one": dict(kv_lens=[700, 1, 300, 257], pre_tokens=0, first_tokens=1),
    "many_first": dict(kv_lens=[3000, 1, 300, 257], pre_tokens=100, first_tokens=1030),
    "first_past_the_end": dict(kv_lens=[300, 40, 1, 0], pre_tokens=16, first_tokens=1 << 30),
    "empty_and_ahead": dict(kv_lens=[0, 64, 2, 1], pre_tokens=-1, first_tokens=2, next_tokens=1),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("name", sorted(WINDOW_DECODE))
def test_window_decode(name, rows, fp8):
    c = dict(WINDOW_DECODE[name])
    _check(_window(B=4, q_lens=[rows, 1, rows, rows], seed=3, with_sinks=rows == 3,
                   kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16, **c))


@pytest.mark.parametrize("QN,KVN,D", [(1, 1, 64), (7, 1, 128), (16, 1, 128), (12, 2, 64),
                                      (64, 4, 128)])
def test_window_decode_heads(QN, KVN, D):
    _check(_window(B=2, QN=QN, KVN=KVN, D=D, q_lens=[1, 1], kv_lens=[1111, 300], seed=5,
                   pre_tokens=200, first_tokens=5, layout=fi.LAYOUT_BSND))


@pytest.mark.parametrize("block,kv_layout,paged", [(16, 0, True), (48, 1, True), (272, 0, True),
                                                   (1024, 1, True), (0, 0, False)])
def test_window_decode_caches(block, kv_layout, paged):
    kw = dict(block_size=block, kv_layout=kv_layout) if paged else dict(paged=False, S_kv=2600)
    _check(_window(B=3, q_lens=[1, 2, 1], kv_lens=[2600, 1000, 77], seed=6, pre_tokens=300,
                   first_tokens=20, **kw))


def test_window_decode_of_long_caches_splits_over_the_window_and_the_first_tokens():
    _check(_window(B=2, QN=8, KVN=1, q_lens=[1, 1], kv_lens=[40000, 33000], seed=7,
                   block_size=128, pre_tokens=20000, first_tokens=6000))
    _check(_window(B=1, QN=4, KVN=1, q_lens=[2], kv_lens=[40000], seed=8, block_size=16,
                   pre_tokens=9000, first_tokens=3000, kv_dtype=fi.KV_BF16))


WINDOW_PREFILL = {
    "fresh": dict(q_lens=[300, 17, 1, 257], kv_lens=[300, 17, 1, 257], pre_tokens=63,
                  first_tokens=4),
    "chunk": dict(q_lens=[130, 40, 0, 1], kv_lens=[1400, 900, 300, 800], pre_tokens=200,
                  first_tokens=4),
    "many_first": dict(q_lens=[200, 33], kv_lens=[1000, 1200], pre_tokens=50, first_tokens=300),
    "query_longer_than_keys": dict(q_lens=[150, 20], kv_lens=[100, 1], pre_tokens=30,
                                   first_tokens=3),
    "window_of_one": dict(q_lens=[300], kv_lens=[700], pre_tokens=0, first_tokens=1),
    "ahead": dict(q_lens=[200, 64], kv_lens=[600, 64], pre_tokens=-2, next_tokens=9,
                  first_tokens=7),
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "d64"])
@pytest.mark.parametrize("name", sorted(WINDOW_PREFILL))
def test_window_prefill(name, kind):
    c = dict(WINDOW_PREFILL[name])
    _check(_window(B=len(c["q_lens"]), seed=11, with_sinks=name == "chunk",
                   D=64 if kind == "d64" else 128, QN=6 if name == "fresh" else 8,
                   kv_dtype=fi.KV_FP8_E4M3 if kind == "fp8" else fi.KV_BF16, **c))


def test_window_prefill_long_gap_head_major_and_negative_scale():
    _check(_window(B=1, q_lens=[140], kv_lens=[5000], pre_tokens=600, first_tokens=150, seed=12,
                   block_size=64, kv_layout=1))
    _check(_window(B=1, q_lens=[140], kv_lens=[1500], pre_tokens=300, first_tokens=10, seed=13,
                   scale=-0.05))


def test_first_tokens_zero_is_the_band():
    for ql in (1, 40):
        a = _window(B=2, q_lens=[ql, ql], kv_lens=[900, 333], pre_tokens=100, seed=14)
        b = _window(B=2, q_lens=[ql, ql], kv_lens=[900, 333], pre_tokens=100, seed=14,
                    first_tokens=1)
        out, lse = fia.FiaCall(a).run()
        bounded.check_attention(a, out, lse)
        out1, _ = fia.FiaCall(b).run()
        assert not torch.equal(out, out1)


def test_window_wider_than_the_cache_is_causal():
    for ql in (1, 3, 70):
        # (a table for long caches, so that the same kernel runs for both)
        kw = dict(B=2, q_lens=[ql, ql], kv_lens=[700, 200], seed=15, max_blocks=300)
        a = _window(pre_tokens=1 << 20, first_tokens=4, **kw)
        b = fi.make_fia(QN=8, KVN=2, D=128, block_size=32, layout=fi.LAYOUT_TND, device=DEV,
                        mask_mode=fi.MASK_RIGHT_DOWN_CAUSAL, **kw)
        ra, rb = fia.FiaCall(a).run(), fia.FiaCall(b).run()
        assert torch.equal(ra[0], rb[0]) and torch.equal(ra[1], rb[1])


# ----------------------------------------------------------------------------
# key weights
# ----------------------------------------------------------------------------

def _check_weights(p, with_in=True, seed=1):
    for num_sms in (0, NO_CLUSTER):
        _check_weights_on(p, num_sms, with_in, seed)


def _check_weights_on(p, num_sms, with_in, seed):
    g = torch.Generator().manual_seed(seed)
    cap = p.S_kv if p.block_table is None else p.block_table.shape[1] * p.block_size
    w_in = (torch.rand(p.B, p.KVN, cap, generator=g).to(DEV) if with_in else None)
    mark = torch.full((p.B, p.KVN, cap), -3.0, device=DEV)
    call = fia.KeyWeightsCall(p, weights=w_in, weights_out=mark.clone(), num_sms=num_sms)
    out, lse, w = call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 0
    bounded.check_attention(p, out, lse, w, w_in)
    for b in range(p.B):
        assert torch.all(w[b, :, p.kv_lens[b]:] == -3.0), "slots past the keys were written"
    plain, plain_lse = fia.FiaCall(p, num_sms=num_sms).run()
    if num_sms == NO_CLUSTER or 9 * p.B * p.KVN > 2 * 152:  # (one kernel runs in both)
        assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
    bounded.check_attention(p, plain, plain_lse)
    first = w.clone()
    call.weights_out.copy_(mark)
    assert torch.equal(call.run()[2], first), "the same bits again"
    if with_in:  # in place
        again = fia.KeyWeightsCall(p, weights=w_in, weights_out=w_in, num_sms=num_sms)
        again.run()
        for b in range(p.B):
            assert torch.equal(w_in[b, :, :p.kv_lens[b]], first[b, :, :p.kv_lens[b]])


WEIGHTS_DECODE = {
    "one_row": dict(q_lens=[1, 1, 1, 1], kv_lens=[1, 130, 777, 64]),
    "ragged_rows": dict(q_lens=[3, 0, 1, 4], kv_lens=[500, 40, 1, 4]),
    "causal_none": dict(q_lens=[5, 2, 1, 1], kv_lens=[3, 1, 0, 9]),
    "all_rows": dict(q_lens=[2, 16, 7, 1], kv_lens=[200, 300, 7, 129], mask_mode=fi.MASK_NONE),
    "left_up": dict(q_lens=[2, 16, 7, 1], kv_lens=[200, 300, 7, 129],
                    mask_mode=fi.MASK_LEFT_UP_CAUSAL),
    "window": dict(q_lens=[1, 3, 1, 2], kv_lens=[900, 1300, 40, 513], mask_mode=fi.MASK_BAND,
                   pre_tokens=200, first_tokens=5),
    "masked": dict(q_lens=[2, 3, 1, 2], kv_lens=[300, 200, 40, 130], mask_mode=fi.MASK_ALL,
                   mask_density=0.6, mask_full_rows=1),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", sorted(WEIGHTS_DECODE))
def test_weights_decode(name, fp8):
    c = dict(WEIGHTS_DECODE[name])
    c.setdefault("mask_mode", fi.MASK_RIGHT_DOWN_CAUSAL)
    _check_weights(fi.make_fia(B=4, QN=8, KVN=2, D=128, block_size=32, layout=fi.LAYOUT_TND,
                               device=DEV, seed=21, with_sinks=name == "one_row",
                               kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16, **c),
                   with_in=name != "left_up")


@pytest.mark.parametrize("QN,KVN,D,rows", [(1, 1, 64, 1), (3, 1, 128, 1), (16, 1, 128, 1),
                                           (21, 3, 64, 2), (64, 1, 128, 1), (6, 2, 128, 16)])
def test_weights_decode_heads(QN, KVN, D, rows):
    _check_weights(fi.make_fia(B=2, QN=QN, KVN=KVN, D=D, q_lens=[rows, rows], kv_lens=[333, 1200],
                               block_size=64, device=DEV, seed=22, mask_mode=3))


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("block,kv_layout,paged", [(16, 1, True), (48, 0, True), (0, 0, False)])
def test_weights_caches(block, kv_layout, paged, rows):
    kw = dict(block_size=block, kv_layout=kv_layout) if paged else dict(paged=False, S_kv=700)
    _check_weights(fi.make_fia(B=2, QN=8, KVN=4, D=128, q_lens=[rows, rows], kv_lens=[700, 77],
                               layout=fi.LAYOUT_TND, device=DEV, seed=23, mask_mode=3, **kw))


def test_weights_of_a_long_cache():
    _check_weights(fi.make_fia(B=2, QN=8, KVN=1, D=128, q_lens=[1, 1], kv_lens=[30000, 20001],
                               block_size=128, device=DEV, seed=24, mask_mode=3))


WEIGHTS_PREFILL = {
    "fresh": dict(q_lens=[300, 17, 1, 257], kv_lens=[300, 17, 1, 257]),
    "chunk": dict(q_lens=[130, 40, 0, 1], kv_lens=[700, 400, 300, 500], with_sinks=True),
    "query_longer": dict(q_lens=[300, 20], kv_lens=[100, 0]),
    "all_keys": dict(q_lens=[200, 33], kv_lens=[150, 300], mask_mode=fi.MASK_NONE),
    "left_up": dict(q_lens=[200, 33], kv_lens=[150, 300], mask_mode=fi.MASK_LEFT_UP_CAUSAL),
    "window": dict(q_lens=[300, 140], kv_lens=[300, 1500], mask_mode=fi.MASK_BAND, pre_tokens=70,
                   first_tokens=5),
    "ahead": dict(q_lens=[200, 64], kv_lens=[600, 64], mask_mode=fi.MASK_BAND, pre_tokens=-2,
                  next_tokens=9),
    "masked": dict(q_lens=[150, 60], kv_lens=[300, 77], mask_mode=fi.MASK_NONE, mask_density=0.5,
                   mask_full_rows=2),
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "d64"])
@pytest.mark.parametrize("name", sorted(WEIGHTS_PREFILL))
def test_weights_prefill(name, kind):
    c = dict(WEIGHTS_PREFILL[name])
    c.setdefault("mask_mode", fi.MASK_RIGHT_DOWN_CAUSAL)
    _check_weights(fi.make_fia(B=len(c["q_lens"]), QN=6 if name == "fresh" else 8, KVN=2,
                               D=64 if kind == "d64" else 128, block_size=32,
                               layout=fi.LAYOUT_TND, device=DEV, seed=25,
                               kv_dtype=fi.KV_FP8_E4M3 if kind == "fp8" else fi.KV_BF16, **c),
                   with_in=name != "chunk")


def test_weights_prefill_batch_layout_and_negative_scale():
    _check_weights(fi.make_fia(B=3, QN=4, KVN=1, D=128, q_lens=[70] * 3, kv_lens=[70, 200, 500],
                               device=DEV, seed=26, mask_mode=3, scale=-0.06))


@pytest.mark.parametrize("layout", [fi.LAYOUT_TND, fi.LAYOUT_BSND])
def test_weights_without_query_rows_are_what_they_were(layout):
    p = fi.make_fia(B=2, QN=4, KVN=2, D=128, q_lens=[1, 1], kv_lens=[50, 3], layout=layout,
                    device=DEV, seed=27, mask_mode=3)
    w_in = torch.rand(2, 2, p.block_table.shape[1] * p.block_size, device=DEV)
    call = fia.KeyWeightsCall(p, weights=w_in)
    if layout == fi.LAYOUT_TND:
        p.cu_seqlens_q.zero_()
        call.params.total_q = 0
    else:
        call.params.max_seqlen_q = 0
    got = call.run()[2]
    for b, n in enumerate(p.kv_lens):
        assert torch.equal(got[b, :, :n], w_in[b, :, :n]) and torch.all(got[b, :, n:] == 0)


def test_weights_without_a_plan_are_not_written():
    for ql in (1, 40):
        p = fi.make_fia(B=1, QN=4, KVN=2, D=128, q_lens=[ql], kv_lens=[90], device=DEV, seed=28,
                        mask_mode=3)
        call = fia.KeyWeightsCall(p)
        call.ws.zero_()
        call.weights_out.fill_(5.0)
        call.execute()
        torch.cuda.synchronize()
        assert call.error_word() == 2
        assert torch.all(call.weights_out == 5.0)


# ----------------------------------------------------------------------------
# evict
# ----------------------------------------------------------------------------

def _evict_case(lens, budget, first=0, recent=0, positions=True, seen=True, KVN=3, D=128,
                fp8=False, kv_layout=0, paged=True, block=32, pages=None, kind="spread", seed=0,
                in_place=False, extra=0):
    B = len(lens)
    pages = pages or -(-max(max(lens), budget, 1) // block)
    cache, t = _empty_cache(B, KVN, D, pages, block, fp8, kv_layout, paged, seed)
    g = torch.Generator().manual_seed(seed + 1)
    cap = pages * block
    w = torch.randn(B, KVN, cap + extra, generator=g)
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float() * torch.where(
            torch.rand(w.shape, generator=g) < 0.5, 1.0, -0.0)
    elif kind == "equal":
        w.fill_(0.25)
    elif kind == "hard":
        pick = torch.tensor([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 3e38])
        w = pick[torch.randint(0, len(pick), w.shape, generator=g)]
    elif kind == "near":  # equal but for the last bits
        w = (torch.randint(0, 700, w.shape, generator=g) + 0x3F800000).int().view(torch.float32)
    for b, n in enumerate(lens):
        w[b, :, max(n, 0):] = float("nan")  # behind the keys: anything
    seen_n = [max(n, 0) + (37 * (b + 1) if seen else 0) for b, n in enumerate(lens)]
    pos = None
    if positions:
        pos = torch.zeros(B, KVN, cap + extra, dtype=torch.int32)
        for b, n in enumerate(lens):
            for h in range(KVN):
                m = min(max(n, 0), cap)
                pos[b, h, :m] = torch.randperm(seen_n[b], generator=g)[:m].int()
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    wd = w.to(DEV)
    pd = None if pos is None else pos.to(DEV)
    kw = {}
    if in_place:
        kw = dict(weights_out=wd, positions_out=pd)
    else:
        kw = dict(weights_out=torch.full_like(wd, -9.0),
                  positions_out=torch.full_like(wd, -9, dtype=torch.int32))
    before = [None if a is None else a.cpu().clone() for a in t]
    call = fia.KvEvictCall(cache, lens_t, wd, budget=budget, first_tokens=first,
                           recent_tokens=recent, positions=pd, status=status,
                           tokens_seen=torch.tensor(seen_n, dtype=torch.int32, device=DEV)
                           if seen else None, **kw)
    n_out, w_out, p_out = call.run()
    torch.cuda.synchronize()
    assert int(status) == 0
    want = [None if a is None else a.clone() for a in before]
    pw = torch.arange(cap + extra).expand(B, KVN, -1) if pos is None else pos
    want_w = w.clone() if in_place else torch.full_like(w, -9.0)
    want_p = (pos.clone() if in_place else torch.full(w.shape, -9)).int() \
        if p_out is not None else None
    clamped = [min(max(n, 0), cap) for n in lens]
    for b, h, m, hole, tail in bounded.evicted(w.numpy(), None if pos is None else pos.numpy(),
                                               clamped, budget, first, recent, seen_n):
        assert int(n_out[b]) == m
        hole, tail = torch.from_numpy(hole), torch.from_numpy(tail)
        assert len(hole) == len(tail)
        want_w[b, h, :m] = w[b, h, :m]
        want_w[b, h, hole] = w[b, h, tail]
        if want_p is not None:
            want_p[b, h, :m] = pw[b, h, :m].int()
            want_p[b, h, hole] = pw[b, h, tail].int()
        for x, y in zip(hole.tolist(), tail.tolist()):
            for name in range(4):
                if want[name] is not None:
                    want[name][_place(t, name, b, h, x, block, kv_layout)] = \
                        before[name][_place(t, name, b, h, y, block, kv_layout)]
    assert torch.equal(w_out.cpu().view(torch.int32), want_w.view(torch.int32))
    if want_p is not None:
        assert torch.equal(p_out.cpu(), want_p)
    for a, x in zip(t, want):
        if a is not None:
            a = a.cpu()
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                               x.view(torch.int16) if x.dtype == torch.bfloat16 else x)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "hard", "near"])
@pytest.mark.parametrize("fp8,kv_layout,paged", [(False, 0, True), (True, 1, True),
                                                 (True, 0, False)])
def test_evict(kind, fp8, kv_layout, paged):
    _evict_case([100, 61, 60, 59, 1, 0, 97], 60, first=4, recent=20, kind=kind, fp8=fp8,
                kv_layout=kv_layout, paged=paged)


@pytest.mark.parametrize("kw", [
    dict(lens=[5, 1, 2], budget=1), dict(lens=[64, 64, 63], budget=64),
    dict(lens=[1000, 300], budget=7, first=3, recent=4, kind="ties"),
    dict(lens=[2000, 1025, 1024], budget=1000, recent=1000, KVN=1, D=64),
    dict(lens=[90, 33], budget=32, first=32, positions=False, seen=False),
    dict(lens=[90, 33], budget=40, recent=5, positions=False, seen=True),
    dict(lens=[90, 33], budget=40, first=8, recent=32, in_place=True),
    dict(lens=[90, 700], budget=40, extra=11, kind="hard", in_place=True),
    dict(lens=[-3, 200], budget=40, pages=6),  # below 0 and past the capacity
])
def test_evict_shapes(kw):
    kw = dict(kw)
    _evict_case(kw.pop("lens"), kw.pop("budget"), **kw)


@pytest.mark.parametrize("lens,budget,KVN", [([9000, 4097, 4096, 12345], 4096, 1),
                                             ([70000], 1024, 1), ([33000, 20000], 20000, 2)])
@pytest.mark.parametrize("kind", ["spread", "near", "equal"])
def test_evict_long(lens, budget, KVN, kind):
    _evict_case(lens, budget, first=4, recent=256, KVN=KVN, D=64, block=128, kind=kind, seed=3)


def test_evict_reports_pages_outside_the_pool():
    cache, t = _empty_cache(1, 2, 64, 4, 16, False, 0)
    t[4][0, 0] = -5
    before = t[0].clone()
    w = torch.arange(64, device=DEV).float().expand(1, 2, 64).contiguous()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    n, wo, po = fia.kv_evict(cache, torch.tensor([64], dtype=torch.int32, device=DEV), w, budget=40,
                             status=status)
    assert int(status) == 3 and int(n) == 40
    # the largest weights are the last slots: 40..63 move into 0..23, of which
    # 0..15 lie in the bad page
    assert torch.equal(po[0, 0, :24].cpu(), torch.arange(40, 64, dtype=torch.int32))
    want = before.clone()
    for k in range(16, 24):
        want[int(t[4][0, k // 16]), k % 16] = before[int(t[4][0, (40 + k) // 16]), (40 + k) % 16]
    assert torch.equal(t[0], want)


# ----------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------

class _Problem:
    """The fields of one attention call over a live cache."""

    def __init__(self, q, cache, t, lens, layout, cu, QN, S_q, scale, kv_layout=0):
        self.q, self.B, self.QN, self.KVN, self.D = q, cache.batch, QN, cache.num_kv_heads, \
            cache.head_dim
        self.layout, self.S_q, self.T = layout, S_q, q.shape[0] if layout else 0
        self.cu_seqlens_q, self.seqused_kv = cu, lens
        self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.block_table = t
        self.kv_dtype = cache.params.kv_dtype
        self.block_size, self.num_blocks = cache.params.block_size, cache.params.num_blocks
        self.S_kv, self.scale, self.kv_layout = cache.capacity, scale, kv_layout
        self.mask_mode, self.pre_tokens, self.next_tokens = fi.MASK_RIGHT_DOWN_CAUSAL, 0, 0
        self.first_tokens, self.sinks, self.atten_mask = 0, None, None
        self.q_lens = self.kv_lens = None

    def to(self, device):
        import copy
        c = copy.copy(self)
        for k, v in vars(self).items():
            if isinstance(v, torch.Tensor):
                setattr(c, k, v.to(device))
        return c


@pytest.mark.parametrize("fp8", [False, True])
def test_a_bounded_chat(fp8):
    """Prompts appended and attended with weights, cut to the budget, then tokens
    one by one: append, attend, evict whenever the budget is passed by a page.
    Every attention is checked in 64 bits against the cache as it then stands,
    the kept keys against the tokens they were."""
    B, QN, KVN, D, block, budget, recent = 3, 8, 2, 128, 32, 96, 40
    cache, t = _empty_cache(B, KVN, D, 8, block, fp8, 0)
    g = torch.Generator().manual_seed(9)
    cap = cache.capacity
    weights = torch.zeros(B, KVN, cap, device=DEV)
    positions = torch.zeros(B, KVN, cap, dtype=torch.int32, device=DEV)
    prompt = [200, 60, 131]
    history = [[], []]  # every token's K and V as it was appended, per sequence

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16)

    seen = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    lens = seen.clone()
    cu = torch.tensor([0] + list(np.cumsum(prompt)), dtype=torch.int32, device=DEV)
    new = [rnd(sum(prompt), KVN, D) for _ in range(2)]
    for kv in range(2):
        history[kv] = [list(x) for x in torch.split(new[kv], prompt)]
    fia.kv_append(cache, new[0].to(DEV), new[1].to(DEV), lens, cu_seqlens_q=cu, weights=weights,
                  positions=positions, tokens_seen=seen)
    steps, evictions = 70, 0
    for step in range(steps + 1):
        if step:
            seen, lens = seen + 1, lens + 1
            new = [rnd(B, 1, KVN, D) for _ in range(2)]
            for kv in range(2):
                for b in range(B):
                    history[kv][b].append(new[kv][b, 0])
            fia.kv_append(cache, new[0].to(DEV), new[1].to(DEV), lens, weights=weights,
                          positions=positions, tokens_seen=seen)
        q = rnd(sum(prompt), QN, D) if step == 0 else rnd(B, 1, QN, D)
        p = _Problem(q.to(DEV), cache, t, lens, 0 if step else 1, None if step else cu, QN,
                     1 if step else max(prompt), D ** -0.5)
        p.q_lens, p.kv_lens = ([1] * B if step else prompt), lens.tolist()
        w_in = weights.clone()
        out, lse, _ = fia.KeyWeightsCall(p, weights=weights, weights_out=weights).run()
        if step % 17 == 0 or step == steps:
            bounded.check_attention(p, out, lse, weights, w_in)
        if step == 0 or int(lens.max()) >= budget + block:
            w0, p0, n0 = weights.cpu().numpy(), positions.cpu().numpy(), lens.tolist()
            lens, weights, positions = fia.kv_evict(
                cache, lens, weights, budget=budget, first_tokens=4, recent_tokens=recent,
                positions=positions, tokens_seen=seen)
            evictions += 1
            for b, h, m, hole, tail in bounded.evicted(w0, p0, n0, budget, 4, recent,
                                                       seen.tolist()):
                want = p0[b, h].copy()
                want[hole] = p0[b, h, tail]
                assert np.array_equal(positions[b, h, :m].cpu().numpy(), want[:m])
    assert evictions >= 2
    # every key left is the token its position says
    for b in range(B):
        n = int(lens[b])
        k, v = (bounded.cache_values(c.cpu(), None if s is None else s.cpu(), t[4].cpu(), b, n,
                                     block, False) for c, s in ((t[0], t[2]), (t[1], t[3])))
        for h in range(KVN):
            pos = positions[b, h, :n].tolist()
            assert len(set(pos)) == n and set(range(4)) <= set(pos)
            total = int(seen[b])
            assert set(range(total - recent, total)) <= set(pos)
            for kv, x in ((0, k), (1, v)):
                want = torch.stack([history[kv][b][i][h] for i in pos])
                if fp8:
                    code, scale = bounded.quantised(want)
                    want = (torch.from_numpy(code).view(torch.float8_e4m3fn).double()
                            .unflatten(-1, (-1, 64))
                            * torch.from_numpy(scale).double()[..., None]).flatten(-2)
                assert torch.equal(x[:, h], want.double())


def test_a_captured_step_replays():
    """append, attend with weights in place and evict in one CUDA graph, on a side
    stream, replayed with new inputs in the same buffers."""
    B, QN, KVN, D, block, budget = 2, 4, 2, 128, 32, 64
    cache, t = _empty_cache(B, KVN, D, 4, block, False, 0)
    t[0].normal_(), t[1].normal_()
    lens = torch.tensor([70, 65], dtype=torch.int32, device=DEV)
    out_lens = torch.zeros_like(lens)
    seen = lens + 5
    w, w2 = (torch.rand(B, KVN, cache.capacity, device=DEV) for _ in range(2))
    pos = torch.arange(cache.capacity, device=DEV).int().expand(B, KVN, -1).contiguous()
    pos2 = torch.zeros_like(pos)
    q, k, v = (torch.randn(B, 1, n, D, device=DEV).to(torch.bfloat16) for n in (QN, KVN, KVN))
    append = fia.KvAppendCall(cache, k, v, lens, weights=w, positions=pos, tokens_seen=seen)
    att = fia.KeyWeightsCall(_Problem(q, cache, t, lens, 0, None, QN, 1, D ** -0.5), weights=w,
                             weights_out=w)
    evict = fia.KvEvictCall(cache, lens, w, budget=budget, recent_tokens=8, positions=pos,
                            tokens_seen=seen, weights_out=w2, positions_out=pos2,
                            seqused_out=out_lens)

    def step():
        append.run()
        att.run()
        evict.run()

    state = [t[0], t[1], w, pos, w2, pos2, out_lens]
    start = [x.clone() for x in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        for x, y in zip(state, start):
            x.copy_(y)
        step()
        want = [x.clone() for x in state + [att.out, att.lse]]
        for x, y in zip(state, start):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(state + [att.out, att.lse], want):
            assert torch.equal(x, y)


# ----------------------------------------------------------------------------
# large offsets, many sequences, other streams, hidden NaNs
# ----------------------------------------------------------------------------

def test_pages_past_two_to_the_31_elements():
    """append and evict on pages whose elements lie past 2^31 in the pool."""
    KVN, D, block = 8, 128, 128
    nb = (1 << 31) // (block * KVN * D) + 20
    k, v = (torch.empty(nb, block, KVN, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.tensor([[nb - 1, nb - 3]], dtype=torch.int32, device=DEV)
    cache = fia.KvCache(k, v, table)
    n = 200
    new = [torch.randn(1, n, KVN, D, device=DEV).to(torch.bfloat16) for _ in range(2)]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    fia.kv_append(cache, *new, lens)
    for x, y in ((k, new[0]), (v, new[1])):
        got = torch.cat([x[nb - 1], x[nb - 3]])[:n]
        assert torch.equal(got, y[0])
    w = torch.arange(256, device=DEV).float().expand(1, KVN, 256).contiguous()
    n_out, _, pos = fia.kv_evict(cache, lens, w, budget=150)
    assert int(n_out) == 150
    for x, y in ((k, new[0]), (v, new[1])):
        got = torch.cat([x[nb - 1], x[nb - 3]])[:150]
        for h in (0, KVN - 1):
            assert torch.equal(got[:, h], y[0, pos[0, h, :150].long(), h])
    p = fi.make_fia(B=1, QN=8, KVN=KVN, D=D, q_lens=[1], kv_lens=[n], device=DEV, seed=31,
                    mask_mode=3)
    p.k_cache, p.v_cache, p.block_table, p.num_blocks = k, v, table, nb
    p.seqused_kv, p.kv_lens = torch.tensor([150], dtype=torch.int32, device=DEV), [150]
    out, lse, wt = fia.KeyWeightsCall(p).run()
    small = fi.make_fia(B=1, QN=8, KVN=KVN, D=D, q_lens=[1], kv_lens=[150], device=DEV, seed=31,
                        mask_mode=3)
    small.q = p.q
    for i, page in enumerate((nb - 1, nb - 3)):
        small.k_cache[int(small.block_table[0, i])] = k[page]
        small.v_cache[int(small.block_table[0, i])] = v[page]
    bounded.check_attention(small, out, lse, wt)


def test_weights_workspace_past_two_to_the_31_elements():
    """Scores of the last (sequence, KV head) of a batch with a wide table lie past
    2^31 elements of the workspace."""
    B, KVN, rows, G = 17, 8, 16, 8
    p = fi.make_fia(B=B, QN=KVN * G, KVN=KVN, D=128, q_lens=[rows] * B, kv_lens=[40] * (B - 1) + [150],
                    block_size=128, max_blocks=1000, device=DEV, seed=32, mask_mode=3)
    assert B * KVN * 128000 * rows * G > 1 << 31
    call = fia.KeyWeightsCall(p)
    out, lse, w = call.run()
    bounded.check_attention(p, out, lse, w)


@pytest.mark.parametrize("kv_dtype,D", [(fi.KV_BF16, 64), (fi.KV_FP8_E4M3, 128)])
def test_weights_prefill_of_many_sequences(kv_dtype, D):
    """More sequences than one window of the step list holds, some without rows or
    keys."""
    g = torch.Generator().manual_seed(33)
    B = 4300
    q = torch.randint(0, 20, (B,), generator=g)
    q[5:4100] *= (torch.rand(4095, generator=g) < 0.2).long()
    q[-1], q[7] = 200, 17
    kv = q + torch.randint(0, 30, (B,), generator=g) * (q > 0)
    kv[100:120] = 0
    p = fi.make_fia(B=B, QN=2, KVN=1, D=D, q_lens=q.tolist(), kv_lens=kv.tolist(), block_size=32,
                    layout=fi.LAYOUT_TND, kv_dtype=kv_dtype, device=DEV, seed=34, mask_mode=3)
    _check_weights(p)


def test_weights_prefill_of_long_prompts_cut_over_many_ctas():
    _check_weights(fi.make_fia(B=1, QN=4, KVN=1, D=128, q_lens=[3000], kv_lens=[4100],
                               layout=fi.LAYOUT_TND, block_size=128, device=DEV, seed=35, mask_mode=3))
    p = fi.make_fia(B=2, QN=16, KVN=2, D=64, q_lens=[1500, 130], kv_lens=[1500, 2600],
                    layout=fi.LAYOUT_TND, block_size=64, device=DEV, seed=36,
                    mask_mode=fi.MASK_BAND, pre_tokens=400, first_tokens=3)
    _check_weights(p)


@pytest.mark.parametrize("kv_dtype", [fi.KV_BF16, fi.KV_FP8_E4M3])
def test_weights_of_short_prompts_behind_long_caches(kv_dtype):
    """More than 32 units of 256 keys in a sequence, ranges that start in any of them."""
    _check_weights(fi.make_fia(B=3, QN=8, KVN=2, D=128, q_lens=[40, 300, 20],
                               kv_lens=[20001, 9000, 8449], layout=fi.LAYOUT_TND, block_size=128,
                               kv_dtype=kv_dtype, device=DEV, seed=35, mask_mode=3))


@pytest.mark.parametrize("rows", [3, 40])
def test_a_nan_row_reaches_only_the_keys_it_sees(rows):
    """A query row of NaN (and a key of NaN) leave every other key's weight alone."""
    p = fi.make_fia(B=1, QN=4, KVN=2, D=128, q_lens=[rows], kv_lens=[300], layout=fi.LAYOUT_TND,
                    device=DEV, seed=37, mask_mode=fi.MASK_BAND, pre_tokens=20, next_tokens=0)
    clean = fia.KeyWeightsCall(p).run()[2].clone()
    p.q[0] = float("nan")  # row 0 sees keys 300 - rows - 20 .. 300 - rows
    got = fia.KeyWeightsCall(p).run()[2]
    first = 300 - rows
    seen = torch.zeros(300, dtype=torch.bool, device=DEV)
    seen[first - 20:first + 1] = True
    assert torch.isnan(got[0, :, :300][:, seen]).all()
    assert torch.equal(got[0, :, :300][:, ~seen], clean[0, :, :300][:, ~seen])


def test_calls_on_another_stream_with_slow_producers():
    """Inputs written on a side stream just before the calls there."""
    B, KVN, D = 2, 2, 128
    cache, t = _empty_cache(B, KVN, D, 4, 32, False, 0)
    side = torch.cuda.Stream()
    k, v = (torch.zeros(B, 3, KVN, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    w = torch.zeros(B, KVN, cache.capacity, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        k.normal_(), v.normal_()
        lens.fill_(100)
        w.uniform_()
        fia.kv_append(cache, k, v, lens, weights=w)
        n, wo, po = fia.kv_evict(cache, lens, w, budget=64, recent_tokens=10)
    side.synchronize()
    assert n.tolist() == [64, 64]
    for b in range(B):
        for h in range(KVN):
            kept = bounded.keep_of(w[b, h].cpu().numpy(), None, 100, 64, 0, 10, 100)
            assert sorted(po[b, h, :64].tolist()) == list(np.nonzero(kept)[0])
            j = 97 + int(torch.tensor(0))  # a new row, newest: kept, moved into a hole
            slot = po[b, h, :64].tolist().index(j)
            page, row = int(t[4][b, slot // 32]), slot % 32
            assert torch.equal(t[0][page, row, h], k[b, 0, h])


def test_python_calls_refuse_tensors_that_do_not_fit():
    cache, t = _empty_cache(2, 2, 128, 2, 32, False, 0)
    lens = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    k = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(2, 2, 64, device=DEV)
    bad = [
        lambda: fia.KvAppendCall(cache, k.float(), k.float(), lens),
        lambda: fia.KvAppendCall(cache, k[:1], k[:1], lens),
        lambda: fia.KvAppendCall(cache, k, k, lens.long()),
        lambda: fia.KvAppendCall(cache, k, k, lens[:1]),
        lambda: fia.KvAppendCall(cache, k, k, lens, weights=w[:, :, :63]),
        lambda: fia.KvAppendCall(cache, k, k, lens, weights=w[:, :, :1].expand(2, 2, 64)),
        lambda: fia.KvAppendCall(cache, k, k, lens, weights=w[:1, :1].expand(2, 2, 64)),
        lambda: fia.KvAppendCall(cache, k[:, :, :, ::2], k[:, :, :, ::2], lens),
        lambda: fia.KvAppendCall(cache, k[:, :1].expand(2, 5, 2, 128), k[:, :1].expand(2, 5, 2, 128),
                                 lens),
        lambda: fia.KvAppendCall(cache, k, k, lens, status=torch.zeros(1, device=DEV)),
        lambda: fia.KvEvictCall(cache, lens, w.double(), budget=8),
        lambda: fia.KvEvictCall(cache, lens, w, budget=8, positions=w),
        lambda: fia.KvEvictCall(cache, lens, w, budget=8, weights_out=torch.zeros(2, 2, 70, device=DEV)),
        lambda: fia.KvEvictCall(cache, None, w, budget=8),
        lambda: fia.KvCache(t[0], t[1], t[4].long()),
        lambda: fia.KvCache(t[0], t[1], t[4], k_scale=w),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: fia.KvEvictCall(cache, lens, w, budget=65),
              lambda: fia.KvEvictCall(cache, lens, w, budget=8, recent_tokens=9),
              lambda: fia.KvEvictCall(cache, lens, w, budget=8, seqused_out=lens)):
        with pytest.raises(fia.FiaError):
            f()


@pytest.mark.parametrize("B,KVN", [(2, 2), (2, 1), (1, 3), (1, 1)])
@pytest.mark.parametrize("wide", ["longer", "slice", "head"])
def test_default_outputs_follow_the_row_stride_of_the_state(B, KVN, wide):
    """State tensors longer than the cache, or slices of such: the outputs that a
    call makes itself have their row stride."""
    cache, t = _empty_cache(B, KVN, 128, 2, 32, False, 0)
    whole = torch.rand(B, KVN, 80, device=DEV)
    w = whole if wide == "longer" else whole[:, :, :64] if wide == "slice" else whole[:, :, :70]
    lens = torch.tensor([50, 64][:B], dtype=torch.int32, device=DEV)
    n, wo, po = fia.kv_evict(cache, lens, w, budget=40)
    assert wo.shape == w.shape and po.shape == w.shape and n.tolist() == [40] * B
    for b in range(B):
        for h in range(KVN):
            kept = bounded.keep_of(w[b, h].cpu().numpy(), None, int(lens[b]), 40, 0, 0, int(lens[b]))
            assert sorted(po[b, h, :40].tolist()) == list(np.nonzero(kept)[0])
            assert torch.equal(wo[b, h, :40], w[b, h][po[b, h, :40].long()])
    p = fi.make_fia(B=B, QN=2 * KVN, KVN=KVN, D=128, q_lens=[1] * B, kv_lens=lens.tolist(),
                    block_size=32, device=DEV, seed=41, mask_mode=3)
    w_in = w.clone()
    out, lse, w2 = fia.KeyWeightsCall(p, weights=w).run()
    assert w2.shape == w.shape
    bounded.check_attention(p, out, lse, w2, w_in)


# ----------------------------------------------------------------------------
# few units: one kernel beside the plan
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "d64"])
@pytest.mark.parametrize("kv_layout,paged", [(0, True), (1, True), (0, False)])
def test_few_units(kind, kv_layout, paged, weights):
    """Several steps a warp, a first token's step beside the window's, rows of a
    batch that has none, tables past the entries kept in shared memory."""
    kw = dict(block_size=32, kv_layout=kv_layout) if paged else dict(paged=False, S_kv=3600)
    if paged and not weights:
        kw["max_blocks"] = 2000
    p = _window(B=3, QN=8, KVN=2, D=64 if kind == "d64" else 128, q_lens=[2, 0, 1],
                kv_lens=[3500, 70, 1111], seed=51, pre_tokens=2000, first_tokens=37,
                with_sinks=True, kv_dtype=fi.KV_FP8_E4M3 if kind == "fp8" else fi.KV_BF16, **kw)
    if weights:
        _check_weights(p)
    else:
        _check(p)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("mode,scale", [(fi.MASK_NONE, None), (fi.MASK_LEFT_UP_CAUSAL, None),
                                        (fi.MASK_RIGHT_DOWN_CAUSAL, -0.07)])
def test_few_units_masks(mode, scale, fp8):
    """Key weights of several rows in the eight columns of a unit."""
    _check_weights(fi.make_fia(B=4, QN=4, KVN=4, D=128, q_lens=[3, 8, 0, 5], kv_lens=[1, 700, 40, 2],
                               layout=fi.LAYOUT_TND, block_size=32, device=DEV, seed=54,
                               mask_mode=mode, scale=scale,
                               kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16))
    _check_weights(fi.make_fia(B=2, QN=7, KVN=1, D=128, q_lens=[1, 1], kv_lens=[300, 0],
                               block_size=96, device=DEV, seed=55, mask_mode=mode, scale=scale,
                               kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16))


def test_pages_behind_those_kept_in_shared_memory():
    """Table entries past the first 1024, in a window call of few units and an eviction."""
    _check(_window(B=1, QN=8, KVN=2, q_lens=[2], kv_lens=[20000], block_size=16, seed=56,
                   pre_tokens=500, first_tokens=20))
    _evict_case([20000, 17000], 16500, first=4, recent=300, KVN=2, D=64, block=16, seed=7)


def test_few_units_after_a_plan_and_without_one():
    """fia_plan then executes of both kinds on one workspace, and a run before them."""
    p = _window(B=2, QN=8, KVN=2, q_lens=[1, 1], kv_lens=[400, 90], seed=52, pre_tokens=100,
                first_tokens=4)
    call = fia.KeyWeightsCall(p)
    want = [x.clone() for x in call.run()]
    call.out.zero_(), call.lse.zero_(), call.weights_out.zero_()
    call.plan()
    for _ in range(2):
        call.execute()
    torch.cuda.synchronize()
    assert call.error_word() == 0
    for x, y in zip((call.out, call.lse, call.weights_out), want):
        assert torch.equal(x, y)
    call.run()
    call.out.zero_()
    fia.FiaCall.execute(call)  # the attention alone, on the run's plan
    assert torch.equal(call.out, want[0]) and call.error_word() == 0
    call.ws.zero_()
    call.out.fill_(3.0)
    fia.FiaCall.execute(call)
    assert call.error_word() == 2 and torch.all(call.out == 3.0)


def test_few_units_wait_for_their_inputs():
    """Inputs written by slow kernels before the call, outputs read after it, on a
    side stream, eager and in a graph."""
    p = _window(B=2, QN=8, KVN=2, q_lens=[1, 1], kv_lens=[400, 90], seed=53, pre_tokens=100,
                first_tokens=4)
    call = fia.KeyWeightsCall(p)
    want = [x.clone() for x in call.run()]
    keep = {n: getattr(p, n).clone() for n in ("q", "k_cache", "v_cache", "seqused_kv")}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def late():
        for n in keep:
            getattr(p, n).zero_()
        torch.cuda._sleep(5_000_000)
        for n, x in keep.items():
            getattr(p, n).copy_(x)
        call.weights_out.zero_()
        call.run()
        got = [x.clone() for x in (call.out, call.lse, call.weights_out)]
        for n in keep:  # (and nothing of the call is left behind these)
            getattr(p, n).zero_()
        return got

    with torch.cuda.stream(side):
        got = late()
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = late()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
