"""A cache in MXFP4 on the GPU: append, attention (decode, prompts, windows, key
weights), eviction."""
import copy

import numpy as np
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import bounded, serving

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

# CTAs too few for a cluster: a call of few units takes the kernel of larger ones
NO_CLUSTER = 7


def _run(p, weights=False, num_sms=0, w_in=None):
    d = p.to(DEV)
    if weights:
        w = None if w_in is None else w_in.to(DEV)
        call = fia.KeyWeightsCall(d, weights=w, num_sms=num_sms)
    else:
        call = fia.FiaCall(d, num_sms=num_sms)
    got = call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 0
    return got


def _check(p, weights=False, num_sms=0):
    w_in = None
    if weights:
        cap = p.S_kv if p.block_table is None else p.block_table.shape[1] * p.block_size
        w_in = torch.rand(p.B, p.KVN, cap, generator=torch.Generator().manual_seed(8))
    # (both decode kernels)
    for n in (num_sms, NO_CLUSTER) if max(p.q_lens) <= 16 and num_sms == 0 else (num_sms,):
        got = _run(p, weights, n, w_in)
        serving.check_mx(p, got[0], got[1], got[2] if weights else None, w_in)


# ----------------------------------------------------------------------------
# append
# ----------------------------------------------------------------------------

def _empty(B, KVN, pages, block, kv_layout, paged=True, seed=0):
    """A cache filled with marks, and its tensors [k, v, k_scale, v_scale, table]."""
    g = torch.Generator().manual_seed(seed)
    nb = B * pages + 3
    shape = ((nb, KVN, block, 64) if kv_layout else (nb, block, KVN, 64)) if paged \
        else (B, pages * block, KVN, 64)
    ss = (nb, KVN, block, 4) if paged else (B, KVN, pages * block, 4)
    t = [torch.randint(0, 256, s, generator=g).to(torch.uint8).to(DEV) for s in (shape, shape, ss, ss)]
    t.append(torch.randperm(nb, generator=g)[:B * pages].reshape(B, pages).int().to(DEV)
             if paged else None)
    return fia.KvCache(t[0], t[1], t[4], k_scale=t[2], v_scale=t[3], kv_layout=kv_layout), t


def _place(t, name, b, h, j, block, kv_layout):
    if t[4] is None:
        return (b, h, j) if name >= 2 else (b, j, h)
    page, row = int(t[4][b, j // block]), j % block
    return (page, h, row) if name >= 2 or kv_layout else (page, row, h)


def _hard_rows(T, KVN, g):
    """Values of every size, ties, zeros, NaN and infinities among them."""
    x = torch.randn(T, KVN, 128, generator=g).to(torch.bfloat16)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) \
        * torch.where(torch.arange(32) % 3 == 0, -1.0, 1.0)
    x[0, 0, :32] = ties.to(torch.bfloat16)                    # ties under a scale of 1
    x[0, 0, 32:64] = (ties * 2.0 ** 60).to(torch.bfloat16)
    x[0, 0, 64:96] = (ties * 2.0 ** -126).to(torch.bfloat16)  # below the normal range
    x[0, 0, 96:] = 0.0
    if T > 1:
        x[1, 0, 3], x[1, 0, 40], x[1, 0, 70] = float("nan"), float("inf"), -float("inf")
        x[1, 0, 100] = torch.finfo(torch.bfloat16).max
        x[1, 1, :32] = 9.2e-41
        x[1, 1, 32:64] = -0.0
        x[1, 1, 64] = 6.03125                                 # just past the border of a scale
    return x


@pytest.mark.parametrize("kv_layout", [0, 1, None])
@pytest.mark.parametrize("q,kv,bsnd", [([1, 1, 1], [1, 33, 96], True), ([4, 4], [4, 70], True),
                                       ([5, 0, 37, 1], [5, 0, 90, 64], False), ([2], [2], False),
                                       ([96, 3], [96, 96], False)])
def test_append_writes_its_rows_and_nothing_else(q, kv, bsnd, kv_layout):
    B, KVN, block, pages = len(q), 3, 32, 3
    cache, t = _empty(B, KVN, pages, block, kv_layout or 0, kv_layout is not None, seed=1)
    g = torch.Generator().manual_seed(2)
    new = [_hard_rows(sum(q), KVN, g), _hard_rows(sum(q), KVN, g).flip(1)]
    want = [None if a is None else a.cpu().clone() for a in t]
    rows = [serving.mx_quantised(x) for x in new]
    i = 0
    for b in range(B):
        for r in range(q[b]):
            for h in range(KVN):
                for n in range(2):
                    at = b, h, kv[b] - q[b] + r, block, kv_layout
                    want[n][_place(t, n, *at)] = torch.from_numpy(rows[n][0][i, h])
                    want[2 + n][_place(t, 2 + n, *at)] = torch.from_numpy(rows[n][1][i, h])
            i += 1
    dev, cu = [x.to(DEV) for x in new], None
    if bsnd:
        dev = [x.unflatten(0, (B, -1)) for x in dev]
    else:
        cu = torch.tensor([0] + list(np.cumsum(q)), dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    fia.kv_append(cache, *dev, torch.tensor(kv, dtype=torch.int32, device=DEV), cu_seqlens_q=cu,
                  status=status)
    for a, w in zip(t, want):
        assert a is None or torch.equal(a.cpu(), w)
    assert int(status) == 0


# ----------------------------------------------------------------------------
# decode
# ----------------------------------------------------------------------------

LENS = {
    "short": dict(q_lens=[1, 1, 1, 1], kv_lens=[1, 129, 700, 17]),
    "one": dict(q_lens=[1], kv_lens=[1]),
    "empty": dict(q_lens=[1, 1, 1], kv_lens=[0, 40, 0]),
    "long": dict(q_lens=[1, 1], kv_lens=[30000, 5001]),
    "rows": dict(q_lens=[4, 1, 0, 3], kv_lens=[500, 1, 60, 2], layout=fi.LAYOUT_TND),
    "sixteen": dict(q_lens=[16, 16], kv_lens=[1000, 9]),
}


@pytest.mark.parametrize("mask", [0, 2, 3, 4])
@pytest.mark.parametrize("name", sorted(LENS))
def test_decode(name, mask):
    kw = dict(pre_tokens=300, next_tokens=2) if mask == 4 else {}
    p = serving.make_mx(B=len(LENS[name]["q_lens"]), QN=8, KVN=2, block_size=64, seed=3,
                        mask_mode=mask, with_sinks=mask == 3, **kw, **LENS[name])
    _check(p)


@pytest.mark.parametrize("QN,KVN,rows", [(1, 1, 1), (3, 1, 1), (7, 7, 2), (12, 2, 1), (16, 1, 1),
                                         (64, 2, 1), (64, 1, 1), (10, 2, 5), (32, 8, 1), (64, 1, 3)])
def test_decode_heads(QN, KVN, rows):
    _check(serving.make_mx(B=2, QN=QN, KVN=KVN, q_lens=[rows] * 2, kv_lens=[333, 1500],
                           block_size=128, seed=4, mask_mode=3))


@pytest.mark.parametrize("num_sms", [0, 1, 5])
@pytest.mark.parametrize("block,kv_layout,paged", [(32, 0, True), (96, 1, True), (160, 0, True),
                                                   (512, 1, True), (0, 0, False)])
def test_decode_caches(block, kv_layout, paged, num_sms):
    kw = dict(block_size=block, kv_layout=kv_layout) if paged else dict(paged=False, S_kv=1204)
    _check(serving.make_mx(B=3, QN=8, KVN=4, q_lens=[1] * 3, kv_lens=[1203, 64, 500], seed=5, **kw),
           num_sms=num_sms)


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("shared", [False, True])
def test_decode_explicit_mask(rows, shared):
    _check(serving.make_mx(B=2, QN=4, KVN=2, q_lens=[rows] * 2, kv_lens=[400, 130], block_size=64,
                           seed=6, mask_mode=1, mask_density=0.4, mask_shared=shared,
                           mask_full_rows=1))


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("rows,lens", [(1, [1500, 300, 2]), (4, [900, 2000, 64]), (1, [9000])])
def test_decode_window(rows, lens, weights):
    _check(serving.make_mx(B=len(lens), QN=8, KVN=2, q_lens=[rows] * len(lens), kv_lens=lens,
                           block_size=64, seed=7, mask_mode=4, pre_tokens=250, first_tokens=5,
                           with_sinks=True), weights)


@pytest.mark.parametrize("QN,rows", [(8, 1), (4, 3), (32, 1)])
def test_decode_weights(QN, rows):
    _check(serving.make_mx(B=3, QN=QN, KVN=2, q_lens=[rows] * 3, kv_lens=[1, 700, 129], seed=8,
                           block_size=32, mask_mode=3), weights=True)


@pytest.mark.parametrize("QN,rows", [(12, 2), (4, 9), (24, 1), (4, 16)])
def test_decode_of_sixteen_columns(QN, rows):
    """Units of more than 8 columns, the last one in part: explicit masks with rows that see
    nothing, key weights, a top-left mask."""
    kw = dict(B=2, QN=QN, KVN=2, q_lens=[rows] * 2, kv_lens=[401, 130], block_size=64, seed=10)
    _check(serving.make_mx(mask_mode=1, mask_density=0.4, mask_full_rows=1, **kw))
    _check(serving.make_mx(mask_mode=2, **kw))
    _check(serving.make_mx(mask_mode=3, **kw), weights=True)


def test_decode_of_a_large_batch():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 300, (200,), generator=g).tolist()
    _check(serving.make_mx(B=200, QN=4, KVN=1, q_lens=[1] * 200, kv_lens=lens, block_size=32, seed=9))


@pytest.mark.parametrize("mult", [2.0 ** 17, 2.0 ** -20])
def test_decode_query_ranges(mult):
    p = serving.make_mx(B=2, QN=4, KVN=2, q_lens=[1] * 2, kv_lens=[200, 77], block_size=32, seed=10,
                        q_mult=mult, scale=2.0 ** -19 if mult > 1 else 1.0)
    _check(p)


@pytest.mark.parametrize("rows,num_sms", [(1, 0), (1, NO_CLUSTER), (40, 0)])
def test_far_scales(rows, num_sms):
    """Scales of V from 2^-20 to 2^20, and of K within what scores stand: the power of
    two that O is kept over moves from tile to tile."""
    p = serving.make_mx(B=2, QN=4, KVN=2, q_lens=[rows] * 2, kv_lens=[3000, 1111], block_size=64,
                        seed=11, mask_mode=3, poison=False)
    g = torch.Generator().manual_seed(12)
    p.v_scale = torch.randint(107, 148, p.v_scale.shape, generator=g).to(torch.uint8)
    p.k_scale = torch.randint(120, 129, p.k_scale.shape, generator=g).to(torch.uint8)
    ref = bounded.attention(serving.decoded(p))
    out = _run(p, num_sms=num_sms)[0].cpu().double()
    for b, (o, l, w, mag, A) in enumerate(ref):
        # P (32 at the least where it is largest) times its scale over the largest, 2^20, is
        # rounded to half a step of fp16, at most 2^-25, and a scale below 2^-24 of the
        # largest counts as 0 (P up to 2^13 over 32: 2^-17 at most, but where P is that large
        # it is the sum too), times codes of up to 6; a prompt's P, in bf16, by half a step
        tl = bounded.lse_tolerance(serving.decoded(p), A, p.kv_lens[b])
        half = bounded.HALF_FP16 if rows <= 16 else bounded.HALF_BF16
        to = 1.01 * (half * mag + bounded.HALF_BF16 * o.abs()) + 2 * tl * mag
        if rows <= 16:
            to = to + 2.0 ** 20 * 6 * (2.0 ** -30 * p.kv_lens[b] + 2.0 ** -25)
        assert torch.all((out[b] - o).abs() <= to)


@pytest.mark.parametrize("num_sms", [0, NO_CLUSTER])
def test_a_nan_scale_reaches_the_rows_that_see_it(num_sms):
    p = serving.make_mx(B=2, QN=4, KVN=2, q_lens=[1, 1], kv_lens=[300, 200], block_size=32, seed=13,
                        mask_mode=3, poison=False)
    clean = _run(p, num_sms=num_sms)
    page, row = int(p.block_table[0, 100 // 32]), 100 % 32
    v = copy.copy(p)
    v.v_scale = p.v_scale.clone()
    v.v_scale[page, 1, row, 2] = 255  # sequence 0, KV head 1 (heads 2, 3), elements 64..95
    got = _run(v, num_sms=num_sms)
    bad = torch.zeros_like(got[0], dtype=torch.bool)
    bad[0, :, 2:, 64:96] = True
    assert torch.equal(torch.isnan(got[0]), bad) and torch.equal(got[0][~bad], clean[0][~bad])
    assert torch.equal(got[1], clean[1])
    k = copy.copy(p)
    k.k_scale = p.k_scale.clone()
    k.k_scale[page, 1, row, 2] = 255
    got = _run(k, num_sms=num_sms)
    bad[0, :, 2:] = True
    assert torch.equal(torch.isnan(got[0]), bad) and torch.equal(got[0][~bad], clean[0][~bad])
    k.seqused_kv = torch.tensor([100, 200], dtype=torch.int32)  # behind the last key: anything
    assert torch.isfinite(_run(k, num_sms=num_sms)[0]).all()


# ----------------------------------------------------------------------------
# prompts
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("mask", [0, 2, 3, 4])
@pytest.mark.parametrize("q,kv,layout", [([17], [17], 0), ([200, 40, 77], [300, 40, 500], 1),
                                         ([130, 130], [60, 400], 0), ([300, 0, 20], [300, 7, 1], 1)])
def test_prompts(q, kv, layout, mask, weights):
    kw = dict(pre_tokens=90, first_tokens=5) if mask == 4 else {}
    _check(serving.make_mx(B=len(q), QN=4, KVN=2, q_lens=q, kv_lens=kv, layout=layout, block_size=64,
                           seed=14, mask_mode=mask, with_sinks=mask != 2, **kw), weights)


@pytest.mark.parametrize("block,kv_layout,paged", [(32, 1, True), (96, 0, True), (0, 0, False)])
def test_prompt_caches(block, kv_layout, paged):
    kw = dict(block_size=block, kv_layout=kv_layout) if paged else dict(paged=False, S_kv=404)
    _check(serving.make_mx(B=2, QN=6, KVN=2, q_lens=[150, 33], kv_lens=[403, 33], seed=15, mask_mode=3,
                           layout=fi.LAYOUT_TND, **kw))


def test_prompt_explicit_mask():
    _check(serving.make_mx(B=2, QN=4, KVN=2, q_lens=[70, 70], kv_lens=[200, 70], block_size=32, seed=16,
                           mask_mode=1, mask_density=0.3, mask_full_rows=2))


# ----------------------------------------------------------------------------
# edges
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("num_sms", [0, NO_CLUSTER])
@pytest.mark.parametrize("page", [1 << 26, -(1 << 26), -1, 5000])
@pytest.mark.parametrize("kind", ["decode", "window", "weights", "prompt", "weights_prompt"])
def test_pages_outside_the_pool_read_as_zeros(kind, page, num_sms):
    prompt = kind.endswith("prompt")
    kw = dict(mask_mode=4, pre_tokens=150, first_tokens=4) if kind == "window" else dict(mask_mode=3)
    p = serving.make_mx(B=3, QN=8, KVN=2, q_lens=[200, 40, 77] if prompt else [1, 2, 1],
                        kv_lens=[300, 40, 500], layout=fi.LAYOUT_TND, block_size=64, seed=31,
                        kv_layout=1, **kw)
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        x = getattr(p, name)
        setattr(p, name, torch.cat([x, torch.zeros_like(x[:1])]))
    p.num_blocks += 1
    got = []
    for entry in (p.num_blocks - 1, page):
        p.block_table[0, 4], p.block_table[2, 0], p.block_table[2, 6] = entry, entry, entry
        d = p.to(DEV)
        call = (fia.KeyWeightsCall if "weights" in kind else fia.FiaCall)(d, num_sms=num_sms)
        call.ws.fill_(0x7f)
        got.append([x.clone() for x in call.run()])
        torch.cuda.synchronize()
        assert call.error_word() == 0
    for a, b in zip(*got):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


@pytest.mark.parametrize("rows,num_sms", [(1, 0), (1, NO_CLUSTER), (3, NO_CLUSTER), (40, 0)])
@pytest.mark.parametrize("bad", ["rows", "keys", "negative_keys"])
def test_lengths_outside_the_tensors(rows, num_sms, bad):
    p = serving.make_mx(B=3, QN=4, KVN=2, q_lens=[rows] * 3, kv_lens=[100, 70, 60], block_size=32,
                        layout=fi.LAYOUT_TND, seed=33, mask_mode=3)
    d = p.to(DEV)
    T = 3 * rows
    out = torch.full((T + 8, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    call = fia.FiaCall(d, out=out[:T], num_sms=num_sms)
    if bad == "rows":
        d.cu_seqlens_q[2:] += 3
        hit, fine = slice(2 * rows, T), [0]
    else:
        d.seqused_kv[1] = 129 if bad == "keys" else -4
        hit, fine = slice(rows, 2 * rows), [0, 2]
    call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 2 and torch.all(out[T:] == 3.0)
    if bad != "rows":
        assert torch.all(out[hit] == 3.0)
    want = bounded.attention(serving.decoded(p))
    for b in fine:
        o, _, _, mag, _ = want[b]
        got = out[b * rows:(b + 1) * rows].cpu().double()
        assert torch.all((got - o).abs() <= 1.1 * bounded.HALF_BF16 * (mag + o.abs()) + 1e-3 * mag)


def test_rows_behind_the_last_sequence_are_left():
    for rows in (2, 40):
        p = serving.make_mx(B=2, QN=4, KVN=2, q_lens=[rows] * 2, kv_lens=[100, 70], block_size=32,
                            layout=fi.LAYOUT_TND, seed=34, mask_mode=3).to(DEV)
        p.q = torch.cat([p.q, p.q])
        p.T = 4 * rows
        out = torch.full_like(p.q, 3.0)
        lse = torch.full((p.T, 4, 1), 3.0, device=DEV)
        fia.FiaCall(p, out=out, lse=lse).run()
        assert torch.all(out[2 * rows:] == 3.0) and torch.all(lse[2 * rows:] == 3.0)
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("B", [3, 40])
def test_without_a_workspace_and_captured(B):
    """The workspace-free entry, a plan used twice, and a replayed graph give the same bits."""
    p = serving.make_mx(B=B, QN=8, KVN=2, q_lens=[1] * B, kv_lens=[3000, 200, 77] + [500] * (B - 3),
                        block_size=64, seed=35, mask_mode=3).to(DEV)
    want = [x.clone() for x in fia.FiaCall(p).run()]
    call = fia.FiaCall(p)
    call.plan()
    for _ in range(2):
        call.out.zero_()
        call.execute()
        assert torch.equal(call.out, want[0])
    free = fia.FiaCall(p)
    status = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    fia.fia_decode_run_noalloc(free.params, status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert torch.equal(free.out, want[0]) and torch.equal(free.lse, want[1]) and int(status) == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call.run()
        call.out.zero_()
        graph.replay()
    s.synchronize()
    assert torch.equal(call.out, want[0])


def test_pools_past_two_to_the_31_bytes():
    """Pages far behind 2^31 bytes of codes (and 2^32 elements)."""
    nb, block, KVN = 70000, 128, 8  # 4.6 GB of codes for K, and for V
    p = serving.make_mx(B=1, QN=8, KVN=KVN, q_lens=[1], kv_lens=[250], block_size=block, seed=36)
    d = p.to(DEV)
    for name in "kv":
        for part, shape in (("_cache", (nb, block, KVN, 64)), ("_scale", (nb, KVN, block, 4))):
            big = torch.zeros(shape, dtype=torch.uint8, device=DEV)
            small = getattr(d, name + part)
            big[nb - 2:] = small[p.block_table[0, :2].long().to(DEV)]
            setattr(d, name + part, big)
    d.block_table = torch.tensor([[nb - 2, nb - 1]], dtype=torch.int32, device=DEV)
    d.num_blocks = nb
    out, lse = fia.FiaCall(d).run()
    serving.check_mx(p, out, lse)
    cache = fia.KvCache(d.k_cache, d.v_cache, d.block_table, k_scale=d.k_scale, v_scale=d.v_scale)
    new = torch.randn(1, 1, KVN, 128, device=DEV).to(torch.bfloat16)
    fia.kv_append(cache, new, new, torch.tensor([251], dtype=torch.int32, device=DEV))
    codes, scale = serving.mx_quantised(new.cpu()[0, 0])
    assert torch.equal(d.k_cache[nb - 1, 122].cpu(), torch.from_numpy(codes))
    assert torch.equal(d.v_scale[nb - 1, :, 122].cpu(), torch.from_numpy(scale))


@pytest.mark.parametrize("B,kv,window,rows", [(40, 3000, None, 1), (7, 20000, None, 3), (1, 100, None, 1),
                                              (40, 9000, 4096, 1), (60, 5000, 1024, 1), (24, 2500, 2048, 1)])
def test_the_plan(B, kv, window, rows):
    """The chunk sizes and counts that fia.h states."""
    kw = dict(mask_mode=4, pre_tokens=window - 1, next_tokens=0, first_tokens=4) if window else dict(mask_mode=3)
    p = serving.make_mx(B=B, QN=8, KVN=2, q_lens=[rows] * B, kv_lens=[kv] * B, block_size=128, seed=60, **kw).to(DEV)
    call = fia.FiaCall(p, num_sms=50)
    call.plan()
    torch.cuda.synchronize()
    lay = fia.fia_get_plan_layout(call.params)
    C, c2, N = call.ws[lay.sched_off:lay.sched_off + 24].view(torch.int64).tolist()
    n, U = 150, 2 * B * (2 if rows * 4 > 16 else 1)
    cost = -(-kv // 128)
    if window and kv > window + 4:
        t0 = (kv - window) // 128
        cost = cost - t0 + min(t0, 1)
    T = U * cost
    want = max(1, -(-T // (2 * n)))
    want = want, max(-(-want // 2), min(want, 6))
    if window and 8 * U >= n:
        def time(s):
            z = -(-cost // s)
            f, r = divmod(-(-T * -(-cost // z) // cost), n)
            return (7 * f + (0 if r == 0 else 5 + (3 * r > n) + (3 * r > 2 * n))) * (z + 1) + 12 * (s > 1), s
        s = min(time(s) for s in range(1, min(16, cost) + 1) if s == 1 or U * s <= 2 * n + 4 * U)[1]
        want = (-(-cost // s),) * 2
    assert (C, c2) == want
    n1 = max(0, cost // C - 1)
    assert N == U * (n1 + -(-(cost - n1 * C) // c2))


def test_calls_side_by_side():
    """Two calls on two streams, each with its workspace, many times: the same bits as alone."""
    ps = [serving.make_mx(B=12, QN=16, KVN=2, q_lens=[2] * 12, kv_lens=[900 + 70 * i for i in range(12)],
                          block_size=32, seed=s, mask_mode=3).to(DEV) for s in (50, 51)]
    want = [[x.clone() for x in fia.FiaCall(p).run()] for p in ps]
    calls, streams = [fia.FiaCall(p) for p in ps], [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(50):
        for c, s in zip(calls, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c.out, w[0]) and torch.equal(c.lse, w[1]) and c.error_word() == 0


def test_the_queue_of_a_plan_of_other_lengths():
    """A plan made for longer sequences: entries past the cache run as empty, nothing outside
    is read or written."""
    p = serving.make_mx(B=20, QN=8, KVN=2, q_lens=[1] * 20, kv_lens=[700 + i for i in range(20)],
                        block_size=32, seed=52, mask_mode=3).to(DEV)
    call = fia.FiaCall(p)
    call.plan()
    short = copy.copy(p)
    short.block_table = p.block_table[:, :5].contiguous()
    other = fia.FiaCall(short, out=torch.full_like(call.out, 3.0))
    n = min(call.ws.numel(), other.ws.numel())
    other.ws[:n].copy_(call.ws[:n])
    other.execute()
    torch.cuda.synchronize()
    assert other.error_word() == 2


def test_python_calls_refuse_tensors_that_do_not_fit():
    p = serving.make_mx(B=2, QN=4, KVN=2, q_lens=[1, 1], kv_lens=[100, 70], block_size=32, seed=37).to(DEV)
    for name, x in (("k_cache", p.k_cache[..., :32].contiguous()), ("v_cache", p.v_cache.to(torch.int8)),
                    ("k_scale", p.k_scale.float()), ("v_scale", p.v_scale[..., :2].contiguous()),
                    ("k_scale", None), ("v_scale", p.v_scale[:, :, ::2])):
        bad = copy.copy(p)
        setattr(bad, name, x)
        with pytest.raises((ValueError, fia.FiaError)):
            fia.FiaCall(bad)
    with pytest.raises(ValueError):
        fia.KvCache(p.k_cache, p.v_cache, p.block_table, k_scale=p.k_scale, v_scale=p.v_scale.float())


# ----------------------------------------------------------------------------
# eviction
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("kv_layout,paged", [(0, True), (1, True), (0, False)])
@pytest.mark.parametrize("lens,budget", [([200, 61, 60, 1, 0, 97], 60), ([700, 300], 33)])
def test_evict_moves_codes_and_scales(lens, budget, kv_layout, paged):
    B, KVN, block = len(lens), 2, 32
    pages = -(-max(lens) // block)
    cache, t = _empty(B, KVN, pages, block, kv_layout, paged, seed=40)
    g = torch.Generator().manual_seed(41)
    w = torch.rand(B, KVN, cache.capacity, generator=g)
    before = [None if a is None else a.cpu().clone() for a in t]
    n, wo, po = fia.kv_evict(cache, torch.tensor(lens, dtype=torch.int32, device=DEV), w.to(DEV),
                             budget=budget, first_tokens=4, recent_tokens=20)
    want = [None if a is None else a.clone() for a in before]
    for b, h, m, hole, tail in bounded.evicted(w.numpy(), None, lens, budget, 4, 20, None):
        assert int(n[b]) == m
        for x, y in zip(hole, tail):
            assert int(po[b, h, x]) == y
            for name in range(4):
                want[name][_place(t, name, b, h, int(x), block, kv_layout)] = \
                    before[name][_place(t, name, b, h, int(y), block, kv_layout)]
    for a, x in zip(t, want):
        assert a is None or torch.equal(a.cpu(), x)
