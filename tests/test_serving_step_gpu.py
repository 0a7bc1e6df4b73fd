"""Pages assigned on the GPU, head norms with the rotation and the append in one pass, and
whole serving steps."""
import itertools
import os
import re

import numpy as np
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
from tests import bounded, serving
from tests.test_bounded_cache_gpu import _Problem

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------------
# pages
# ----------------------------------------------------------------------------

def _pages_case(B, block, cap_pages, seed, *, q_max=3, tnd=False, spare=8, seen=False, in_place=True,
                pad=0, lens=None, q_lens=None, held=None, end=0.2):
    """One call against its definition; returns the call."""
    r = np.random.RandomState(seed)
    old = r.randint(0, cap_pages * block + 1, B)
    if lens is None:
        grown = np.minimum(old + r.randint(0, 3 * block, B), cap_pages * block)
        lens = np.where(r.rand(B) < end, r.randint(0, old + 1), grown)
    lens = np.asarray(lens)
    held = -(-old // block) if held is None else np.asarray(held)
    mine = np.clip(held, 0, cap_pages)
    nb = int(mine.sum()) + spare + 1
    perm = r.permutation(nb).astype(np.int32)
    table = np.full((B, cap_pages), 12345, np.int32)  # (unused entries hold anything)
    at = 0
    for b in range(B):
        table[b, :mine[b]] = perm[at:at + mine[b]]
        at += mine[b]
    free = np.full(nb, -77, np.int32)
    free[:spare] = perm[at:at + spare]
    cu = None
    if q_lens is None:
        q_lens = r.randint(0, q_max + 1, B) if tnd else np.full(B, q_max)
    T = int(np.sum(q_lens))
    if tnd:
        cu = pad + np.concatenate([[0], np.cumsum(q_lens)])
        T += 2 * pad
    seen_n = lens + r.randint(0, 1000, B) if seen else None
    want = serving.pages(table, held, free, spare, lens, block, cu=cu, T=T, seen=seen_n)
    d = dict(block_table=_i32(table), pages_held=_i32(held), free_pages=_i32(free),
             free_count=_i32([spare]), seqused_kv=_i32(lens))
    kw = {}
    if not in_place:
        kw = dict(pages_held_out=_i32(held * 0 - 5), free_count_out=_i32([-5]))
    status = _i32([0])
    call = fia.AssignPagesCall(**d, block_size=block, cu_seqlens_q=None if cu is None else _i32(cu),
                               seqlen_q=0 if tnd else q_max, total_q=T if tnd else None,
                               tokens_seen=None if seen_n is None else _i32(seen_n), status=status, **kw)
    for _ in range(1 if in_place else 3):
        slots, positions = call.run()
        assert np.array_equal(call.params and d["block_table"].cpu().numpy(), want[0])
        assert np.array_equal(call.pages_held_out.cpu().numpy(), want[1])
        got = d["free_pages"].cpu().numpy()
        assert np.array_equal(got[:len(want[2])], want[2])
        assert np.array_equal(got[len(want[2]):], free[len(want[2]):])
        assert int(call.free_count_out) == want[3] and int(status) == want[6]
        if T:
            assert np.array_equal(slots.cpu().numpy().reshape(-1), want[4])
            assert np.array_equal(positions.cpu().numpy().reshape(-1), want[5])
    if not in_place:
        assert np.array_equal(d["pages_held"].cpu().numpy(), held) and int(d["free_count"]) == spare
    return call, want


@pytest.mark.parametrize("B,block,cap_pages", [(1, 16, 1), (3, 32, 4), (64, 128, 32), (1023, 48, 3),
                                               (1024, 16, 2), (1025, 64, 5), (5000, 16, 4), (8192, 16, 2), (9001, 32, 3)])
@pytest.mark.parametrize("tnd,in_place", [(False, True), (True, False)])
def test_assign_pages(B, block, cap_pages, tnd, in_place):
    _pages_case(B, block, cap_pages, seed=B, tnd=tnd, in_place=in_place, q_max=2 if B > 100 else 7,
                seen=B % 2 == 0, spare=4 * B)


@pytest.mark.parametrize("B,spare", [(7, 0), (7, 3), (300, 40), (3000, 500), (40, 1)])
def test_assign_pages_short_of_pages(B, spare):
    _, want = _pages_case(B, 32, 6, seed=B + spare, spare=spare, end=0.05, tnd=True, in_place=False)
    assert want[6] == 3


def test_assign_pages_of_many_rows():
    """Prompts of many rows: a cluster, every CTA rows of others' sequences."""
    _pages_case(5, 128, 200, seed=50, tnd=True, q_lens=[20000, 0, 1, 7000, 25000],
                lens=[20000, 5, 100, 9000, 25600], held=[0, 1, 1, 16, 0], spare=600)
    _pages_case(3000, 16, 40, seed=51, tnd=True, q_max=20, spare=40000, pad=3)


def test_assign_pages_of_the_largest_batch():
    _pages_case(65536, 16, 2, seed=52, tnd=True, q_max=1, spare=200000)


def test_assign_pages_edges():
    """Lengths below 0 and past the capacity, counts outside their ranges, more rows than
    keys, rows of no sequence."""
    _pages_case(6, 16, 4, seed=53, q_max=5, lens=[-7, 64, 65, 3, 0, 1000], held=[2, -3, 9, 0, 4, 4],
                spare=30)
    _pages_case(4, 16, 4, seed=54, tnd=True, q_max=5, pad=4, lens=[2, 0, 64, 30], spare=30)
    for count in (-4, 1000):
        table, held = _i32(np.zeros((2, 3))), _i32([0, 0])
        free, n, status = _i32([4, 3, 2, 1, 0]), _i32([count]), _i32([0])
        fia.assign_pages(table, held, free, n, _i32([40, 10]), block_size=16, status=status)
        if count < 0:
            assert table.tolist() == [[-1] * 3, [-1, 0, 0]] and int(n) == 0 and int(status) == 3
        else:
            assert table.tolist() == [[0, 1, 2], [3, 0, 0]] and int(n) == 1 and int(status) == 0
    # no room for what comes back
    table, held, free = _i32([[7, 8]]), _i32([2]), _i32([1, 2])
    n, status = _i32([1]), _i32([0])
    fia.assign_pages(table, held, free, n, _i32([0]), block_size=16, status=status)
    assert free.tolist() == [1, 7] and int(n) == 2 and int(held) == 0 and int(status) == 3


def test_assign_pages_of_bad_row_counts():
    """cu_seqlens_q below 0 or past the rows: nothing is written outside."""
    lens, T = [40, 33, 70], 10
    for cu in ([-3, 2, 6, 9], [0, 4, 12, 30], [5, 5, 8, 8]):
        table, held, free, n = _i32(np.full((3, 5), -1)), _i32([0] * 3), _i32(range(20)), _i32([20])
        big = torch.full((2, T + 40), 77, dtype=torch.int32, device=DEV)
        fia.assign_pages(table, held, free, n, _i32(lens), block_size=16, cu_seqlens_q=_i32(cu),
                         slots=big[0, 20:20 + T], positions=big[1, 20:20 + T])
        assert torch.all(big[:, :20] == 77) and torch.all(big[:, 20 + T:] == 77)
        want = serving.pages(np.full((3, 5), -1), [0] * 3, list(range(20)), 20, lens, 16, cu=cu, T=T)
        assert big[0, 20:20 + T].tolist() == want[4].tolist()
        assert big[1, 20:20 + T].tolist() == want[5].tolist()


@pytest.mark.parametrize("block", [16, 144, 256, 1024])
def test_assign_pages_of_long_pages(block):
    _pages_case(9, block, 6, seed=55, tnd=True, q_lens=[0, 1, 700, 130, 128, 129, 2, 1500, 64],
                lens=[3, 5, 700, 1000, 129, 128, 1, 1600, 64], held=[1] * 9, spare=400, seen=True)


def test_assign_pages_without_rows_and_on_a_stream():
    table, held, free, n = _i32(np.zeros((2, 3))), _i32([0, 0]), _i32([4, 3, 2, 1, 0]), _i32([5])
    lens = _i32([0, 0])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        lens.copy_(_i32([40, 10]))
    got = fia.assign_pages(table, held, free, n, lens, block_size=16, stream=s)
    assert got == (None, None)
    slots, pos = fia.assign_pages(table, held, free, n, lens, block_size=16, seqlen_q=1, stream=s)
    s.synchronize()
    assert table.tolist() == [[0, 1, 2], [3, 0, 0]] and held.tolist() == [3, 1] and int(n) == 1
    assert slots.tolist() == [2 * 16 + 7, 3 * 16 + 9] and pos.tolist() == [39, 9]


# ----------------------------------------------------------------------------
# head norms and rotation
# ----------------------------------------------------------------------------

def _cache(kind, D, KVN, block, nb, kv_layout, B=None, seed=60):
    """A cache of marks: paged, or contiguous [B, block, KVN, D] where B is given."""
    g = torch.Generator().manual_seed(seed)
    row = {"bf16": D, "fp8": D, "mx": D // 2}[kind]
    n = nb if B is None else B
    shape = (n, KVN, block, row) if kv_layout else (n, block, KVN, row)
    t = [torch.randint(0, 120, shape, generator=g).to(torch.bfloat16 if kind == "bf16" else torch.uint8)
         .to(DEV) for _ in "kv"]
    scales = [None, None]
    if kind != "bf16":
        ss = (n, KVN, block, D // (64 if kind == "fp8" else 32))
        scales = [torch.randint(0, 120, ss, generator=g).to(torch.float32 if kind == "fp8" else torch.uint8)
                  .to(DEV) for _ in "kv"]
    table = None if B is not None else torch.arange(nb, dtype=torch.int32, device=DEV).reshape(1, nb)
    cache = fia.KvCache(*t, table, k_scale=scales[0], v_scale=scales[1], kv_layout=kv_layout)
    return cache, t + scales


def _near_codes(got_codes, got_scale, y, tol, kind):
    """Whether the rows [.., D] are the nearest codes of y (each known to `tol`), under the
    scale of its tile."""
    tile = 64 if kind == "fp8" else 32
    t, tt = y.unflatten(-1, (-1, tile)), tol.unflatten(-1, (-1, tile))
    amax, at = t.abs().amax(-1), tt.amax(-1)
    if kind == "fp8":
        want = torch.where(amax > 0, amax / 448, 1.0)
        assert torch.all((got_scale.double() - want).abs() <= 2 * bounded.HALF_FP32 * want + at / 448)
        scale = got_scale.double()
        v = got_codes.view(torch.float8_e4m3fn).float().double().unflatten(-1, (-1, tile)) * scale[..., None]
        step = 2.0 ** -4 * t.abs() + 2.0 ** -10 * scale[..., None]
    else:
        lo, hi = (serving.mx_quantised((t * f).flatten(-2).numpy())[1].astype(int) for f in (1 - 1e-5, 1 + 1e-5))
        s = got_scale.numpy().astype(int)
        assert np.all((s >= lo) & (s <= hi))
        scale = 2.0 ** (got_scale.double() - 127)
        v = serving.mx_values(got_codes, got_scale).unflatten(-1, (-1, tile))
        a = t.abs() / scale[..., None]
        # (half a step: 0.25 below 2, 0.5 below 4, 1 above)
        step = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0)) * scale[..., None]
    assert torch.all((v - t).abs() <= step * (1 + 2 * bounded.HALF_FP32) + 2 * tt)


def _rope_case(kind, D, QN, KVN, T, rot, pairs, *, norm="both", kv_layout=0, paged=True, strided=False,
               in_place=False, block=32, seed=61, mult=1.0):
    g = torch.Generator().manual_seed(seed)
    nb = -(-T // block) + 3
    cache, t = _cache(kind, D, KVN, block if paged else nb * block // 2 // 4 * 4, nb, kv_layout,
                      B=None if paged else 2)
    unit = t[0].shape[2 if kv_layout else 1]
    total = t[0].shape[0] * unit
    qkv = (torch.randn(T, QN + 2 * KVN, D, generator=g) * mult).to(torch.bfloat16).to(DEV)
    parts = list(qkv.split((QN, KVN, KVN), 1))
    if not strided:
        parts = [x.contiguous() for x in parts]
    q, k, v = parts
    slots = torch.randperm(total, generator=g)[:T].int()
    positions = torch.randint(0, 5000, (T,), generator=g).int()
    table = serving.cos_sin(5000, rot).to(DEV) if rot else None
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in "qk"]
    qw, kw = {"both": w, "none": (None, None), "q": (w[0], None), "k": (None, w[1])}[norm]
    want_q, size_q = serving.turned(q, qw, 1e-6, table, positions, pairs)
    want_k, size_k = serving.turned(k, kw, 1e-6, table, positions, pairs)
    before = [None if x is None else x.cpu().clone() for x in t]
    v_cpu = v.cpu().clone()
    status = _i32([0])
    out = fia.norm_rope_append(cache, q, k, v, slots.to(DEV), positions.to(DEV), table, q_weight=qw,
                               k_weight=kw, eps=1e-6, interleaved=pairs, q_out=q if in_place else None,
                               status=status)
    assert int(status) == 0
    if in_place:
        assert out.data_ptr() == q.data_ptr()
    tol = serving.turned_tolerance(size_q, D)
    off = (out.cpu().double() - want_q).abs()
    assert torch.all(off <= bounded.HALF_BF16 * want_q.abs() + 1.01 * tol + 1e-38), float((off / (tol + 1e-38)).max())
    page, row = slots.long() // unit, slots.long() % unit

    def at(x, scales):
        x = x.cpu()
        return x[page, :, row] if scales or kv_layout else x[page, row]

    tol = serving.turned_tolerance(size_k, D)
    if kind == "bf16":
        off = (at(t[0], False).double() - want_k).abs()
        assert torch.all(off <= bounded.HALF_BF16 * want_k.abs() + 1.01 * tol + 1e-38)
        assert torch.equal(at(t[1], False).view(torch.int16), v_cpu.view(torch.int16))
    else:
        _near_codes(at(t[0], False), at(t[2], True), want_k, tol, kind)
        if kind == "fp8":
            codes, scale = bounded.quantised(v_cpu)
        else:
            codes, scale = serving.mx_quantised(v_cpu)
        assert np.array_equal(at(t[1], False).numpy(), codes) and np.array_equal(at(t[3], True).numpy(), scale)
    # nothing else is written
    for n, x in enumerate(t):
        if x is not None:
            x, y = x.cpu(), before[n]
            for z in (x, y):
                if n >= 2 or kv_layout:
                    z[page, :, row] = 0
                else:
                    z[page, row] = 0
            assert torch.equal(x, y)


@pytest.mark.parametrize("rot,pairs", [(128, False), (128, True), (64, False), (32, True), (16, False),
                                       (96, False), (48, True), (0, False)])
@pytest.mark.parametrize("kind,kv_layout", [("bf16", 0), ("fp8", 1), ("mx", 0), ("mx", 1), ("bf16", 1)])
def test_norm_rope(kind, kv_layout, rot, pairs):
    _rope_case(kind, 128, 8, 2, 37, rot, pairs, kv_layout=kv_layout, strided=rot % 64 == 0)


@pytest.mark.parametrize("rot,pairs", [(64, False), (64, True), (16, True), (48, False), (0, True)])
def test_norm_rope_of_64(rot, pairs):
    _rope_case("bf16", 64, 6, 3, 29, rot, pairs, kv_layout=1)


@pytest.mark.parametrize("norm", ["none", "q", "k"])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "mx"])
def test_norm_rope_weights(kind, norm):
    _rope_case(kind, 128, 4, 4, 11, 128, False, norm=norm, paged=False)


@pytest.mark.parametrize("QN,KVN,T", [(1, 1, 1), (0, 1, 3), (3, 1, 2), (64, 8, 5), (7, 5, 100), (32, 8, 700)])
@pytest.mark.parametrize("kind", ["bf16", "mx"])
def test_norm_rope_sizes(kind, QN, KVN, T):
    _rope_case(kind, 128, QN, KVN, T, 128, False, strided=True, in_place=QN > 2, block=64)


@pytest.mark.parametrize("mult", [2.0 ** 40, 2.0 ** -40])
def test_norm_rope_ranges(mult):
    _rope_case("bf16", 128, 4, 2, 9, 64, False, mult=mult, norm="none")
    if mult > 1:
        _rope_case("fp8", 128, 4, 2, 9, 64, True, mult=mult)


def test_norm_rope_leaves_rows_out():
    """Rows of no sequence, slots and positions outside."""
    D, QN, KVN, T, P = 128, 4, 2, 6, 50
    cache, t = _cache("bf16", D, KVN, 32, 4, 0)
    before = [x.clone() for x in t[:2]]
    x = torch.randn(T, QN + 2 * KVN, D, device=DEV).to(torch.bfloat16)
    q, k, v = x.split((QN, KVN, KVN), 1)
    table = serving.cos_sin(P, D).to(DEV)
    out = torch.full((T, QN, D), 3.0, dtype=torch.bfloat16, device=DEV)
    status = _i32([0])
    #            fine, nobody, nobody, no slot, slot past the pool, position past the table
    slots, positions = _i32([5, -1, 7, -1, 128, 9]), _i32([0, -1, -3, 4, 5, 50])
    fia.norm_rope_append(cache, q, k, v, slots, positions, table, q_out=out, status=status)
    assert int(status) == 3
    assert torch.all(out[[1, 2, 5]] == 3.0) and not torch.any(torch.all(out[[0, 3, 4]] == 3.0, -1))
    want = before[1].clone()
    want[0, 5] = v[0]
    assert torch.equal(t[1], want)
    assert torch.equal(t[0].view(-1, KVN, D)[6:], before[0].view(-1, KVN, D)[6:])
    status.zero_()
    fia.norm_rope_append(cache, q[1:3], k[1:3], v[1:3], slots[1:3].clone(), positions[1:3].clone(), table,
                         q_out=out[1:3], status=status)
    assert int(status) == 0 and torch.all(out[1:3] == 3.0)
    # without a rotation there is no table to leave
    fia.norm_rope_append(cache, q[5:], k[5:], v[5:], slots[5:].clone(), _i32([1 << 30]), q_out=out[5:],
                         status=status)
    assert int(status) == 0 and torch.equal(out[5:], q[5:]) and torch.equal(t[0][0, 9], k[5])


def test_norm_rope_hard_values():
    """Zeros, infinities and NaN: a NaN stays in its head, values are kept bit by bit."""
    D, QN, KVN = 128, 2, 2
    cache, t = _cache("bf16", D, KVN, 32, 2, 0)
    x = torch.randn(3, QN + 2 * KVN, D, device=DEV).to(torch.bfloat16)
    q, k, v = (y.contiguous() for y in x.split((QN, KVN, KVN), 1))
    q[0, 0] = 0
    q[1, 1, 5], k[0, 1, 7] = float("nan"), float("inf")
    v.view(torch.int16)[2, 1, 3], v[2, 0, 9] = 0x7fa5, -float("inf")
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    out = fia.norm_rope_append(cache, q, k, v, _i32([1, 2, 3]), _i32([0, 1, 2]),
                               serving.cos_sin(3, D).to(DEV), q_weight=w, k_weight=w, eps=1e-5)
    assert torch.all(out[0, 0] == 0)
    nan = torch.isnan(out)
    assert nan[1, 1].all() and int(nan.sum()) == D
    assert torch.isnan(t[0][0, 1, 1]).any() and torch.isfinite(t[0][0, 1, 0].float()).all()
    assert torch.equal(t[1][0, 1:4].view(torch.int16), v.view(torch.int16))


def test_norm_rope_far_slots_and_positions():
    """A pool past 2^31 elements, and rotations past 2^31 table entries' bytes."""
    D, KVN, block, nb = 128, 8, 128, 20000
    k_pool = torch.zeros(nb, block, KVN, D, dtype=torch.bfloat16, device=DEV)
    cache = fia.KvCache(k_pool, torch.zeros_like(k_pool), torch.zeros(1, 1, dtype=torch.int32, device=DEV))
    table = torch.zeros(5_000_000, D, device=DEV)
    table[-1, :64], table[-1, 64:] = 0.6, 0.8
    x = torch.randn(1, 3 * KVN, D, device=DEV).to(torch.bfloat16)
    q, k, v = x.split((KVN, KVN, KVN), 1)
    slot = nb * block - 1
    out = fia.norm_rope_append(cache, q, k, v, _i32([slot]), _i32([4_999_999]), table)
    a, b = k[0].double().chunk(2, -1)
    want = torch.cat([a * 0.6 - b * 0.8, b * 0.6 + a * 0.8], -1)
    assert torch.allclose(k_pool[-1, -1].double(), want, rtol=2.0 ** -8, atol=1e-5)
    assert int((k_pool != 0).any(-1).sum()) == KVN and torch.isfinite(out).all()


def test_norm_rope_python_refusals():
    cache, t = _cache("bf16", 128, 2, 32, 2, 0)
    x = torch.randn(3, 8, 128, device=DEV).to(torch.bfloat16)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    s, table = _i32([0, 1, 2]), serving.cos_sin(9, 128).to(DEV)
    for a in ((q[:2], k, v, s, s), (q, k[..., :64], v[..., :64], s, s), (q, k, v, s[:2], s),
              (q, k, v, s.long(), s), (q, k, v, s, s.cpu()), (q.float(), k, v, s, s),
              (q.transpose(0, 1), k, v, s, s), (q, k[:, :1], v[:, :1], s, s)):
        with pytest.raises(ValueError):
            fia.norm_rope_append(cache, *a, table)
    for kw in (dict(q_out=q[:, :2]), dict(q_weight=torch.ones(128, device=DEV)),
               dict(k_weight=torch.ones(64, dtype=torch.bfloat16, device=DEV)), dict(status=s)):
        with pytest.raises(ValueError):
            fia.norm_rope_append(cache, q, k, v, s, s, table, **kw)
    with pytest.raises(ValueError):
        fia.norm_rope_append(cache, q, k, v, s, s, table.half())
    with pytest.raises(fia.FiaError):
        fia.norm_rope_append(cache, q, k, v, s, s, serving.cos_sin(9, 24).to(DEV))


# ----------------------------------------------------------------------------
# whole steps
# ----------------------------------------------------------------------------

def _serving_state(kind, B, KVN, D, block, cap_pages, nb, kv_layout):
    cache, t = _cache(kind, D, KVN, block, nb, kv_layout)
    table = torch.full((B, cap_pages), -1, dtype=torch.int32, device=DEV)
    cache = fia.KvCache(t[0], t[1], table, k_scale=t[2], v_scale=t[3], kv_layout=kv_layout)
    return cache, t + [table]


@pytest.mark.parametrize("kind,kv_layout", [("bf16", 0), ("fp8", 1), ("mx", 0), ("mx", 1)])
def test_serving_steps(kind, kv_layout):
    """Prompts, then tokens one by one, requests that end and their rows of the batch taken
    by new prompts: pages, norms with rotation and append, attention.  Every attention is
    checked in 64 bits against the cache, the cache's keys against all tokens so far."""
    B, QN, KVN, D, block, cap_pages, nb = 3, 8, 2, 128, 32, 8, 20
    cache, t = _serving_state(kind, B, KVN, D, block, cap_pages, nb, kv_layout)
    g = torch.Generator().manual_seed(70)
    cs = serving.cos_sin(cap_pages * block, D).to(DEV)
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in "qk")
    held, free, count = _i32([0] * B), _i32(torch.randperm(nb, generator=g)), _i32([nb])
    status = _i32([0])
    lens = [0] * B
    keys = [[] for _ in range(B)]  # every token's K before the rotation, and its V
    todo = [[90, 7, 33]] + [[1, 1, 1]] * 40 + [[1, -1, 1], [1, 50, 1]] + [[1, 1, 1]] * 20
    for step, rows in enumerate(todo):
        for b in range(B):
            if rows[b] < 0:
                lens[b], keys[b] = 0, []
        n = [max(r, 0) for r in rows]
        lens = [a + r for a, r in zip(lens, n)]
        T, S = sum(n), max(n)
        x = torch.randn(T, QN + 2 * KVN, D, generator=g).to(torch.bfloat16)
        cu = np.concatenate([[0], np.cumsum(n)])
        for b in range(B):
            keys[b] += [x[i, QN:] for i in range(cu[b], cu[b + 1])]
        q, k, v = x.to(DEV).split((QN, KVN, KVN), 1)
        lens_t, cu_t = _i32(lens), _i32(cu)
        slots, positions = fia.assign_pages(t[4], held, free, count, lens_t, block_size=block,
                                            cu_seqlens_q=cu_t, total_q=T, status=status)
        out_q = fia.norm_rope_append(cache, q, k, v, slots, positions, cs, q_weight=qw, k_weight=kw,
                                     status=status)
        p = _Problem(out_q, cache, t, lens_t, 1, cu_t, QN, S, D ** -0.5, kv_layout)
        p.q_lens, p.kv_lens = n, lens
        out, lse = fia.fused_infer_attention(p)
        if S > 1 or step % 13 == 0 or step == len(todo) - 1:
            assert int(status) == 0
            if kind == "mx":
                serving.check_mx(p, out, lse)
            else:
                bounded.check_attention(p, out, lse)
    assert int(count) == nb - sum(-(-a // block) for a in lens)
    # the cache holds every token's K, normed and rotated, and V
    c = serving.decoded(p) if kind == "mx" else p.to("cpu")
    for b in range(B):
        x = torch.stack(keys[b])
        want, size = serving.turned(x[:, :KVN], kw, 1e-6, cs, torch.arange(lens[b]), False)
        got = bounded.cache_values(c.k_cache, c.k_scale, c.block_table, b, lens[b], block, kv_layout == 1)
        step = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -3, "mx": 0.5}[kind]
        amax = want.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
        assert torch.all((got - want).abs() <= step * want.abs() + (0.1 * amax if kind == "mx" else 1e-2))


def test_a_captured_serving_step_replays():
    """Pages, norms, append and attention in one CUDA graph, replayed for 70 tokens of every
    sequence: pages are taken on the way; the same as the calls one by one."""
    B, QN, KVN, D, block, cap_pages, nb = 2, 4, 2, 128, 32, 4, 9
    outs = []
    for captured in (False, True):
        cache, t = _serving_state("mx", B, KVN, D, block, cap_pages, nb, 0)
        g = torch.Generator().manual_seed(71)
        held, free, count, lens = _i32([0] * B), _i32(range(nb)), _i32([nb]), _i32([0] * B)
        x = torch.zeros(B, QN + 2 * KVN, D, dtype=torch.bfloat16, device=DEV)
        q, k, v = x.split((QN, KVN, KVN), 1)
        pages = fia.AssignPagesCall(t[4], held, free, count, lens, block_size=block, seqlen_q=1)
        rope = fia.NormRopeAppendCall(cache, q, k, v, pages.slots, pages.positions,
                                      serving.cos_sin(128, D).to(DEV))
        att = fia.FiaCall(_Problem(rope.q_out.view(B, 1, QN, D), cache, t, lens, 0, None, QN, 1, D ** -0.5))

        def step():
            lens.add_(1)
            pages.run()
            rope.run()
            att.run()

        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            if captured:
                x.normal_()
                step()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    step()
                torch.cuda.synchronize()
                for a, b in ((held, 0), (lens, 0), (count, nb)):
                    a.fill_(b)
                free.copy_(_i32(range(nb)))
            seen = []
            for _ in range(70):
                x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
                graph.replay() if captured else step()
                seen.append(att.out.clone())
        s.synchronize()
        outs.append((torch.stack(seen), t[4].clone(), count.clone()))
        assert att.error_word() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert int(outs[0][2]) == nb - 6


def test_the_readme_step():
    """The README's step as it stands, against the calls' definitions."""
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    code = re.search(r"A serving step over a.*?```python\n(.*?)```", text, re.S).group(1)
    B, QN, KVN, D, page, cap_pages = 2, 4, 2, 128, 32, 2
    _, t = _serving_state("mx", B, KVN, D, page, cap_pages, 5, 0)
    g = torch.Generator().manual_seed(72)
    names = dict(fia=fia, k_codes=t[0], v_codes=t[1], k_scales=t[2], v_scales=t[3], block_table=t[4],
                 lens=_i32([0] * B), held=_i32([0] * B), free_pages=_i32(range(5)), free_count=_i32([5]),
                 page=page, cos_sin=serving.cos_sin(page * cap_pages, D).to(DEV),
                 q_norm=torch.ones(D, dtype=torch.bfloat16, device=DEV), k_norm=None)
    for n in range(1, 36):
        x = torch.randn(B, 1, QN + 2 * KVN, D, generator=g).to(torch.bfloat16)
        names["q_new"], names["k_new"], names["v_new"] = x.to(DEV).split((QN, KVN, KVN), 2)
        exec(code, names)
        assert names["lens"].tolist() == [n] * B and names["q"].shape == (B, 1, QN, D)
        want, size = serving.turned(x[:, 0, :QN], names["q_norm"], 1e-6, names["cos_sin"],
                                 torch.full((B,), n - 1), False)
        got = names["q"].cpu().double()[:, 0]
        assert torch.all((got - want).abs() <= 2.0 ** -8 * want.abs() + 1.01 * serving.turned_tolerance(size, D))
        v = x[:, 0, QN + KVN:]
        codes, scales = serving.mx_quantised(v)
        at = names["slots"].long().cpu()
        assert torch.equal(t[1].view(-1, KVN, D // 2).cpu()[at], torch.from_numpy(codes))
        assert torch.equal(t[3].permute(0, 2, 1, 3).reshape(-1, KVN, D // 32).cpu()[at], torch.from_numpy(scales))
    assert int(names["free_count"]) == 1
