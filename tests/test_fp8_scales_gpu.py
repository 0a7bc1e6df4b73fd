"""V scales of an FP8 cache far apart, in decode: hidden keys take no part however large their V
is; calls of few units hold every spread among the keys that count."""
import numpy as np
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import bounded
from tests.test_mx_cache_gpu import NO_CLUSTER

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KERNELS = [0, NO_CLUSTER]
# a window over everything: what few units with first tokens go by
FEW = dict(mask_mode=4, pre_tokens=1 << 20, first_tokens=4)


def _problem(**kw):
    return fi.make_fia(D=128, kv_dtype=fi.KV_FP8_E4M3, poison=False, block_size=64, **kw)


def _run(p, weights=False, num_sms=0):
    call = (fia.KeyWeightsCall if weights else fia.FiaCall)(p.to(DEV), num_sms=num_sms)
    got = call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 0
    return got


def _check(p, weights=False, num_sms=0):
    got = _run(p, weights, num_sms)
    bounded.check_attention(p, got[0], got[1], got[2] if weights else None)


def _at(p, j, b=0):
    return int(p.block_table[b, j // p.block_size]), j % p.block_size


@pytest.mark.parametrize("power", [14, 40, 90])
@pytest.mark.parametrize("num_sms", KERNELS)
@pytest.mark.parametrize("kind", ["explicit", "explicit_rows", "left_up", "columns", "band", "window"])
def test_hidden_keys_take_no_part(kind, num_sms, power):
    """Keys that a mask hides from every row hold any finite codes under a large scale."""
    rows = {"explicit": 1, "explicit_rows": 3, "left_up": 3, "columns": 1, "band": 1, "window": 4}[kind]
    kw = {"explicit": dict(mask_mode=1, mask_density=0.5), "explicit_rows": dict(mask_mode=1, mask_density=0.5),
          "left_up": dict(mask_mode=2), "columns": dict(mask_mode=1, mask_density=0.5),
          "band": dict(mask_mode=4, pre_tokens=40),
          "window": dict(mask_mode=4, pre_tokens=40, first_tokens=3)}[kind]
    p = _problem(B=2, QN=32 if kind == "columns" else 4, KVN=2, q_lens=[rows] * 2, kv_lens=[300, 150], seed=41, **kw)
    g = torch.Generator().manual_seed(42)
    hit = 0
    for b, n in enumerate(p.kv_lens):
        see = bounded.visible(p, b, rows, n).any(0)
        for j in np.flatnonzero(~see.numpy()):
            page, row = _at(p, int(j), b)
            code = torch.randint(0, 126, p.v_cache[page, row].shape, generator=g).to(torch.uint8)
            p.v_cache[page, row] = code.view(p.v_cache.dtype)
            p.v_scale[page, :, row] = 2.0 ** power
            hit += 1
    assert hit > 30
    _check(p, num_sms=num_sms)


@pytest.mark.parametrize("power", [16, 60, 100])
@pytest.mark.parametrize("QN,rows", [(4, 3), (8, 16), (32, 1)])
def test_few_units_with_a_large_key(QN, rows, power):
    """The newest key, which the last row alone sees, has a large V."""
    p = _problem(B=1, QN=QN, KVN=2, q_lens=[rows], kv_lens=[333], seed=43, **FEW)
    page, row = _at(p, 332)
    p.v_scale[page, :, row] *= 2.0 ** power
    _check(p)


@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("at", [0, 200, 2999])
@pytest.mark.parametrize("half,power", [(0.5, 30), (0.5, 45), (1, 60), (1, 90), (2, 90)])
def test_few_units_with_a_large_key_of_little_weight(half, power, at, G):
    """One key's score lies about 27, 54 or 108 below the others' (weights of 2^-39, 2^-78 and
    2^-156), its V up to 2^90 above."""
    p = _problem(B=1, QN=G, KVN=1, q_lens=[1], kv_lens=[3000], seed=44, **FEW)
    p.q[:] = p.q[:, :, :1]
    page, row = _at(p, at)
    six = torch.tensor([6.0]).to(torch.float8_e4m3fn).view(torch.uint8)
    against = torch.where(p.q[0, 0, 0].float() > 0, six | 128, six)
    p.k_cache[page, row, 0] = against.view(p.k_cache.dtype)
    p.k_scale[page, 0, row] = half
    p.v_scale[page, 0, row] *= 2.0 ** power
    _check(p)


@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("power", [-17, -27, -60])
def test_few_units_with_small_values_beside_rows_of_zeros(power, G):
    """64 zeros have a scale of 1, whatever the others' are."""
    p = _problem(B=2, QN=2 * G, KVN=2, q_lens=[1, 1], kv_lens=[700, 130], seed=45, **FEW)
    p.v_scale *= 2.0 ** power
    for b, j in ((0, 3), (0, 400), (1, 128)):
        page, row = _at(p, j, b)
        p.v_cache[page, row] = 0
        p.v_scale[page, :, row] = 1.0
    _check(p)


@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("lo,hi", [(-4, 4), (-8, 7), (-8, 9), (-40, 40), (-90, 90), (-100, -95), (95, 110)])
@pytest.mark.parametrize("kind", ["row", "rows", "columns", "window", "weights"])
def test_scales_of_any_spread(kind, lo, hi, num_sms):
    QN, rows, kw = {"row": (8, 1, {}), "rows": (4, 5, {}), "columns": (32, 1, {}),
                    "window": (8, 2, dict(mask_mode=4, pre_tokens=900, first_tokens=5)),
                    "weights": (8, 1, {})}[kind]
    p = _problem(**{**dict(B=2, QN=QN, KVN=2, q_lens=[rows] * 2, kv_lens=[3000, 1111], seed=46, mask_mode=3), **kw})
    g = torch.Generator().manual_seed(47)
    p.v_scale *= torch.ldexp(torch.ones(()), torch.randint(lo, hi + 1, p.v_scale.shape, generator=g))
    _check(p, weights=kind == "weights", num_sms=num_sms)


@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("steps", [(-30, 0), (0, -30), (0, 14, -27, 0), (-37, -22, -7, 8, 23), (-110, 0)])
def test_scales_that_move_along_the_sequence(steps, num_sms):
    p = _problem(B=1, QN=4, KVN=2, q_lens=[1], kv_lens=[2500], seed=48, mask_mode=3)
    for j in range(2500):
        page, row = _at(p, j)
        p.v_scale[page, :, row] *= 2.0 ** steps[j * len(steps) // 2500]
    _check(p, num_sms=num_sms)


@pytest.mark.parametrize("num_sms", KERNELS)
def test_a_nan_scale_beside_far_ones(num_sms):
    """A NaN stays in its 64 elements, and far scales of one half change the other's by roundings
    alone."""
    p = _problem(B=1, QN=4, KVN=2, q_lens=[1], kv_lens=[300], seed=49, mask_mode=3)
    clean = _run(p, num_sms=num_sms)
    o, l, _, mag, A = bounded.attention(p)[0]
    to = 1.01 * bounded.HALF_BF16 * (mag + o.abs()) + 2 * (bounded.lse_tolerance(p, A, 300) + bounded.HALF_FP16) * mag
    page, row = _at(p, 100)
    p.v_scale[page, 1, row, 1] = 2.0 ** 50
    _check(p, num_sms=num_sms)
    same = torch.ones_like(clean[0], dtype=torch.bool)
    same[0, :, 2:, 64:] = False
    page, row = _at(p, 120)
    p.v_scale[page, 1, row, 1] = float("nan")
    got = _run(p, num_sms=num_sms)
    assert torch.equal(torch.isnan(got[0]), ~same)
    assert torch.all(((got[0][0].cpu().double() - o).abs() <= to)[same[0].cpu()])
    assert torch.all((got[1][0, :, :, 0].T.cpu().double() - l).abs() <= bounded.lse_tolerance(p, A, 300))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("QN,kw", [(4, dict(mask_mode=3)), (16, dict(mask_mode=3)), (4, FEW)])
def test_rows_that_do_not_see_an_infinite_scale(QN, kw, num_sms, value):
    """The newest key's scale is no number: the row that sees it gives NaN, and the others give
    NaN or what they are, nothing between."""
    p = _problem(B=1, QN=QN, KVN=2, q_lens=[4], kv_lens=[700], seed=50, **kw)
    o, _, _, mag, A = bounded.attention(p)[0]
    page, row = _at(p, 699)
    p.v_scale[page, :, row] = value
    got = _run(p, num_sms=num_sms)[0][0].cpu().double()
    # (infinities times codes of either sign, or of 0)
    assert not torch.isfinite(got[3]).any()
    to = 1.01 * bounded.HALF_BF16 * (mag + o.abs()) + 2 * (bounded.lse_tolerance(p, A, 700) + bounded.HALF_FP16) * mag
    assert torch.all(((got - o).abs() <= to)[:3] | torch.isnan(got[:3]))


@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("QN,rows,kw", [(8, 1, {}), (32, 1, {}), (4, 3, {}), (4, 3, FEW)])
def test_scales_of_either_sign(QN, rows, kw, num_sms):
    """A value is its code times its scale, whatever the scale's sign."""
    p = _problem(**{**dict(B=2, QN=QN, KVN=2, q_lens=[rows] * 2, kv_lens=[900, 333], seed=51, mask_mode=3), **kw})
    g = torch.Generator().manual_seed(52)
    for s in (p.k_scale, p.v_scale):
        s *= torch.where(torch.rand(s.shape, generator=g) < 0.5, -1.0, 1.0)
    _check(p, num_sms=num_sms)
