"""V scales of an MXFP4 cache far apart: a key counts by its weight, however large its V is
and whichever rows it is hidden from."""
import numpy as np
import pytest
import torch

import fia_inputs as fi
from tests import bounded, serving
from tests.test_mx_cache_gpu import NO_CLUSTER, _check, _run

pytestmark = pytest.mark.gpu

KERNELS = [0, NO_CLUSTER]


def _at(p, j, b=0):
    return int(p.block_table[b, j // p.block_size]), j % p.block_size


def _spread(p, lo, hi, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, p.v_scale.shape, generator=g).to(torch.uint8)


@pytest.mark.parametrize("code", [140, 200, 250])
@pytest.mark.parametrize("num_sms", KERNELS)
@pytest.mark.parametrize("kind", ["explicit", "explicit_rows", "left_up", "left_up_16", "band", "band_rows"])
def test_hidden_keys_take_no_part(kind, num_sms, code):
    """Keys that a mask hides from every row hold any finite bytes under a large scale."""
    rows = {"explicit": 1, "explicit_rows": 3, "left_up": 3, "left_up_16": 16, "band": 1, "band_rows": 4}[kind]
    kw = {"e": dict(mask_mode=1, mask_density=0.5), "l": dict(mask_mode=2),
          "b": dict(mask_mode=4, pre_tokens=40)}[kind[0]]
    p = serving.make_mx(B=2, QN=4, KVN=2, q_lens=[rows] * 2, kv_lens=[300, 150], block_size=64, seed=41,
                        poison=False, **kw)
    g = torch.Generator().manual_seed(42)
    hit = 0
    for b, n in enumerate(p.kv_lens):
        see = bounded.visible(p, b, rows, n).any(0)
        for j in np.flatnonzero(~see.numpy()):
            page, row = _at(p, int(j), b)
            p.v_cache[page, row] = torch.randint(0, 256, p.v_cache[page, row].shape, generator=g).to(torch.uint8)
            p.v_scale[page, :, row] = code
            hit += 1
    assert hit > 30
    _check(p, num_sms=num_sms)


@pytest.mark.parametrize("code", [150, 187, 247])
@pytest.mark.parametrize("QN,rows", [(4, 3), (8, 16), (2, 2)])
@pytest.mark.parametrize("num_sms", KERNELS)
def test_a_key_that_only_another_row_sees(num_sms, QN, rows, code):
    """The newest key, which the last row alone sees, has a large V."""
    p = serving.make_mx(B=1, QN=QN, KVN=2, q_lens=[rows], kv_lens=[333], block_size=64, seed=43,
                        mask_mode=3, poison=False)
    page, row = _at(p, 332)
    p.v_scale[page, :, row] = code
    _check(p, num_sms=num_sms)


@pytest.mark.parametrize("num_sms", KERNELS)
@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("at", [0, 200, 2999])
@pytest.mark.parametrize("half,code", [(126, 157), (126, 172), (127, 187), (127, 217), (128, 220)])
def test_a_large_key_of_little_weight(half, code, at, G, num_sms):
    """One key's score lies 27, 54 or 108 below the others' (weights of 2^-39, 2^-78 and
    2^-156), its V up to 2^90 above: what it counts for is neither lost nor others' loss."""
    p = serving.make_mx(B=1, QN=G, KVN=1, q_lens=[1], kv_lens=[3000], block_size=64, seed=44,
                        mask_mode=3, poison=False)
    p.q[:] = p.q[:, :, :1]
    page, row = _at(p, at)
    against = torch.where(p.q[0, 0, 0].float() > 0, 15, 7)  # -6 or 6
    p.k_cache[page, row, 0] = (against[0::2] | against[1::2] << 4).to(torch.uint8)
    p.k_scale[page, 0, row] = half
    p.v_scale[page, 0, row] = code
    _check(p, num_sms=num_sms)


@pytest.mark.parametrize("num_sms", KERNELS)
@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("power", [-17, -27, -60])
def test_small_values_beside_rows_of_zeros(power, G, num_sms):
    """32 zeros have a scale of 1, whatever the others' are."""
    p = fi.make_fia(B=2, QN=2 * G, KVN=2, D=128, q_lens=[1, 1], kv_lens=[700, 130], block_size=64, seed=45,
                    mask_mode=3, poison=False)
    p.v_cache = p.v_cache * 2.0 ** power
    for b, j in ((0, 3), (0, 400), (1, 128)):
        page, row = _at(p, j, b)
        p.v_cache[page, row] = 0
    p = serving.as_mx(p)
    assert int(p.v_scale[page, 0, row, 0]) == 127
    _check(p, num_sms=num_sms)


@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("lo,hi", [(120, 134), (120, 135), (120, 136), (107, 147), (30, 220), (0, 20), (235, 250)])
@pytest.mark.parametrize("kind", ["row", "rows", "columns", "window", "weights"])
def test_scales_of_any_spread(kind, lo, hi, num_sms):
    QN, rows, kw = {"row": (8, 1, {}), "rows": (4, 5, {}), "columns": (32, 1, {}),
                    "window": (8, 2, dict(mask_mode=4, pre_tokens=900, first_tokens=5)),
                    "weights": (8, 1, {})}[kind]
    p = serving.make_mx(**{**dict(B=2, QN=QN, KVN=2, q_lens=[rows] * 2, kv_lens=[3000, 1111], block_size=64,
                                  seed=46, mask_mode=3, poison=False), **kw})
    p.v_scale = _spread(p, lo, hi, 47)
    _check(p, weights=kind == "weights", num_sms=num_sms)


@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("steps", [(97, 127), (127, 97), (127, 141, 100, 127), (90, 105, 120, 135, 150), (0, 127)])
def test_scales_that_move_along_the_sequence(steps, num_sms):
    """Runs of keys of one scale: the reference moves up, down, and past a window's ends."""
    p = serving.make_mx(B=1, QN=4, KVN=2, q_lens=[1], kv_lens=[2500], block_size=64, seed=48, mask_mode=3,
                        poison=False)
    for j in range(2500):
        page, row = _at(p, j)
        p.v_scale[page, :, row] = steps[j * len(steps) // 2500]
    _check(p, num_sms=num_sms)


@pytest.mark.parametrize("num_sms", KERNELS)
def test_a_nan_scale_beside_far_ones(num_sms):
    """A NaN stays in its 32 elements where their scales are far apart too, and those of
    other groups leave a group's bits alone."""
    p = serving.make_mx(B=1, QN=4, KVN=2, q_lens=[1], kv_lens=[300], block_size=32, seed=49, mask_mode=3,
                        poison=False)
    clean = _run(p, num_sms=num_sms)
    page, row = _at(p, 100)
    p.v_scale[page, 1, row, 1] = 180
    far = _run(p, num_sms=num_sms)
    same = torch.ones_like(clean[0], dtype=torch.bool)
    same[0, :, 2:, 32:64] = False
    assert torch.equal(far[0][same], clean[0][same])
    page, row = _at(p, 120)
    p.v_scale[page, 1, row, 1] = 255
    got = _run(p, num_sms=num_sms)
    assert torch.equal(torch.isnan(got[0]), ~same) and torch.equal(got[0][same], clean[0][same])
    assert torch.equal(got[1], clean[1])


def test_many_rows_of_far_scales():
    """A large call, every chunk with far groups, twice: the same bits."""
    p = serving.make_mx(B=24, QN=16, KVN=2, q_lens=[2] * 24, kv_lens=list(range(40, 2440, 100)), block_size=32,
                        seed=50, mask_mode=3, poison=False)
    p.v_scale = _spread(p, 100, 150, 51)
    _check(p)
    assert all(torch.equal(x, y) for x, y in zip(_run(p), _run(p)))


@pytest.mark.parametrize("lo,hi", [(120, 134), (107, 147), (30, 220)])
@pytest.mark.parametrize("QN,rows,weights", [(32, 1, True), (4, 9, True), (4, 3, True), (8, 1, True), (4, 3, False),
                                             (8, 1, False), (32, 1, False), (4, 16, False)])
def test_every_kernel_with_far_scales(QN, rows, weights, lo, hi):
    """8 and 16 columns, one row and several, with and without key weights."""
    p = serving.make_mx(B=2, QN=QN, KVN=2, q_lens=[rows] * 2, kv_lens=[1500, 333], block_size=64, seed=52,
                        mask_mode=3, poison=False)
    p.v_scale = _spread(p, lo, hi, 53)
    _check(p, weights=weights, num_sms=NO_CLUSTER)


@pytest.mark.parametrize("code", [252, 253, 254])
@pytest.mark.parametrize("rows,num_sms", [(40, 0), (3, 0), (3, NO_CLUSTER)])
@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
def test_the_largest_scales_reach_their_rows_alone(name, rows, num_sms, code):
    """The newest key's values lie at bf16's end and past it: the rows that do not see it keep
    their bits."""
    p = serving.make_mx(B=1, QN=4, KVN=2, q_lens=[rows], kv_lens=[300], block_size=32, seed=54, mask_mode=3,
                        poison=False)
    clean = [x.cpu().clone() for x in _run(p, num_sms=num_sms)]
    page, row = _at(p, 299)
    getattr(p, name)[page, :, row] = code
    got = [x.cpu() for x in _run(p, num_sms=num_sms)]
    before = slice(0, rows - 1)
    assert torch.isfinite(got[0][:, before]).all()
    if rows > 16:
        assert torch.equal(got[0][:, before], clean[0][:, before])
    else:  # (a far group's products are made in other roundings)
        o, _, _, mag, A = bounded.attention(serving.decoded(p))[0]
        tl = bounded.lse_tolerance(p, min(A, 100.0), 300)
        to = 1.01 * bounded.HALF_BF16 * (mag + o.abs()) + 2 * tl * mag
        assert torch.all(((got[0][0].double() - o).abs() <= to)[before])
    assert torch.equal(got[1][:, :, before], clean[1][:, :, before])
