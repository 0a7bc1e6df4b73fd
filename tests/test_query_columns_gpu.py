"""Decode calls whose query heads and rows differ by far: each column stands by itself."""
import copy

import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import serving
from tests.test_mx_cache_gpu import NO_CLUSTER

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _problem(fmt, QN, KVN, rows, kv, **kw):
    args = dict(B=2, QN=QN, KVN=KVN, q_lens=[rows] * 2, kv_lens=kv, block_size=64, seed=61, poison=False,
                mask_mode=3)
    args.update(kw)
    if fmt == "mx":
        return serving.make_mx(**args)
    return fi.make_fia(D=128, kv_dtype=fi.KV_FP8_E4M3 if fmt == "fp8" else fi.KV_BF16, **args)


def _out(p, num_sms, weights=False):
    call = (fia.KeyWeightsCall if weights else fia.FiaCall)(p.to(DEV), num_sms=num_sms)
    got = call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 0
    return [x.cpu() for x in got]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 2.0 ** 100])
@pytest.mark.parametrize("fmt", ["mx", "fp8", "bf16"])
@pytest.mark.parametrize("QN,KVN,rows", [(4, 1, 1), (32, 2, 1), (4, 2, 3), (4, 1, 16)])
@pytest.mark.parametrize("num_sms", [0, NO_CLUSTER])
@pytest.mark.parametrize("window", [False, True])
def test_an_outlying_query_stays_in_its_column(fmt, QN, KVN, rows, value, num_sms, window):
    kw = dict(mask_mode=4, pre_tokens=300, first_tokens=4) if window else {}
    p = _problem(fmt, QN, KVN, rows, [700, 1500], **kw)
    clean = _out(p, num_sms)
    head, row = QN - 1, rows - 1
    p.q[1, row, head, 77] = value
    got = _out(p, num_sms)
    same = torch.ones_like(clean[0], dtype=torch.bool)
    same[1, row, head] = False
    assert torch.equal(got[0][same], clean[0][same])
    assert torch.isfinite(got[0][same]).all()
    lse_same = torch.ones_like(clean[1], dtype=torch.bool)
    lse_same[1, head, row] = False  # [B, QN, S, 1]
    assert torch.equal(got[1][lse_same], clean[1][lse_same])
    assert not torch.equal(got[0][~same], clean[0][~same])


@pytest.mark.parametrize("fmt", ["mx", "fp8"])
@pytest.mark.parametrize("num_sms", [0, NO_CLUSTER])
def test_heads_of_every_size(fmt, num_sms):
    """Heads from 2^-90 to 2^90 side by side have the outputs that they have alone."""
    p = _problem(fmt, 8, 1, 1, [900, 300], scale=0.09)
    mult = torch.tensor([2.0 ** e for e in (-90, -40, -10, 0, 5, 30, 60, 90)]).to(torch.bfloat16)
    p.q *= mult[:, None]
    got = _out(p, num_sms)
    for h in range(8):
        alone = copy.copy(p)
        alone.q = p.q.clone()
        alone.q[:, :, [i for i in range(8) if i != h]] = 0
        want = _out(alone, num_sms)
        assert torch.equal(got[0][:, :, h], want[0][:, :, h]) and torch.equal(got[1][:, h], want[1][:, h])


@pytest.mark.parametrize("fmt", ["mx", "fp8"])
def test_key_weights_beside_a_nan_query(fmt):
    """The other sequence's and the other KV head's weights stay."""
    p = _problem(fmt, 4, 2, 1, [700, 1500])
    clean = _out(p, 0, weights=True)
    p.q[1, 0, 3, 5] = float("nan")
    got = _out(p, 0, weights=True)
    assert torch.equal(got[2][0, :, :700], clean[2][0, :, :700])
    assert torch.equal(got[2][1, 0, :1500], clean[2][1, 0, :1500])
