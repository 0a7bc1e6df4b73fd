"""Rows whose scores are NaN give NaN, in one chunk or in many, and rows without keys zeros."""
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import serving
from tests.test_mx_cache_gpu import NO_CLUSTER

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LENS = [2049, 1025, 0, 129, 1]


def _problem(fmt, rows=1, QN=4, **kw):
    args = dict(B=len(LENS), QN=QN, KVN=2, q_lens=[rows] * len(LENS), kv_lens=LENS, block_size=32, seed=71,
                poison=False, mask_mode=3)
    args.update(kw)
    if fmt == "mx":
        return serving.make_mx(**args)
    return fi.make_fia(D=128, kv_dtype=fi.KV_FP8_E4M3 if fmt == "fp8" else fi.KV_BF16, **args)


def _poison_key(p, fmt, b, j):
    page, row = int(p.block_table[b, j // p.block_size]), j % p.block_size
    if fmt == "mx":
        p.k_scale[page, :, row, 1] = 255
    elif fmt == "fp8":
        p.k_cache[page, row, :, 40] = 0x7F
    else:
        p.k_cache[page, row, :, 40] = float("nan")


def _out(p, num_sms, weights=False):
    call = (fia.KeyWeightsCall if weights else fia.FiaCall)(p.to(DEV), num_sms=num_sms)
    got = call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 0
    return [x.cpu() for x in got]


def _check(got, clean, bad):
    """bad [B, S, QN]: the rows that are NaN; the others' bits stay."""
    assert torch.equal(torch.isnan(got[0]), bad[..., None].expand(got[0].shape))
    assert torch.equal(got[0][~bad], clean[0][~bad])
    lse, was = (x[1][..., 0].transpose(1, 2) for x in (got, clean))
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(lse[~bad], was[~bad])


@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("kind", ["plain", "sinks", "window", "weights", "columns"])
@pytest.mark.parametrize("fmt", ["mx", "fp8", "bf16"])
def test_a_nan_key_alone_in_the_last_chunk(fmt, kind, num_sms):
    kw = {"window": dict(mask_mode=4, pre_tokens=5000, first_tokens=4), "sinks": dict(with_sinks=True),
          "columns": dict(QN=32)}.get(kind, {})
    p = _problem(fmt, **kw)
    clean = _out(p, num_sms, kind == "weights")
    bad = torch.zeros(clean[0].shape[:3], dtype=torch.bool)
    for b, n in enumerate(LENS):
        if n:
            _poison_key(p, fmt, b, n - 1)
            bad[b] = True
    _check(_out(p, num_sms, kind == "weights"), clean, bad)


@pytest.mark.parametrize("num_sms", [0, 1, NO_CLUSTER])
@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("fmt", ["mx", "fp8", "bf16"])
def test_a_nan_query_over_many_chunks(fmt, rows, num_sms):
    p = _problem(fmt, rows)
    clean = _out(p, num_sms)
    bad = torch.zeros(clean[0].shape[:3], dtype=torch.bool)
    for b, n in enumerate(LENS):
        p.q[b, rows - 1, 1, 9] = float("nan")
        bad[b, rows - 1, 1] = n > 0
    _check(_out(p, num_sms), clean, bad)


@pytest.mark.parametrize("fmt", ["mx", "fp8", "bf16"])
def test_prompts(fmt):
    p = _problem(fmt, 30, kv_lens=[2049, 1025, 0, 129, 1])
    clean = _out(p, 0)
    bad = torch.zeros(clean[0].shape[:3], dtype=torch.bool)
    for b, n in enumerate(LENS):
        p.q[b, 29, 1, 9] = float("nan")
        bad[b, 29, 1] = n > 0
    _check(_out(p, 0), clean, bad)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("parts", [[1], [0, 1, 2], [2]])
def test_a_part_that_is_nan(parts, sinks):
    """Rows of which some parts are NaN, or all, and rows that no part sees."""
    T, N, D, n = 5, 3, 128, 3
    g = torch.Generator().manual_seed(72)
    outs = [torch.randn(T, N, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(n)]
    lses = [torch.randn(T, N, 1, generator=g).to(DEV) for _ in range(n)]
    for l in lses:
        l[4] = float("inf")
    kw = dict(layout=fi.LAYOUT_TND, num_heads=N, total_q=T,
              sinks=torch.randn(N, generator=g).to(DEV) if sinks else None)
    clean = [x.clone() for x in fia.lse_combine(outs, lses, **kw)]
    for k in parts:
        outs[k][2, 1] = float("nan")
        lses[k][2, 1] = float("nan")
    out, lse = fia.lse_combine(outs, lses, **kw)
    bad = torch.zeros(T, N, dtype=torch.bool, device=DEV)
    bad[2, 1] = True
    assert torch.equal(torch.isnan(out), bad[..., None].expand(out.shape)) and torch.equal(torch.isnan(lse)[..., 0], bad)
    assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])
    assert torch.all(out[4] == 0) and torch.all(lse[4] == float("inf"))
