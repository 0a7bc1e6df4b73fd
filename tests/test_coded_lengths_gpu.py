"""Lengths at the ends of 32 bits, over coded caches."""
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import bounded, serving
from tests.test_mx_cache_gpu import NO_CLUSTER

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("length", [-(1 << 31), 3 - (1 << 31), -1200, -1, (1 << 31) - 1])
@pytest.mark.parametrize("rows,num_sms", [(40, 0), (1, 0), (1, NO_CLUSTER)])
@pytest.mark.parametrize("fmt", ["mx", "fp8"])
@pytest.mark.parametrize("paged", [False, True])
def test_lengths_at_the_ends_of_32_bits(fmt, rows, num_sms, length, paged):
    """The last sequence's length lies outside its cache, whose 1204 rows are no multiple of
    what a block of the conversion takes: nothing behind the workspace is written, and the
    other sequence has its outputs."""
    kw = dict(B=2, QN=8, KVN=8, q_lens=[rows] * 2, kv_lens=[1203, 700], seed=81, mask_mode=3, poison=False)
    kw.update(dict(block_size=32) if paged else dict(paged=False, S_kv=1204))
    p = serving.make_mx(**kw) if fmt == "mx" else fi.make_fia(D=128, kv_dtype=fi.KV_FP8_E4M3, **kw)
    d = p.to(DEV)
    clean = [x.clone() for x in fia.FiaCall(d, num_sms=num_sms).run()]
    ref = bounded.attention(serving.decoded(p) if fmt == "mx" else p)[0]
    d.seqused_kv[1] = length
    call = fia.FiaCall(d, num_sms=num_sms)
    call.ws = torch.full((call.ws_bytes + (1 << 20),), 0x5A, dtype=torch.uint8, device=DEV)
    out, lse = call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 2
    if rows > 16:
        assert torch.equal(out[0], clean[0][0]) and torch.equal(lse[0], clean[1][0])
    else:  # (chunks go by all lengths together: other chunks, other roundings of 64 bits' values)
        o, l, _, mag, A = ref
        tl = bounded.lse_tolerance(p, A, 1203)
        assert torch.all((out[0].cpu().double() - o).abs()
                         <= 1.01 * bounded.HALF_BF16 * (mag + o.abs()) + 2 * (tl + bounded.HALF_FP16) * mag)
        assert torch.all((lse[0, :, :, 0].T.cpu().double() - l).abs() <= tl)
    assert torch.all(call.ws[call.ws_bytes:] == 0x5A)
