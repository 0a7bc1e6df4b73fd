"""Decode calls with scores past fp32's whole numbers."""
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import bounded, serving
from tests.test_mx_cache_gpu import NO_CLUSTER

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("QN", [8, 32])
@pytest.mark.parametrize("fmt", ["mx", "fp8", "bf16"])
@pytest.mark.parametrize("num_sms", [0, NO_CLUSTER])
def test_scores_past_fp32s_steps(fmt, num_sms, QN):
    """Scores of up to 2^60: one key takes all, and nothing overflows."""
    kw = dict(B=2, QN=QN, KVN=2, q_lens=[1, 1], kv_lens=[900, 300], block_size=64, seed=61, poison=False,
              mask_mode=3, scale=2.0 ** 50)
    if fmt == "mx":
        p = serving.make_mx(**kw)
    else:
        p = fi.make_fia(D=128, kv_dtype=fi.KV_FP8_E4M3 if fmt == "fp8" else fi.KV_BF16, **kw)
    call = fia.FiaCall(p.to("cuda:0"), num_sms=num_sms)
    out, lse = (x.cpu().double() for x in call.run())
    ref = bounded.attention(serving.decoded(p) if fmt == "mx" else p)
    for b, (o, l, w, mag, A) in enumerate(ref):
        assert torch.isfinite(out[b]).all()
        # (fp32 sums of products: 2 D / 16 truncations of A at most, four more roundings)
        assert torch.all((lse[b, :, :, 0].T - l).abs() <= (2 * 128 / 16 + 4) * bounded.HALF_FP32 * 1.45 * A)
