"""Edges of the attention and bounded-cache calls on the GPU: tables, lengths and
tensors that lie outside what a call was given."""
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from tests import bounded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

# CTAs too few for a cluster: a call of few units takes the kernels of larger ones
NO_CLUSTER = 7


# ----------------------------------------------------------------------------
# pages outside the pool
# ----------------------------------------------------------------------------

def _with_zero_page(p):
    """The problem with a page of zeros at its pool's end; its number."""
    def longer(t):
        return None if t is None else torch.cat([t, torch.zeros_like(t[:1])])
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        setattr(p, name, longer(getattr(p, name)))
    p.num_blocks += 1
    return p.num_blocks - 1


# 64-row pages: 2^26 of them are 2^32 rows, which is row 0 in 32 bits
@pytest.mark.parametrize("page", [1 << 26, -(1 << 26), (1 << 26) + 1, -1, 5000])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["decode", "window", "weights", "prompt", "window_prompt",
                                  "weights_prompt"])
@pytest.mark.parametrize("kv_layout", [0, 1])
def test_pages_outside_the_pool_read_as_zeros(kind, fp8, page, kv_layout):
    """The same bits as with a page of zeros in their place, on every path."""
    prompt = kind.endswith("prompt")
    kw = dict(mask_mode=fi.MASK_BAND, pre_tokens=150, first_tokens=4) if "window" in kind \
        else dict(mask_mode=fi.MASK_RIGHT_DOWN_CAUSAL)
    p = fi.make_fia(B=3, QN=8, KVN=2, D=128, q_lens=[200, 40, 77] if prompt else [1, 2, 1],
                    kv_lens=[300, 40, 500], layout=fi.LAYOUT_TND, block_size=64, seed=31,
                    kv_layout=kv_layout, kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16,
                    device=DEV, **kw)
    zero = _with_zero_page(p)
    for num_sms in (0, NO_CLUSTER):
        got = []
        for entry in (zero, page):
            p.block_table[0, 4], p.block_table[2, 0], p.block_table[2, 6] = entry, entry, entry
            call = (fia.KeyWeightsCall if "weights" in kind else fia.FiaCall)(p, num_sms=num_sms)
            call.ws.fill_(0x7f)  # (bf16, fp16 and fp32 bytes of huge numbers or NaN)
            got.append([x.clone() for x in call.run()])
            torch.cuda.synchronize()
            assert call.error_word() == 0
        for a, b in zip(*got):
            assert torch.isfinite(a.float()).all() and torch.equal(a, b)
