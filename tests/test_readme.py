"""The README's bounded chat, run as it stands."""
import os
import re
from types import SimpleNamespace

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _chat():
    text = open(os.path.join(ROOT, "README.md")).read()
    return re.search(r"A bounded chat.*?```python\n(.*?)```", text, re.S).group(1)


class _Host:
    """The calls of the example without a GPU: the live length, and who used what."""

    def __init__(self, live):
        self.live, self.evictions = live, 0

    def KvCache(self, *a, **kw):
        return SimpleNamespace()

    def kv_append(self, cache, k, v, lens, **kw):
        self.live = self.live + 1
        assert torch.equal(lens, self.live)

    def KeyWeightsCall(self, problem, weights, weights_out):
        assert torch.equal(problem.seqused_kv, self.live), "attention over other keys than are left"
        return SimpleNamespace(run=lambda: (0, 0, weights_out))

    def kv_evict(self, cache, lens, w, budget, positions, weights_out=None, positions_out=None, **kw):
        assert torch.equal(lens, self.live)
        self.evictions += 1
        self.live = self.live.clamp(max=budget)
        return (self.live.clone(), torch.empty_like(w) if weights_out is None else weights_out,
                torch.empty_like(positions) if positions_out is None else positions_out)


def test_the_chat_keeps_one_length():
    """Attention goes on with the lengths that an eviction left."""
    lens = torch.tensor([60, 31], dtype=torch.int32)
    host = _Host(lens.clone())
    names = dict(fia=host, problem=SimpleNamespace(seqused_kv=lens.clone()), k_pool=0, v_pool=0,
                 block_table=0, lens=lens, seen=lens.clone(), k_new=0, v_new=0, w=torch.zeros(2, 1, 99),
                 pos=torch.zeros(2, 1, 99), budget=64, page=16)
    names["problem"].seqused_kv = names["lens"]
    for _ in range(60):
        names["longest"] = int(host.live.max())
        exec(_chat(), names)
    assert host.evictions >= 2


@pytest.mark.gpu
def test_the_chat_on_the_gpu():
    """Each step's attention against 64 bits, over the cache as it stands."""
    import decode_tile_scheduler_gb300 as fia
    import fia_inputs as fi
    from tests import bounded
    dev, B, KVN, page = "cuda:0", 2, 2, 128
    p = fi.make_fia(B=B, QN=4, KVN=KVN, D=128, q_lens=[1] * B, kv_lens=[7 * page] * B,
                    block_size=page, mask_mode=fi.MASK_RIGHT_DOWN_CAUSAL, seed=3, device=dev)
    g = torch.Generator().manual_seed(4)
    for t in (p.k_cache, p.v_cache):
        t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
    p.seqused_kv.copy_(torch.tensor([640, 500]))
    names = dict(fia=fia, problem=p, k_pool=p.k_cache, v_pool=p.v_cache, block_table=p.block_table,
                 lens=p.seqused_kv, seen=p.seqused_kv.clone(), budget=512, page=page, longest=640,
                 w=torch.rand(B, KVN, 7 * page, generator=g).to(dev),
                 pos=torch.arange(7 * page, device=dev).int().repeat(B, KVN, 1))
    evictions = 0
    for step in range(6):
        for n in ("k_new", "v_new"):
            names[n] = torch.randn(B, 1, KVN, 128, generator=g).to(torch.bfloat16).to(dev)
        p.q.copy_(torch.randn(p.q.shape, generator=g).to(p.q.dtype))
        before = names["longest"]
        exec(_chat(), names)
        torch.cuda.synchronize()
        if names["longest"] < before:
            evictions += 1
            assert p.seqused_kv.tolist() == [512, 501]
        else:
            p.kv_lens = p.seqused_kv.tolist()
            bounded.check_attention(p, names["out"], names["lse"])
    assert evictions == 1
