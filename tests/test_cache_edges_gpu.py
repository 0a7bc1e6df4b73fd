"""Edges of the attention and bounded-cache calls on the GPU: tables, lengths and
tensors that lie outside what a call was given."""
import copy
import math

import pytest
import torch

import decode_tile_scheduler_gb300 as fia
import fia_inputs as fi
from decode_tile_scheduler_gb300 import api
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


# ----------------------------------------------------------------------------
# lengths outside a decode call's tensors
# ----------------------------------------------------------------------------

def _alone(p, b):
    """Sequence b of a TND problem, for the 64-bit check."""
    one, t0 = copy.copy(p), sum(p.q_lens[:b])
    one.B, one.T, one.q_lens, one.kv_lens = 1, p.q_lens[b], p.q_lens[b:b + 1], p.kv_lens[b:b + 1]
    one.q, one.block_table = p.q[t0:t0 + one.T], p.block_table[b:b + 1]
    return one


@pytest.mark.parametrize("bad", ["rows", "negative_row", "keys", "negative_keys"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("num_sms", [0, NO_CLUSTER])
def test_decode_lengths_outside_the_tensors(num_sms, weights, fp8, bad):
    """A sequence whose rows lie outside q, or whose length is past the capacity:
    it runs as empty, the error word says 2, the others get their results (not the
    same bits: the plan cuts by the lengths of all), and nothing is written outside
    the outputs (which lie inside larger ones here)."""
    T, slack = 6, 40
    p = fi.make_fia(B=3, QN=8, KVN=2, D=128, q_lens=[2, 2, 2], kv_lens=[1500, 700, 300],
                    layout=fi.LAYOUT_TND, block_size=32, seed=33, mask_mode=fi.MASK_BAND,
                    pre_tokens=900, first_tokens=4, device=DEV,
                    kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16)
    p.q = torch.cat([p.q.new_zeros(slack, 8, 128), p.q, p.q.new_zeros(slack, 8, 128)])[slack:-slack]
    cap = p.block_table.shape[1] * 32
    big = {"out": torch.full((T + 2 * slack, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV),
           "lse": torch.full((T + 2 * slack, 8, 1), 3.0, device=DEV),
           "w": torch.full((5, 2, cap), 3.0, device=DEV)}

    def run():
        for x in big.values():
            x.fill_(3.0)
        kw = dict(num_sms=num_sms, out=big["out"][slack:-slack], lse=big["lse"][slack:-slack])
        call = fia.KeyWeightsCall(p, weights_out=big["w"][1:4], **kw) if weights \
            else fia.FiaCall(p, **kw)
        call.run()
        torch.cuda.synchronize()
        return call.error_word(), {n: x.clone() for n, x in big.items()}

    assert run()[0] == 0
    if bad == "rows":
        p.cu_seqlens_q[3] += 7   # sequence 2: rows 4 and on; two of them at most are taken
        p.cu_seqlens_q[2] += 1   # and it starts a row later, so that they pass the last one
        hit, fine = [2], [0]
    elif bad == "negative_row":
        p.cu_seqlens_q[0] = -1
        hit, fine = [0], [1, 2]
    else:
        p.seqused_kv[1] = cap + 1 if bad == "keys" else -3
        hit, fine = [1], [0, 2]
    word, got = run()
    assert word == 2
    rows = {0: slice(slack, slack + 2), 1: slice(slack + 2, slack + 4), 2: slice(slack + 4, slack + 6)}
    for name in ("out", "lse"):
        assert torch.all(got[name][:slack] == 3.0) and torch.all(got[name][slack + T:] == 3.0)
    if bad != "negative_row":  # (the rows before the first belong to nobody)
        last = rows[hit[0]]
        assert torch.all(got["out"][last.stop - 1] == 3.0)
    assert torch.all(got["w"][0] == 3.0) and torch.all(got["w"][4] == 3.0)
    for b in fine:
        bounded.check_attention(_alone(p, b), got["out"][rows[b]], got["lse"][rows[b]],
                                got["w"][1 + b:2 + b] if weights else None)


# ----------------------------------------------------------------------------
# the stream argument
# ----------------------------------------------------------------------------

def _handle(s, as_int):
    return s.cuda_stream if as_int else s


@pytest.mark.parametrize("as_int", [False, True])
def test_evict_on_a_stream_while_the_current_one_is_busy(as_int):
    """kv_evict(stream=s): the fills of the tensors that it makes come before its
    kernel, whatever the current stream still has to do."""
    B, KVN, D, block = 2, 2, 128, 32
    g = torch.Generator().manual_seed(3)
    pools = [torch.randn(20, block, KVN, D, generator=g).to(torch.bfloat16).to(DEV) for _ in "kv"]
    table = torch.arange(8, dtype=torch.int32, device=DEV).reshape(B, 4)
    cache = fia.KvCache(*pools, table)
    lens = torch.tensor([100, 128], dtype=torch.int32, device=DEV)
    w = torch.rand(B, KVN, cache.capacity, device=DEV)
    side = torch.cuda.Stream()
    fia.kv_evict(cache, lens.clone(), w, budget=128)  # (the library is loaded)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    n, wo, po = fia.kv_evict(cache, lens, w, budget=64, recent_tokens=10,
                             stream=_handle(side, as_int))
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream was to be busy"
    torch.cuda.synchronize()
    assert n.tolist() == [64, 64]
    for b in range(B):
        for h in range(KVN):
            kept = bounded.keep_of(w[b, h].cpu().numpy(), None, int(lens[b]), 64, 0, 10, int(lens[b]))
            slots = po[b, h, :64].tolist()
            assert sorted(slots) == list(kept.nonzero()[0])
            assert torch.equal(wo[b, h, :64], w[b, h][slots])


@pytest.mark.parametrize("as_int", [False, True])
def test_the_workspace_of_a_call_on_a_slow_stream_stays_its_own(as_int, monkeypatch):
    """fused_infer_attention(stream=s): its workspace is not the current stream's
    to give away while s has not run the call."""
    p = fi.make_fia(B=40, QN=8, KVN=2, D=128, q_lens=[1] * 40, kv_lens=[700] * 40, block_size=64,
                    seed=35, device=DEV)
    want = [x.clone() for x in fia.fused_infer_attention(p)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    made_on = []

    class Spied(fia.FiaCall):
        def __init__(self, *args, **kw):
            made_on.append(torch.cuda.current_stream().cuda_stream)
            super().__init__(*args, **kw)

    monkeypatch.setattr(api, "FiaCall", Spied)
    got = fia.fused_infer_attention(p, stream=_handle(side, as_int))
    # (a block of the side stream's: the next tensor of that size there comes behind the call)
    assert made_on == [side.cuda_stream]
    torch.full((64 << 20,), 0x7f, dtype=torch.uint8, device=DEV)  # the current stream's next tensor
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------
# no rows
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("layout", [fi.LAYOUT_TND, fi.LAYOUT_BSND])
@pytest.mark.parametrize("fp8", [False, True])
def test_calls_of_no_rows(layout, fp8):
    """A batch of which no sequence has a query row: real tensors, which are empty."""
    B, KVN, D = 3, 2, 128
    p = fi.make_fia(B=B, QN=8, KVN=KVN, D=D, q_lens=[0] * B, kv_lens=[70, 0, 33], layout=layout,
                    block_size=32, seed=37, device=DEV, mask_mode=fi.MASK_RIGHT_DOWN_CAUSAL,
                    kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16)
    assert p.q.numel() == 0
    call = fia.FiaCall(p)
    call.ws.fill_(0x7f)
    out, lse = call.run()
    assert out.numel() == 0 and lse.numel() == 0 and call.error_word() == 0
    w = torch.rand(B, KVN, p.block_table.shape[1] * 32, device=DEV)
    call = fia.KeyWeightsCall(p, weights=w)
    got = call.run()[2]
    assert call.error_word() == 0
    for b, n in enumerate(p.kv_lens):
        assert torch.equal(got[b, :, :n], w[b, :, :n]) and torch.all(got[b, :, n:] == 0)
    assert torch.all(fia.KeyWeightsCall(p).run()[2] == 0)

    cache = fia.KvCache(p.k_cache, p.v_cache, p.block_table, k_scale=p.k_scale, v_scale=p.v_scale)
    before = [x.clone() for x in (p.k_cache, p.v_cache, w)]
    new = torch.zeros((0, KVN, D) if layout == fi.LAYOUT_TND else (B, 0, KVN, D),
                      dtype=torch.bfloat16, device=DEV)
    fia.kv_append(cache, new, new, p.seqused_kv, cu_seqlens_q=p.cu_seqlens_q, weights=w)
    for x, y in zip((p.k_cache, p.v_cache, w), before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ----------------------------------------------------------------------------
# the bits of P over an FP8 cache
# ----------------------------------------------------------------------------

def _check_fp16_p(p, weights):
    """P times its V scale is multiplied in fp16 on both decode paths: half a step
    of fp16 on each term (in the subnormal range of P over a power of two of at
    most the largest scale: 2^-25 of it, times the code), half a step of bf16 on
    the output, and what a score and its row's sum may be off."""
    ref = bounded.attention(p)
    codes = p.v_cache.view(torch.float8_e4m3fn).float().abs().cpu()
    for num_sms in (0, NO_CLUSTER):
        call = (fia.KeyWeightsCall if weights else fia.FiaCall)(p, num_sms=num_sms)
        out = call.run()[0].double().cpu()
        for b, (o, l, w, mag, A) in enumerate(ref):
            kl = p.kv_lens[b]
            tiny = torch.zeros(p.KVN, p.D, dtype=torch.float64)
            for j in range(kl):
                tiny += codes[b, j].double() * 2.0 ** -25
            top = p.v_scale[b, :, :kl].amax(1).double().cpu().repeat_interleave(64, -1)
            tiny = (tiny * top).repeat_interleave(p.QN // p.KVN, 0)
            tl = bounded.lse_tolerance(p, A, kl)
            to = 1.01 * (bounded.HALF_FP16 * mag + bounded.HALF_BF16 * o.abs()) + 2 * tl * mag + tiny
            off = (out[b] - o).abs()
            assert torch.all(off <= to), (num_sms, b, float((off / to).max()))


@pytest.mark.parametrize("weights", [False, True])
def test_p_over_an_fp8_cache_keeps_fp16_bits(weights):
    """Of 16 keys each, 15 have a probability of the first's that lies next to the
    middle between two bf16 values, and values that cancel the first's: rounded to
    bf16, all 15 are off to one side by 2^-8, four times the tolerance."""
    n, p_star = 64, 0.5 + 0.49 * 2.0 ** -8
    p = fi.make_fia(B=1, QN=1, KVN=1, D=128, q_lens=[1], kv_lens=[n], paged=False, S_kv=n,
                    kv_dtype=fi.KV_FP8_E4M3, scale=1.0, device=DEV,
                    **({"mask_mode": fi.MASK_RIGHT_DOWN_CAUSAL} if weights else
                       {"mask_mode": fi.MASK_BAND, "pre_tokens": 100, "first_tokens": 4}))
    first = torch.arange(n, device=DEV) % 16 == 0
    p.q.zero_()
    p.q[..., 0] = 1.0
    p.k_cache.zero_()
    p.k_cache[..., 0] = 0xfe  # -448
    p.k_scale[0, 0] = torch.where(first, 0.0, -math.log(p_star) / 448)[:, None]
    p.v_cache[0, :, 0] = torch.where(first, 0xfe, 0x7e).to(torch.uint8)[:, None]
    for half, unit in ((0, 2.0 ** -9), (1, 2.0 ** 7)):
        p.v_scale[0, 0, :, half] = torch.where(first, 15 * p_star * unit, unit)
    _check_fp16_p(p, weights)


@pytest.mark.parametrize("weights", [False, True])
def test_p_over_an_fp8_cache_with_far_scales(weights):
    """V scales from 2^-20 to 2^20, several steps a warp: the power of two that O is
    kept over moves."""
    n = 3500
    p = fi.make_fia(B=2, QN=4, KVN=2, D=128, q_lens=[1, 1], kv_lens=[n, 1111], paged=False, S_kv=n,
                    kv_dtype=fi.KV_FP8_E4M3, device=DEV, seed=39, poison=False,
                    **({"mask_mode": fi.MASK_RIGHT_DOWN_CAUSAL} if weights else
                       {"mask_mode": fi.MASK_BAND, "pre_tokens": 3000, "first_tokens": 300}))
    g = torch.Generator().manual_seed(40)
    p.v_scale.copy_(2.0 ** (torch.rand(p.v_scale.shape, generator=g) * 40 - 20))
    p.v_scale[1, :, :400] = 0.0  # zeros first
    p.v_scale[1, :, 400:500, 1] *= 2.0 ** -100
    _check_fp16_p(p, weights)


# ----------------------------------------------------------------------------
# the chunks of a window call
# ----------------------------------------------------------------------------

def _chunk_sizes(costs, A, n, k, window):
    """(C, c2) of the decode schedule: tiles per sequence, units per sequence, CTAs."""
    T, U, W, cmax = sum(costs) * A, len(costs) * A, 5, max(costs)
    if window:
        fits = [s for s in range(1, min(16, cmax) + 1) if s == 1 or U * s <= n * W + 2 * k * U]
        times = [(-(-(-(-T // -(-cmax // s))) // n) * (5 * -(-cmax // s) + 13) + (13 if s > 1 else 0), s)
                 for s in fits]
        C = -(-cmax // min(times)[1])
        if C <= 24 or 4 * T >= 3 * U * cmax:
            return C, C
    C = max(1, -(-T // (n * W)))
    return C, -(-C // k)


@pytest.mark.parametrize("fp8,rows", [(False, 1), (True, 1), (False, 2)])
@pytest.mark.parametrize("window,lens", [
    (1 << 20, [60000] + [600] * 9),                  # one long chat among short ones
    (1 << 20, [300, 20000, 9000, 700, 14000, 3000]),
    (1 << 20, [20000, 19000, 18000, 20000]),         # of one size, whatever the window
    (1000, [300, 20000, 9000, 700, 14000, 3000]),    # short units
    (5000, [60000] + [600] * 9),
    (9000, [9500, 16000, 12345]),
])
def test_window_calls_of_unequal_units_are_cut_as_other_calls(window, lens, fp8, rows):
    p = fi.make_fia(B=len(lens), QN=32, KVN=8, D=128, q_lens=[rows] * len(lens), kv_lens=lens,
                    mask_mode=fi.MASK_BAND, pre_tokens=window - 1, first_tokens=4, block_size=128,
                    kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16, device=DEV, poison=False)
    call = fia.FiaCall(p, num_sms=152)
    call.plan()
    torch.cuda.synchronize()
    lay = call.plan_layout()
    C, c2 = call.ws[lay.sched_off:lay.sched_off + 16].view(torch.int64).tolist()
    costs = []
    for n in lens:
        lo, last = max(n - rows - (window - 1), 0) // 128, (n - 1) // 128
        costs.append(last + 1 if lo <= 1 else last - lo + 2)
    k = 2 if not fp8 and rows == 1 else 1
    assert (C, c2) == _chunk_sizes(costs, 8, 152, k, 8 * 8 * len(lens) >= 152)
    if len(lens) == 10 and window > 5000:  # (the rule that this is about)
        assert C < 24


# ----------------------------------------------------------------------------
# table entries that nobody uses
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("any_id", [1 << 30, -(1 << 31), 1 << 26])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_sms", [0, NO_CLUSTER])
@pytest.mark.parametrize("rows", [1, 40])
def test_unused_table_entries_hold_anything(rows, num_sms, fp8, any_id, monkeypatch):
    """Behind a sequence's last page, and in whole tiles between the first tokens and
    the window: the same bits, and nothing to report."""
    p = fi.make_fia(B=2, QN=8, KVN=2, D=128, q_lens=[rows] * 2, kv_lens=[1500, 600], block_size=64,
                    layout=fi.LAYOUT_TND, mask_mode=fi.MASK_BAND, pre_tokens=200, first_tokens=5,
                    seed=43, max_blocks=30, device=DEV,
                    kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16)
    want = [x.clone() for x in fia.FiaCall(p, num_sms=num_sms).run()]
    p.block_table[0, 24:] = any_id
    p.block_table[1, 10:] = any_id
    for b, n in ((0, 1500), (1, 600)):
        p.block_table[b, 2:(n - rows - 200) // 128 * 2] = any_id
    for debug in "01":
        monkeypatch.setenv("FIA_DEBUG", debug)
        call = fia.FiaCall(p, num_sms=num_sms)
        got = call.run()
        torch.cuda.synchronize()
        assert call.error_word() == 0
        if debug == "0":
            assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("fp8", [False, True])
def test_evict_takes_no_page_behind_the_last(fp8):
    B, KVN, D, block, g = 2, 2, 128, 32, torch.Generator().manual_seed(44)
    shape = (40, block, KVN, D)
    pools = [torch.randint(0, 100, shape, generator=g).to(torch.uint8 if fp8 else torch.bfloat16)
             .to(DEV) for _ in "kv"]
    sc = dict(k_scale=torch.rand(40, KVN, block, 2, device=DEV),
              v_scale=torch.rand(40, KVN, block, 2, device=DEV)) if fp8 else {}
    w = torch.rand(B, KVN, 10 * block, device=DEV)
    lens = torch.tensor([150, 97], dtype=torch.int32, device=DEV)
    got = []
    for entry in (3, 1 << 30):
        table = torch.arange(20, dtype=torch.int32, device=DEV).reshape(B, 10)
        table[0, 5:], table[1, 4:] = entry, entry
        mine = [x.clone() for x in pools]
        cache = fia.KvCache(*mine, table, **{k: x.clone() for k, x in sc.items()})
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got.append([*fia.kv_evict(cache, lens, w, budget=64, status=status), *cache.tensors, status])
    for i, (x, y) in enumerate(zip(*got)):
        assert i == 5 or x is None or torch.equal(x, y)  # (5: the table itself)
    assert int(got[1][-1]) == 0


# ----------------------------------------------------------------------------
# lengths outside a prompt call's tensors
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("bad", ["rows", "negative_row", "keys", "negative_keys", "falling"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["causal", "window", "weights"])
@pytest.mark.parametrize("stale", [False, True])
def test_prompt_lengths_outside_the_tensors(stale, kind, fp8, bad):
    """As for decode; `stale`: the lengths go wrong between the plan and the call."""
    T, slack, q_lens = 500, 300, [150, 140, 210]
    kw = dict(mask_mode=fi.MASK_BAND, pre_tokens=90, first_tokens=4) if kind == "window" \
        else dict(mask_mode=fi.MASK_RIGHT_DOWN_CAUSAL)
    p = fi.make_fia(B=3, QN=8, KVN=2, D=128, q_lens=q_lens, kv_lens=[400, 150, 300],
                    layout=fi.LAYOUT_TND, block_size=32, seed=45, device=DEV,
                    kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16, **kw)
    wide = torch.zeros(T + 2 * slack, 8, 128, dtype=torch.bfloat16, device=DEV)
    wide[slack:-slack] = p.q
    p.q = wide[slack:-slack]
    cap = p.block_table.shape[1] * 32
    big = {"out": torch.full((T + 2 * slack, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV),
           "lse": torch.full((T + 2 * slack, 8, 1), 3.0, device=DEV),
           "w": torch.full((5, 2, cap), 3.0, device=DEV)}
    ends = dict(out=big["out"][slack:-slack], lse=big["lse"][slack:-slack])
    weights = kind == "weights"
    call = fia.KeyWeightsCall(p, weights_out=big["w"][1:4], **ends) if weights \
        else fia.FiaCall(p, **ends)
    if stale:
        call.plan()
    if bad == "rows":
        p.cu_seqlens_q[3] += 150
        hit = 2
    elif bad == "negative_row":
        p.cu_seqlens_q[0] = -130
        hit = 0
    elif bad == "falling":
        p.cu_seqlens_q[2] = 140   # sequence 1 has -10 rows, sequence 2 some of sequence 0's
        hit = 1
    else:
        p.seqused_kv[1] = cap + 33 if bad == "keys" else -3
        hit = 1
    call.execute() if stale else call.run()
    torch.cuda.synchronize()
    assert call.error_word() == 2
    for name in ("out", "lse"):
        assert torch.all(big[name][:slack] == 3.0) and torch.all(big[name][slack + T:] == 3.0)
    assert torch.all(big["w"][0] == 3.0) and torch.all(big["w"][4] == 3.0)
    at = slack
    for b, n in enumerate(q_lens):
        rows, at = slice(at, at + n), at + n
        if bad == "falling":
            continue  # (two sequences share rows)
        if b == hit:
            assert torch.all(big["out"][rows] == 3.0) and torch.all(big["lse"][rows] == 3.0)
        else:
            bounded.check_attention(_alone(p, b), big["out"][rows], big["lse"][rows],
                                    big["w"][1 + b:2 + b] if weights else None)


# ----------------------------------------------------------------------------
# keys of a window call that no row sees
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 3, 40, 150])
@pytest.mark.parametrize("kind", ["bf16", "d64", "fp8"])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("ahead", [0, -2])
def test_keys_that_no_row_sees_hold_anything(ahead, weights, kind, rows):
    """NaN, infinities and scales of any size between the first tokens and the window,
    in tiles of which other keys are seen: the same bits as with zeros there."""
    fp8 = kind == "fp8"
    p = fi.make_fia(B=2, QN=8, KVN=2, D=64 if kind == "d64" else 128, q_lens=[rows] * 2,
                    kv_lens=[1500, 700], layout=fi.LAYOUT_TND, block_size=32, seed=47,
                    mask_mode=fi.MASK_BAND, pre_tokens=260, first_tokens=37, next_tokens=ahead,
                    kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16, device=DEV)
    hidden = []
    for b, n in enumerate(p.kv_lens):
        for j in list(range(37, n - rows - 260)) + list(range(n + ahead, n)):
            hidden.append((int(p.block_table[b, j // 32]), j % 32))
    page, row = torch.tensor(hidden).T.to(DEV)
    scales = [3e38, float("nan"), float("inf"), 1e-3]
    for num_sms in (0, NO_CLUSTER):
        got = []
        for garbage in (False, True):
            for i, c in enumerate((p.k_cache, p.v_cache)):
                if fp8:
                    c[page, row] = 0x7f if garbage else 0
                    s = (p.k_scale, p.v_scale)[i].permute(0, 2, 1, 3)
                    s[page, row] = torch.tensor(scales, device=DEV)[row % 4][:, None, None] \
                        if garbage else 1.0
                else:
                    fill = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38],
                                        device=DEV).to(c.dtype)[row % 4]
                    c[page, row] = fill[:, None, None] if garbage else 0.0
            call = (fia.KeyWeightsCall if weights else fia.FiaCall)(p, num_sms=num_sms)
            got.append([x.clone() for x in call.run()])
        for x, y in zip(*got):
            assert torch.isfinite(y.float()).all() and torch.equal(x, y)
        # (as kept tensors: the 64-bit check leaves keys out that nobody sees)
        bounded.check_attention(p, *got[1][:2], *(got[1][2:] if weights else []))


# ----------------------------------------------------------------------------
# a padded batch, and a decode without a workspace
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 3, 70])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_rows_behind_the_last_sequence_are_left(weights, fp8, rows):
    """q longer than cu_seqlens_q says: out and lse keep what they held there."""
    pad = 9
    p = fi.make_fia(B=3, QN=8, KVN=2, D=128, q_lens=[rows, 0, rows], kv_lens=[800, 90, 260],
                    layout=fi.LAYOUT_TND, block_size=32, seed=49, mask_mode=fi.MASK_BAND,
                    pre_tokens=200, first_tokens=4, device=DEV,
                    kv_dtype=fi.KV_FP8_E4M3 if fp8 else fi.KV_BF16)
    n = p.T
    p.q, p.T = torch.cat([p.q, torch.full_like(p.q[:1], float("nan")).expand(pad, -1, -1)]), n + pad
    for num_sms in (0, NO_CLUSTER):
        out = torch.full_like(p.q, 3.0)
        lse = torch.full((n + pad, 8, 1), 3.0, device=DEV)
        call = (fia.KeyWeightsCall if weights else fia.FiaCall)(p, num_sms=num_sms, out=out, lse=lse)
        got = call.run()
        torch.cuda.synchronize()
        assert call.error_word() == 0
        assert torch.all(out[n:] == 3.0) and torch.all(lse[n:] == 3.0)
        bounded.check_attention(p, *got)


def test_a_window_of_few_units_without_a_workspace():
    p = fi.make_fia(B=2, QN=8, KVN=2, D=128, q_lens=[1, 1], kv_lens=[900, 70], block_size=64, seed=51,
                    mask_mode=fi.MASK_BAND, pre_tokens=300, first_tokens=4, device=DEV)
    want = fia.FiaCall(p).run()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    status = torch.full((1,), 7, dtype=torch.int32, device=DEV)
    params = api.params_from_problem(p, out, lse)
    for bad in (False, True):
        if bad:
            p.seqused_kv[1] = 1 << 20
            out.fill_(3.0)
        fia.fia_decode_run_noalloc(params, status.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert int(status) == (2 if bad else 0)
        assert torch.equal(out[0], want[0][0])
        assert torch.all(out[1] == 3.0) if bad else torch.equal(out[1], want[0][1])
