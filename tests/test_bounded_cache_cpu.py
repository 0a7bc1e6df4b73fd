"""The bounded cache's calls without a GPU: what they refuse, workspace sizes, and
the test suite's own statements of their definitions."""
import ctypes

import numpy as np
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
from decode_tile_scheduler_gb300 import _abi, api
from tests import bounded

FAKE = 0x10000  # aligned, never dereferenced by a refused call


def _cache(**kw):
    c = _abi.KvCacheParams()
    c.batch, c.num_kv_heads, c.head_dim = 4, 2, 128
    c.k_cache = c.v_cache = FAKE
    c.block_table = FAKE
    c.max_blocks_per_seq, c.block_size, c.num_blocks = 8, 128, 40
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(cache=None, **kw):
    p = _abi.AppendParams()
    p.cache = cache or _cache()
    p.layout, p.seqlen_q = fia.LAYOUT_BSND, 1
    p.k_new = p.v_new = p.seqused_kv = FAKE
    p.weights = p.positions = FAKE
    p.state_stride = 1024
    for k, v in kw.items():
        setattr(p, k, v)
    return fia.lib().fia_kv_append(ctypes.byref(p), None)


def _evict(cache=None, **kw):
    p = _abi.EvictParams()
    p.cache = cache or _cache()
    p.seqused_kv, p.seqused_out = FAKE, FAKE + 64
    p.weights_in = p.weights_out = FAKE
    p.state_stride, p.budget, p.first_tokens, p.recent_tokens = 1024, 512, 4, 100
    for k, v in kw.items():
        setattr(p, k, v)
    n = ctypes.c_size_t(0)
    return fia.lib().fia_get_evict_workspace_size(ctypes.byref(p), ctypes.byref(n)), n.value, p


BAD_CACHE = [
    (dict(batch=0), fia.FIA_ERR_BAD_SHAPE), (dict(num_kv_heads=257), fia.FIA_ERR_BAD_SHAPE),
    (dict(head_dim=96), fia.FIA_ERR_UNSUPPORTED), (dict(kv_dtype=2), fia.FIA_ERR_BAD_DTYPE),
    (dict(kv_layout=2), fia.FIA_ERR_BAD_SHAPE), (dict(k_cache=0), fia.FIA_ERR_NULL_ARG),
    (dict(v_cache=FAKE + 8), fia.FIA_ERR_BAD_SHAPE), (dict(block_size=24), fia.FIA_ERR_BAD_SHAPE),
    (dict(num_blocks=0), fia.FIA_ERR_BAD_SHAPE), (dict(kv_dtype=1), fia.FIA_ERR_NULL_ARG),
    (dict(kv_dtype=1, k_scale=FAKE, v_scale=FAKE, quant_tile=32), fia.FIA_ERR_BAD_SHAPE),
    (dict(kv_dtype=1, k_scale=FAKE, v_scale=FAKE, quant_tile=64, head_dim=64),
     fia.FIA_ERR_UNSUPPORTED),
    (dict(kv_dtype=1, k_scale=FAKE, v_scale=FAKE, quant_tile=64, block_size=16),
     fia.FIA_ERR_BAD_SHAPE),
    (dict(block_table=0, max_seqlen_kv=-1), fia.FIA_ERR_BAD_SHAPE),
    (dict(num_blocks=1 << 24, block_size=256), fia.FIA_ERR_BAD_SHAPE),
]


@pytest.mark.parametrize("fields,status", BAD_CACHE)
def test_a_bad_cache_is_refused(fields, status):
    assert _append(_cache(**fields)) == status
    assert _evict(_cache(**fields))[0] == status


@pytest.mark.parametrize("fields,status", [
    (dict(layout=2), fia.FIA_ERR_BAD_SHAPE), (dict(seqlen_q=-1), fia.FIA_ERR_BAD_SHAPE),
    (dict(layout=1, total_q=5), fia.FIA_ERR_NULL_ARG), (dict(k_new=0), fia.FIA_ERR_NULL_ARG),
    (dict(seqused_kv=0), fia.FIA_ERR_NULL_ARG), (dict(v_new=FAKE + 8), fia.FIA_ERR_BAD_SHAPE),
    (dict(k_token_stride=128), fia.FIA_ERR_BAD_SHAPE),
    (dict(v_token_stride=260), fia.FIA_ERR_BAD_SHAPE),
    (dict(state_stride=1023), fia.FIA_ERR_BAD_SHAPE), (dict(weights=FAKE + 2), fia.FIA_ERR_BAD_SHAPE),
])
def test_append_refuses(fields, status):
    assert _append(**fields) == status


def test_append_of_no_rows_is_done_without_a_launch():
    assert _append(seqlen_q=0) == fia.FIA_OK
    assert fia.lib().fia_kv_append(None, None) == fia.FIA_ERR_NULL_ARG


@pytest.mark.parametrize("fields,status", [
    (dict(budget=0), fia.FIA_ERR_BAD_SHAPE), (dict(budget=1025), fia.FIA_ERR_BAD_SHAPE),
    (dict(first_tokens=-1), fia.FIA_ERR_BAD_SHAPE), (dict(recent_tokens=509), fia.FIA_ERR_BAD_SHAPE),
    (dict(state_stride=1000), fia.FIA_ERR_BAD_SHAPE), (dict(weights_in=0), fia.FIA_ERR_NULL_ARG),
    (dict(seqused_out=FAKE), fia.FIA_ERR_BAD_SHAPE), (dict(seqused_out=0), fia.FIA_ERR_NULL_ARG),
    (dict(positions_in=FAKE), fia.FIA_ERR_NULL_ARG), (dict(weights_out=FAKE + 1), fia.FIA_ERR_BAD_SHAPE),
])
def test_evict_refuses(fields, status):
    assert _evict(**fields)[0] == status


def test_evict_workspace():
    st, n, p = _evict()
    assert st == fia.FIA_OK and n > 0
    L = fia.lib()
    assert L.fia_kv_evict(ctypes.byref(p), None, n, None) == fia.FIA_ERR_WORKSPACE_TOO_SMALL
    assert L.fia_kv_evict(ctypes.byref(p), FAKE, n - 1, None) == fia.FIA_ERR_WORKSPACE_TOO_SMALL
    p.reserved[0] = 1
    assert L.fia_kv_evict(ctypes.byref(p), FAKE, n, None) == fia.FIA_ERR_BAD_SHAPE


def _fia_params(**kw):
    p = _abi.FiaParams()
    p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim = 4, 8, 2, 128
    p.layout, p.max_seqlen_q = fia.LAYOUT_BSND, 1
    p.q = p.out = p.k_cache = p.v_cache = p.lse = FAKE
    p.block_table = p.seqused_kv = FAKE
    p.max_blocks_per_seq, p.block_size, p.num_blocks = 8, 128, 40
    p.scale, p.num_sms = 0.088, 152
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _weights_status(p, **kw):
    w = _abi.WeightsParams()
    w.weights_out, w.state_stride = FAKE, 1024
    for k, v in kw.items():
        setattr(w, k, v)
    n = ctypes.c_size_t(0)
    L = fia.lib()
    st = L.fia_get_weights_workspace_size(ctypes.byref(p), ctypes.byref(w), ctypes.byref(n))
    for f in (L.fia_execute_weights, L.fia_run_weights):
        got = f(ctypes.byref(p), ctypes.byref(w), FAKE, 16, None)
        assert got == (st if st != fia.FIA_OK else fia.FIA_ERR_WORKSPACE_TOO_SMALL)
    return st, n.value


@pytest.mark.parametrize("fields,status", [
    (dict(weights_out=0), fia.FIA_ERR_NULL_ARG), (dict(weights_out=FAKE + 2), fia.FIA_ERR_BAD_SHAPE),
    (dict(weights_in=FAKE + 1), fia.FIA_ERR_BAD_SHAPE), (dict(state_stride=1023), fia.FIA_ERR_BAD_SHAPE),
])
def test_weights_refuse(fields, status):
    assert _weights_status(_fia_params(), **fields)[0] == status


def test_weights_need_the_lse():
    assert _weights_status(_fia_params(lse=0))[0] == fia.FIA_ERR_NULL_ARG
    assert _weights_status(_fia_params(head_dim=96))[0] == fia.FIA_ERR_UNSUPPORTED
    st, n = _weights_status(_fia_params())
    m = ctypes.c_size_t(0)
    p = _fia_params()
    assert fia.lib().fia_get_workspace_size(ctypes.byref(p), ctypes.byref(m)) == fia.FIA_OK
    assert st == fia.FIA_OK and n >= m.value


@pytest.mark.parametrize("fields,status", [
    (dict(mask_mode=4, pre_tokens=10, first_tokens=4), fia.FIA_OK),
    (dict(mask_mode=4, pre_tokens=10, first_tokens=-1), fia.FIA_ERR_BAD_SHAPE),
    (dict(mask_mode=3, first_tokens=4), fia.FIA_ERR_BAD_SHAPE),
    (dict(mask_mode=0, first_tokens=1), fia.FIA_ERR_BAD_SHAPE),
    (dict(mask_mode=4, first_tokens=1 << 30), fia.FIA_OK),
])
def test_first_tokens_belong_to_the_band(fields, status):
    p, n = _fia_params(**fields), ctypes.c_size_t(0)
    assert fia.lib().fia_get_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status


def test_python_calls_check_their_tensors():
    k = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fia.KvCache(k, k)
    with pytest.raises(ValueError, match="alike"):
        fia.KvCache(k, k[:2])
    with pytest.raises(ValueError, match="bfloat16"):
        fia.KvCache(k.float(), k.float())
    with pytest.raises(ValueError, match="k_scale"):
        fia.KvCache(k.to(torch.uint8), k.to(torch.uint8))


@pytest.mark.parametrize("shape,cut", [((2, 3, 80), 80), ((2, 3, 80), 64), ((2, 1, 80), 70),
                                       ((1, 4, 80), 64), ((1, 1, 80), 64)])
def test_new_state_has_the_row_stride_of_the_old(shape, cut):
    w = torch.zeros(shape)[:, :, :cut]
    B, heads, _ = shape
    new = api._new_state(w, torch.int32, B, heads, 64, w.device)
    assert new.shape == w.shape and new.dtype == torch.int32
    if heads > 1:
        assert new.stride(1) == w.stride(1)
    if B > 1:
        assert new.stride(0) == w.stride(0)
    assert api._new_state(None, torch.float32, B, heads, 64, w.device).shape == (B, heads, 64)


def test_numbers_past_32_bits_are_refused():
    assert api._int32(-(1 << 31), "x") == -(1 << 31)
    for x in (1 << 31, (1 << 32) + 4, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="32 bits"):
            api._int32(x, "budget")


# ---- the suite's own definitions ----

def test_e4m3_of_every_code_and_border():
    codes = np.arange(256, dtype=np.uint8)
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    fine = ~np.isnan(v)
    assert np.array_equal(bounded.e4m3(v[fine]), codes[fine])
    pos = np.sort(v[fine & (codes < 128)])
    mid = (pos[1:] + pos[:-1]) / 2  # exact in fp32: ties go to the even code
    for x in (mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))):
        want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
        assert np.array_equal(bounded.e4m3(x), want.numpy())
    assert list(bounded.e4m3([np.nan, np.inf, -np.inf, 500.0])) == [0x7F, 0x7E, 0xFE, 0x7E]


def test_quantised_matches_the_cache_generator():
    import fia_inputs as fi
    x = torch.randn(40, 3, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    x[3, 1, 64:] = 0
    want, ws = fi.quantize_e4m3_per_tile(x)
    codes, scale = bounded.quantised(x)
    assert np.array_equal(codes, want.numpy()) and np.array_equal(scale, ws.numpy())


def test_keep_orders_protected_weights_and_slots():
    w = [5.0, np.nan, 3.0, 3.0, -1.0, 0.0, -0.0, 2.0]
    assert list(np.nonzero(bounded.keep_of(w, None, 8, 3, 0, 0, 8))[0]) == [0, 2, 3]
    assert list(np.nonzero(bounded.keep_of(w, None, 8, 2, 0, 0, 8))[0]) == [0, 2]
    assert list(np.nonzero(bounded.keep_of(w, None, 8, 3, 2, 0, 8))[0]) == [0, 1, 2]
    assert list(np.nonzero(bounded.keep_of(w, None, 8, 5, 0, 2, 8))[0]) == [0, 2, 3, 6, 7]
    assert list(np.nonzero(bounded.keep_of(w, None, 8, 7, 0, 0, 8))[0]) == [0, 2, 3, 4, 5, 6, 7]
    # -0 and 0 tie: the lower slot first
    assert list(np.nonzero(bounded.keep_of([-0.0, 0.0, 0.0], None, 3, 2, 0, 0, 3))[0]) == [0, 1]
