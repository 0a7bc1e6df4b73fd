"""The calls of a serving step without a GPU: what they refuse, and the test suite's own
statements of their definitions."""
import contextlib
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import decode_tile_scheduler_gb300 as fia
from decode_tile_scheduler_gb300 import _abi, api
from tests import serving
from tests.test_bounded_cache_cpu import FAKE, _append, _cache, _evict, _fia_params

MX = dict(kv_dtype=fia.KV_MXFP4, quant_tile=32, k_scale=FAKE, v_scale=FAKE)


def _size(p):
    n = ctypes.c_size_t(0)
    return fia.lib().fia_get_workspace_size(ctypes.byref(p), ctypes.byref(n)), n.value


BAD_MX = [
    (dict(k_scale=0), fia.FIA_ERR_NULL_ARG), (dict(v_scale=0), fia.FIA_ERR_NULL_ARG),
    (dict(quant_tile=64), fia.FIA_ERR_BAD_SHAPE), (dict(v_scale=FAKE + 8), fia.FIA_ERR_BAD_SHAPE),
    (dict(head_dim=64), fia.FIA_ERR_UNSUPPORTED), (dict(block_size=16), fia.FIA_ERR_BAD_SHAPE),
    (dict(block_size=1024), fia.FIA_ERR_BAD_SHAPE),
    (dict(block_table=0, max_seqlen_kv=1022), fia.FIA_ERR_BAD_SHAPE),
    (dict(kv_dtype=3), fia.FIA_ERR_BAD_DTYPE), (dict(kv_dtype=5), fia.FIA_ERR_BAD_DTYPE),
]


@pytest.mark.parametrize("fields,status", BAD_MX)
def test_a_bad_mxfp4_cache_is_refused(fields, status):
    kw = {**MX, **fields}
    assert _append(_cache(**kw)) == status
    assert _evict(_cache(**kw))[0] == status
    assert _rope(_cache(**kw)) == status
    for rows in (1, 40):
        assert _size(_fia_params(max_seqlen_q=rows, **kw))[0] == status


@pytest.mark.parametrize("rows", [1, 16, 40])
def test_mxfp4_workspaces(rows):
    """Decode: the slots of its plan, of three CTAs to each of num_sms; a prompt its 16-bit
    copies of K and V."""
    p = _fia_params(max_seqlen_q=rows, **MX)
    st, n = _size(p)
    st8, n8 = _size(_fia_params(max_seqlen_q=rows, kv_dtype=1, quant_tile=64, k_scale=FAKE,
                                v_scale=FAKE))
    assert st == st8 == fia.FIA_OK
    if rows <= 16:
        GH = 8 if rows * 4 <= 8 else 16
        lay = _abi.fia_get_plan_layout(p)
        assert lay.num_ctas == 3 * 152 and lay.num_units == 4 * 2 * -(-rows * 4 // GH)
        assert lay.max_chunks == 2 * lay.num_ctas + 4 * lay.num_units
        slots = lay.max_chunks * (16 + 4 * GH * (128 + 2))  # queue entries and partial sums
        assert slots <= n <= slots + 8192 and n == lay.total_bytes
    else:
        assert 4 * 4 * 1024 * 2 * 128 < n <= n8
    assert _size(_fia_params(max_seqlen_q=rows, block_table=0, max_seqlen_kv=1024, **MX))[0] == 0


# ----------------------------------------------------------------------------
# pages
# ----------------------------------------------------------------------------

def _pages(**kw):
    p = _abi.PagesParams()
    p.batch, p.block_size, p.max_blocks_per_seq, p.num_blocks = 4, 128, 8, 40
    p.layout, p.seqlen_q = fia.LAYOUT_BSND, 1
    for k, name in enumerate(("seqused_kv", "block_table", "pages_held", "pages_held_out",
                              "free_pages", "free_count", "free_count_out", "slots", "positions")):
        setattr(p, name, FAKE + 4096 * k)
    for k, v in kw.items():
        setattr(p, k, v)
    return fia.lib().fia_assign_pages(ctypes.byref(p), None)


@pytest.mark.parametrize("fields,status", [
    (dict(batch=0), 2), (dict(batch=65537), 2), (dict(block_size=0), 2), (dict(block_size=24), 2),
    (dict(block_size=2048), 2), (dict(num_blocks=0), 2), (dict(max_blocks_per_seq=0), 2),
    (dict(num_blocks=1 << 24, block_size=128), 2), (dict(max_blocks_per_seq=1 << 18), 2),
    (dict(batch=65536, max_blocks_per_seq=1 << 15), 2), (dict(layout=2), 2), (dict(seqlen_q=-1), 2),
    (dict(layout=1, total_q=5), 1), (dict(layout=1, total_q=-1, cu_seqlens_q=FAKE), 2),
    (dict(seqused_kv=0), 1), (dict(block_table=0), 1), (dict(pages_held=0), 1),
    (dict(pages_held_out=0), 1), (dict(free_pages=0), 1), (dict(free_count=0), 1),
    (dict(free_count_out=0), 1), (dict(slots=FAKE + 2), 2), (dict(status=FAKE + 1), 2),
    (dict(pages_held=FAKE, pages_held_out=FAKE + 4), 2),
    (dict(batch=65536, seqlen_q=1 << 15), 2),
])
def test_assign_pages_refuses(fields, status):
    assert _pages(**fields) == status


def test_assign_pages_refuses_reserved_words_and_null():
    p = _abi.PagesParams()
    p.reserved[3] = 1
    assert fia.lib().fia_assign_pages(ctypes.byref(p), None) == fia.FIA_ERR_BAD_SHAPE
    assert fia.lib().fia_assign_pages(None, None) == fia.FIA_ERR_NULL_ARG
    assert fia.lib().fia_norm_rope_append(None, None) == fia.FIA_ERR_NULL_ARG


def test_pages_statement():
    """A small step worked out by hand: pages of 16, a pool of 8."""
    table = np.array([[0, 1, -1], [2, 3, 4], [-1, -1, -1]])
    held, lens = [2, 3, 0], [40, 16, 17]
    got = serving.pages(table, held, [5, 6, 7, 9, 9, 9, 9, 9], 2, lens, 16, T=3)
    # sequence 1 gives 3 and 4 back behind 5, 6; sequence 0 takes 4, sequence 2 3 and 6
    assert got[0].tolist() == [[0, 1, 4], [2, 3, 4], [3, 6, -1]]
    assert got[1].tolist() == [3, 1, 2] and got[2] == [5, 6, 3, 4] and got[3] == 1
    assert got[4].tolist() == [4 * 16 + 7, 2 * 16 + 15, 6 * 16] and got[5].tolist() == [39, 15, 16]
    assert got[6] == 0
    short = serving.pages(table, held, [5] * 8, 0, [40, 48, 17], 16)
    assert short[0].tolist() == [[0, 1, -1], [2, 3, 4], [-1, -1, -1]]
    assert short[1].tolist() == [2, 3, 0] and short[6] == 3


# ----------------------------------------------------------------------------
# norms and rotation
# ----------------------------------------------------------------------------

def _rope(cache=None, **kw):
    p = _abi.NormRopeParams()
    p.cache = cache or _cache()
    p.tokens, p.num_q_heads, p.rotary_dim, p.max_positions, p.eps = 0, 8, 128, 4096, 1e-6
    for name in ("q", "k", "v", "q_out", "q_weight", "k_weight", "cos_sin", "positions", "slots"):
        setattr(p, name, FAKE)
    for k, v in kw.items():
        setattr(p, k, v)
    return fia.lib().fia_norm_rope_append(ctypes.byref(p), None)


@pytest.mark.parametrize("fields,status", [
    (dict(tokens=-1), 2), (dict(num_q_heads=257), 2), (dict(num_q_heads=-1), 2),
    (dict(rotary_dim=8), 2), (dict(rotary_dim=144), 2), (dict(rotary_dim=-16), 2),
    (dict(interleaved=2), 2), (dict(max_positions=-1), 2), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(tokens=1, k=0), 1),
    (dict(tokens=1, v=0), 1), (dict(tokens=1, q=0), 1), (dict(tokens=1, q_out=0), 1),
    (dict(tokens=1, cos_sin=0), 1), (dict(tokens=1, positions=0), 1), (dict(tokens=1, slots=0), 1),
    (dict(q=FAKE + 8), 2), (dict(q_weight=FAKE + 4), 2), (dict(cos_sin=FAKE + 8), 2),
    (dict(slots=FAKE + 2), 2), (dict(q_token_stride=1020), 2), (dict(k_token_stride=260), 2),
    (dict(v_token_stride=128), 2), (dict(q_out_token_stride=1028), 2),
    (dict(q_token_stride=2048, q_out_token_stride=1024), 2),
])
def test_norm_rope_refuses(fields, status):
    assert _rope(**fields) == status


def test_norm_rope_of_no_rows_is_done_without_a_launch():
    assert _rope() == fia.FIA_OK
    assert _rope(q=0, k=0, v=0, q_out=0, positions=0, slots=0, cos_sin=0) == fia.FIA_OK


def test_python_calls_refuse_tensors_that_do_not_fit():
    """On the CPU: every tensor is refused before its address is taken."""
    i32 = torch.int32
    table, held, free = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(9, dtype=i32)
    for kw in (dict(block_table=held), dict(free_pages=table), dict(pages_held=None),
               dict(pages_held=held.long()), dict(seqused_kv=torch.zeros(3, dtype=i32))):
        a = dict(block_table=table, pages_held=held, free_pages=free,
                 free_count=torch.zeros(1, dtype=i32), seqused_kv=held)
        a.update(kw)
        with pytest.raises(ValueError):
            fia.AssignPagesCall(**a, block_size=16)


@pytest.mark.parametrize("kind,name", [(fia.AssignPagesCall, "fia_assign_pages"),
                                       (fia.NormRopeAppendCall, "fia_norm_rope_append")])
def test_calls_launch_on_their_tensors_device(kind, name, monkeypatch):
    seen, current = [], [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    monkeypatch.setattr(api, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "_current_stream", lambda index: 1000 + index)
    monkeypatch.setattr(_abi, name, lambda params, stream: seen.append((current[0], stream)))
    call, far = object.__new__(kind), torch.device("cuda", 1)
    for k, v in dict(device=far, cache=SimpleNamespace(device=far), params=None, slots=None,
                     positions=None, q_out=None).items():
        setattr(call, k, v)
    call.run()
    call.run(77)
    assert seen == [(1, 1001), (1, 77)] and current[0] == 0
    with pytest.raises(ValueError, match="cuda:0"):
        call.run(SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=5))


def test_mxfp4_statement():
    """Codes and scales of values worked out by hand."""
    x = torch.zeros(6, 32)
    x[0, :7] = torch.tensor([6.0, -5.0, 0.25, 0.75, 1.25, 2.5, -0.2])
    x[1, :2] = torch.tensor([6.001, 3.0])
    x[2, :2] = torch.tensor([float("inf"), 1.0])
    x[3, :2] = torch.tensor([float("nan"), 1.0])
    x[4, 0] = 2.0 ** -133
    codes, scale = serving.mx_quantised(x)
    assert scale[:, 0].tolist() == [127, 128, 253, 255, 0, 127]
    assert codes[0, :4].tolist() == [7 | 14 << 4, 0 | 2 << 4, 2 | 4 << 4, 8]
    assert codes[1, 0] == 5 | 3 << 4 and codes[2, 0] == 6 and codes[3, 0] == 0
    assert codes[4, 0] == 0 and not codes[5].any()
    v = serving.mx_values(codes, scale)
    assert v[0, :7].tolist() == [6.0, -4.0, 0.0, 1.0, 1.0, 2.0, -0.0] and torch.isnan(v[3]).all()
