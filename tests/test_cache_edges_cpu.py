"""Edges of the attention and bounded-cache calls that need no GPU: what they take
and refuse, and which device they launch on."""
import contextlib
import ctypes
from types import SimpleNamespace

import pytest
import torch

import decode_tile_scheduler_gb300 as fia
from decode_tile_scheduler_gb300 import _abi, api
from tests.test_bounded_cache_cpu import FAKE, _append, _evict, _fia_params, _weights_status


# ----------------------------------------------------------------------------
# tensors of no rows have no address
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [dict(seqlen_q=0), dict(layout=1, total_q=0, cu_seqlens_q=FAKE)])
def test_append_of_no_rows_takes_no_address(rows):
    assert _append(k_new=0, v_new=0, **rows) == fia.FIA_OK
    assert _append(k_new=0, v_new=0, seqused_kv=0, **rows) == fia.FIA_ERR_NULL_ARG
    assert _append(k_new=0) == _append(v_new=0) == fia.FIA_ERR_NULL_ARG


@pytest.mark.parametrize("rows", [dict(max_seqlen_q=0),
                                  dict(layout=1, total_q=0, cu_seqlens_q=FAKE)])
def test_attention_of_no_rows_takes_no_address(rows):
    n = ctypes.c_size_t(0)
    p = _fia_params(q=0, out=0, lse=0, **rows)
    assert fia.lib().fia_get_workspace_size(ctypes.byref(p), ctypes.byref(n)) == fia.FIA_OK
    assert _weights_status(p)[0] == fia.FIA_OK
    for name in ("q", "out"):
        p = _fia_params(**{name: 0})
        assert fia.lib().fia_get_workspace_size(ctypes.byref(p), ctypes.byref(n)) == \
            fia.FIA_ERR_NULL_ARG
    p = _fia_params(k_cache=0, **rows)
    assert fia.lib().fia_get_workspace_size(ctypes.byref(p), ctypes.byref(n)) == fia.FIA_ERR_NULL_ARG


# ----------------------------------------------------------------------------
# the device that a call launches on (stand-ins for a second GPU)
# ----------------------------------------------------------------------------

OTHER = torch.device("cuda", 1)


class _Tensor:
    """What the calls ask of a tensor on the other device."""
    device, is_cuda, shape = OTHER, True, (4, 8, 128)

    def data_ptr(self):
        return FAKE

    def is_contiguous(self):
        return True

    def numel(self):
        return 1 << 20


@pytest.fixture
def launches(monkeypatch):
    """Every C call as (name, current device, stream handle), device 0 current."""
    seen, current = [], [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    monkeypatch.setattr(api, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "_current_stream", lambda index: 1000 + index)
    for name in ("fia_plan", "fia_execute", "fia_run", "fia_execute_weights", "fia_run_weights",
                 "fia_kv_append", "fia_kv_evict", "sparse_attn_metadata", "sparse_attn_run",
                 "fia_lse_combine", "fia_get_plan_layout"):
        monkeypatch.setattr(_abi, name, lambda *a, name=name: seen.append(
            (name, current[0], a[-1] if name != "fia_get_plan_layout" else None)) or 0)
    yield seen
    assert current[0] == 0


def _call(kind, **attrs):
    c = object.__new__(kind)
    for k, v in dict(device=OTHER, params=None, weights_params=None, ws=_Tensor(), ws_bytes=0,
                     out=_Tensor(), lse=None, metadata=_Tensor(), weights_out=None,
                     seqused_out=None, positions_out=None,
                     cache=SimpleNamespace(device=OTHER), **attrs).items():
        setattr(c, k, v)
    return c


CALLS = [(fia.KvAppendCall, "run"), (fia.KvEvictCall, "run"), (fia.KeyWeightsCall, "run"),
         (fia.KeyWeightsCall, "execute"), (fia.KeyWeightsCall, "plan"), (fia.FiaCall, "run"),
         (fia.FiaCall, "execute"), (fia.FiaCall, "plan"), (fia.SparseCall, "plan"),
         (fia.SparseCall, "run")]


@pytest.mark.parametrize("kind,method", CALLS)
def test_calls_launch_on_their_tensors_device(kind, method, launches):
    getattr(_call(kind), method)()
    assert launches and all(x[1:] == (1, 1001) for x in launches)
    del launches[:]
    getattr(_call(kind), method)(77)
    assert all(x[1:] == (1, 77) for x in launches)
    del launches[:]
    for own in (OTHER, 1, None):  # (another library's stream names its device in its own way)
        getattr(_call(kind), method)(SimpleNamespace(device=own, cuda_stream=78))
        assert launches and all(x[1:] == (1, 78) for x in launches)
    del launches[:]
    for cuda_stream in (0, 5):
        with pytest.raises(ValueError, match="cuda:0"):
            getattr(_call(kind), method)(SimpleNamespace(device=torch.device("cuda", 0),
                                                         cuda_stream=cuda_stream))
    assert not launches


def test_combine_and_plan_layout_on_their_tensors_device(launches):
    t = _Tensor()
    fia.lse_combine([t], [t], layout=fia.LAYOUT_TND, num_heads=8, total_q=4, out=t, lse=t)
    _call(fia.FiaCall).plan_layout()
    assert launches == [("fia_lse_combine", 1, 1001), ("fia_get_plan_layout", 1, None)]


def test_a_problem_on_two_devices_is_refused():
    t, far = _Tensor(), _Tensor()
    far.device = torch.device("cuda", 0)
    names = ("out", "k_cache", "v_cache", "lse", "block_table", "seqused_kv", "sinks")
    for name in names:
        kw = dict.fromkeys(names, t)
        kw[name] = far
        with pytest.raises(ValueError, match=name):
            api.make_fia_params(q=t, num_q_heads=8, num_kv_heads=2, head_dim=128, batch=4,
                                layout=fia.LAYOUT_BSND, max_seqlen_q=1, **kw)


# ----------------------------------------------------------------------------
# state that overlaps
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("shift,refused", [(0, False), (4, True), (-4, True), (1020 * 4, True),
                                           (1024 * 4, False), (2000 * 4, True), (2048 * 4, True),
                                           (1024 * 4 + 2048 * 4, False), (7 * 2048 * 4, True),
                                           (8 * 2048 * 4, False), (-(7 * 2048 * 4 + 4092), True),
                                           (-(7 * 2048 * 4 + 4096), False)])
def test_state_rows_that_overlap_are_refused(shift, refused):
    """Eight rows of 1024 slots, 2048 apart, against the same rows `shift` bytes on.
    Rows between each other's, and the same tensor, are fine."""
    far = 1 << 20
    want = fia.FIA_ERR_BAD_SHAPE if refused else fia.FIA_OK
    assert _evict(state_stride=2048, weights_in=far, weights_out=far + shift)[0] == want
    assert _evict(state_stride=2048, weights_in=far, weights_out=1 << 24, positions_in=far,
                  positions_out=far + shift)[0] == want
    assert _weights_status(_fia_params(), state_stride=2048, weights_in=far,
                           weights_out=far + shift)[0] == want


def test_lengths_that_overlap_are_refused():
    for shift in (4, 12, -4, -12):
        assert _evict(seqused_kv=FAKE, seqused_out=FAKE + shift)[0] == fia.FIA_ERR_BAD_SHAPE
    for shift in (16, -16):
        assert _evict(seqused_kv=FAKE, seqused_out=FAKE + shift)[0] == fia.FIA_OK


# ----------------------------------------------------------------------------
# outputs that a caller brings
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("layout", [fia.LAYOUT_BSND, fia.LAYOUT_TND])
def test_outputs_of_another_size_or_type_are_refused(layout):
    B, S, N, D = 3, 2, 4, 64
    q = torch.zeros((B * S, N, D) if layout else (B, S, N, D), dtype=torch.bfloat16)
    prob = SimpleNamespace(q=q, layout=layout, T=B * S, B=B, QN=N, S_q=S)
    shape = (B * S, N, 1) if layout else (B, N, S, 1)
    out, lse = api._outputs(prob, None, None, True)
    assert out.shape == q.shape and out.dtype == q.dtype and tuple(lse.shape) == shape
    assert api._outputs(prob, None, None, False)[1] is None
    mine = torch.empty_like(q), torch.empty(shape)
    assert all(x is y for x, y in zip(api._outputs(prob, *mine, True), mine))
    api._outputs(prob, None, torch.empty(shape[:-1]), False)  # (without the last 1)
    for out, lse in [(q[:1], None), (q.float(), None), (None, torch.empty(shape[1:])),
                     (None, torch.empty(shape).double()), (None, torch.empty(*shape, 2)[..., 0])]:
        for with_lse in (False, True):
            with pytest.raises(ValueError):
                api._outputs(prob, out, lse, with_lse)
