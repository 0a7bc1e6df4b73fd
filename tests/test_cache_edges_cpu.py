"""Edges of the attention and bounded-cache calls that need no GPU: what they take
and refuse, and which device they launch on."""
import ctypes

import pytest

import decode_tile_scheduler_gb300 as fia
from tests.test_bounded_cache_cpu import FAKE, _append, _fia_params, _weights_status


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
