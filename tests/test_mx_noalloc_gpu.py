"""The decode call without a workspace over MXFP4 caches."""
import ctypes

import pytest
import torch

import decode_tile_scheduler_gb300 as fia
from tests import serving

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _noalloc(p):
    """(status, call) of fia_decode_run_noalloc, its error word checked."""
    call = fia.FiaCall(p)
    word = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    st = fia.lib().fia_decode_run_noalloc(ctypes.byref(call.params), ctypes.c_void_p(word.data_ptr()),
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert int(word) == (0 if st == fia.FIA_OK else -1)
    return st, call


@pytest.mark.parametrize("B,KVN,G,rows,kv", [(1, 1, 16, 1, 700), (4, 8, 16, 1, 3000), (4, 8, 16, 1, 300),
                                             (20, 8, 16, 1, 900), (40, 4, 4, 4, 500), (32, 4, 8, 1, 2000)])
def test_calls_whose_plan_fits_with_fewer_ctas(B, KVN, G, rows, kv):
    p = serving.make_mx(B=B, QN=KVN * G, KVN=KVN, q_lens=[rows] * B, kv_lens=[kv - 7 * b for b in range(B)],
                        block_size=64, seed=91, mask_mode=3).to(DEV)
    for _ in range(2):
        st, call = _noalloc(p)
        assert st == fia.FIA_OK
        serving.check_mx(p, call.out, call.lse)


def test_a_call_of_too_many_units_is_refused():
    p = serving.make_mx(B=64, QN=64, KVN=4, q_lens=[1] * 64, kv_lens=[64] * 64, block_size=64, seed=92,
                        mask_mode=3).to(DEV)
    call = fia.FiaCall(p)
    before = call.params.num_sms
    st, call = _noalloc(p)
    assert st == fia.FIA_ERR_WORKSPACE_TOO_SMALL and call.params.num_sms == before
