"""Bounded waits of the shared keys' kernel of many rows: with the copies withheld they run out, every result of a
sequence with shared keys is NaN, and the next call is right."""
import ctypes

import pytest
import torch

from tests.test_gpu_decode_shared import DEV, _args, _case, _check, _run, _want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


@pytest.mark.parametrize("m,d", [(12, 64), (12, 128), (12, 256), (40, 64), (40, 128), (40, 256), (80, 128)])
def test_timeout(ga, m, d):
    c = _case([m], [9], [1, 40, 9], 1, 4, 1, d, 32, seed=m)
    c["lens"][3] = 0
    args, shared, start = _args(c), c["shared"].to(DEV), c["start"].to(DEV)
    out, lse = (torch.zeros(m, 1, 4, d, device=DEV), torch.zeros(m, 4, 1, device=DEV))
    base, index, _, _ = ga._decode_params(*args, -1, 0, None, out, lse, True)
    p = ga._shared_params(base, index, m, shared, start, m)
    ref = ctypes.byref(p)
    ws = torch.empty(ga.lib().attn_decode_shared_workspace_bytes(ref), dtype=torch.uint8, device=DEV)
    p.base.workspace, p.base.workspace_bytes = ws.data_ptr(), ws.nbytes
    assert ga.lib().attn_decode_shared_test_timeout(ref, ga._stream(index)) == 0
    torch.cuda.synchronize()
    empty = torch.zeros(m, dtype=torch.bool, device=DEV)
    empty[3] = True
    assert torch.isnan(out[~empty]).all() and torch.isnan(lse[~empty]).all()
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    _check(_run(ga, c, -1, 0, out_fp32=True), _want(c, -1, 0), False)


def test_no_such_waits_with_few_rows(ga):
    c = _case([3], [9], [1, 40, 9], 1, 4, 1, 64, 32, seed=1)
    args = _args(c)
    base, index, out, lse = ga._decode_params(*args, -1, 0, None, None, None, True)
    p = ga._shared_params(base, index, 3, c["shared"].to(DEV), None, 3)
    ref = ctypes.byref(p)
    ws = torch.empty(ga.lib().attn_decode_shared_workspace_bytes(ref), dtype=torch.uint8, device=DEV)
    p.base.workspace, p.base.workspace_bytes = ws.data_ptr(), ws.nbytes
    assert ga.lib().attn_decode_shared_test_timeout(ref, ga._stream(index)) == ga.ATTN_ERR_UNSUPPORTED
