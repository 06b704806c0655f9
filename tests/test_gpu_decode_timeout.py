"""The bounded waits of the decode kernel of many rows, without a GPU fault: the test hook withholds
all copies of the cache, so the waits run out (a second), and every result is NaN."""
import ctypes

import pytest
import torch

from tests.test_gpu_decode import DEV, _case, _check, _want, _wide, ga  # noqa: F401

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _hook(ga, args, out_fp32, fill):
    """The hook's status and the results it leaves in tensors that were full of `fill`."""
    q = args[0]
    out = torch.full(q.shape, fill, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=DEV)
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), fill, device=DEV)
    p, _, _, _ = ga._decode_params(*args, -1, 0, 0.1, out, lse, out_fp32)
    ws = torch.empty(ga.lib().attn_decode_workspace_bytes(ctypes.byref(p)), dtype=torch.uint8, device=DEV)
    p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
    rc = ga.lib().attn_decode_test_timeout(ctypes.byref(p), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    return rc, out, lse


def _args(c):
    return [c["q"].to(DEV), c["k"].to(DEV).view(F8), c["v"].to(DEV).view(F8), c["ks"].to(DEV), c["vs"].to(DEV),
            c["table"].to(DEV), c["lens"].to(DEV)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sq,g", [(5, 8), (10, 12)])  # 64 and 128 rows a tile
def test_withheld_copies_give_nan_and_the_next_call_is_right(ga, d, sq, g):
    c = _wide(_case(4, sq, g, 1, d, 32, [900, 0, 4100, 33], seed=d), 32)
    args = _args(c)
    for out_fp32 in (True, False):
        rc, out, lse = _hook(ga, args, out_fp32, 3.0)
        assert rc == ga.ATTN_OK
        full = [0, 2, 3]
        assert torch.isnan(out[full]).all() and torch.isnan(lse[full]).all()
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()  # a sequence without keys
    _check(ga.attn_decode(*args, scale=0.1, out_fp32=True), _want(c, -1, 0, 0.1), False)


def test_kernels_without_waits_refuse_the_hook(ga):
    for c in (_case(2, 1, 8, 1, 64, 16, [40, 3], seed=1), _wide(_case(2, 2, 16, 1, 64, 16, [40, 3], seed=1), 16)):
        rc, out, lse = _hook(ga, _args(c), True, 3.0)
        assert rc == ga.ATTN_ERR_UNSUPPORTED
        assert (out == 3).all() and (lse == 3).all()
