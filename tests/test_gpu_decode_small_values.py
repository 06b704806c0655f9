"""Decoding of V that is small everywhere: scales down to 2^-126, the least that the append writes,
and below (the cache may hold any finite scale).  Tolerances: tests/decode_tol.py."""
import pytest
import torch

from tests.decode_tol import check, floor
from tests.test_gpu_decode import _case, _run, _want, _wide, ga  # noqa: F401

pytestmark = pytest.mark.gpu

# query tokens, group: up to 8, 16 and 32 rows; 40, 64, 120 and 200 rows
ROWS = [(1, 4), (4, 2), (3, 5), (2, 16), (20, 2), (8, 8), (20, 6), (40, 5)]


@pytest.mark.parametrize("sq,g", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("low", [-112, -119, -126, -133])
@pytest.mark.parametrize("wide", [False, True])
def test_small_values(ga, sq, g, d, low, wide):
    c = _case(2, sq, g, 1, d, 16, [112, 333], seed=d - low)
    c["vs"] = torch.where(torch.isnan(c["vs"]), c["vs"], torch.full_like(c["vs"], 2.0 ** low))
    want = _want(c, -1, 0, d ** -0.5)
    check(_run(ga, _wide(c, 16) if wide else c, -1, 0, d ** -0.5, out_fp32=True), want, floor(c, -1, 0))
