"""Decoding where the scales of V lie as far apart as appended pages can bring them (2^-126 for a
page of zeros) within one tile of keys, some of them out of a query's sight or of next to no weight.
Tolerances: tests/decode_tol.py; they go by what a row sees, so one that sees only small values has
to be as near to them as any other."""
import math

import pytest
import torch

from tests.decode_tol import check, floor
from tests.test_gpu_decode import _case, _run, _want, _wide, ga  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS = [(20, 1), (20, 2), (20, 6), (40, 5)]  # query tokens, group: 20, 40, 120 and 200 rows


@pytest.mark.parametrize("sq,g", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("top", [2, 4, 100, 118])
def test_large_scale_out_of_sight(ga, sq, g, d, top):
    """The first queries see pages of V with scales 0 and 2^-126 only, while later tokens, whose
    scale is 2^top, lie in the same tile."""
    c = _case(1, sq, g, 1, d, 16, [112], seed=d + top)
    ids = c["table"][0, :7].long()
    c["vs"][ids[::2], 0] = 2.0 ** -126
    c["vs"][ids[1::2], 0] = 0.0
    c["vs"][ids[6], 0] = 2.0 ** top
    want = _want(c, -1, 0, d ** -0.5)
    check(_run(ga, _wide(c, 16), -1, 0, d ** -0.5, out_fp32=True), want, floor(c, -1, 0))


@pytest.mark.parametrize("sq,g", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lower,top,rest", [(100, 10, 0.0), (100, 27, 0.0), (158, 4, 2.0 ** -126), (158, 100, 0.0)])
def test_large_scale_of_little_weight(ga, sq, g, d, lower, top, rest):
    """The last page's keys have 2^-lower of the others' weight and a scale of V of 2^top; the
    others' is `rest`.  A weight below 2^-126 is zero in 32 bits: at most the page's 16 keys times
    2^(top - lower) times their code, 448, is then left out."""
    c = _case(1, sq, g, 1, d, 16, [112], seed=d)
    ids = c["table"][0, :7].long()
    c["q"].fill_(1.0)
    c["ks"][ids] = 1.0
    c["k"][ids] = 0
    c["k"][ids[6]] = 0xb8  # -1
    c["vs"][ids] = rest
    c["vs"][ids[6]] = 2.0 ** top
    scale = lower * math.log(2.0) / d
    want = _want(c, -1, 0, scale)
    # (weights that are next to nothing: P * v_scale goes by the page's own, not by its scale)
    least = floor(dict(c, vs=torch.clamp(c["vs"], max=2.0 ** (top - lower))), -1, 0)
    if lower > 126:
        least = least + 16 * 448 * 2.0 ** (top - lower)
    check(_run(ga, _wide(c, 16), -1, 0, scale, out_fp32=True), want, least)
