"""Decoding behind shared pages whose scales of V lie as far apart as a cache may hold them (2^-126 for a page of
zeros, 0, and values below): out of a row's sight, of next to no weight, or everywhere, in tiles that every row sees
as a whole and in others.  Tolerances: tests/decode_tol.py, whose floors hold for both lists (the fold weighs finished
partials in fp32, one more term of 2^-149 each)."""
import math

import pytest
import torch

from tests import paged
from tests.decode_tol import check, floor
from tests.test_gpu_decode_shared import _case, _run, _want, ga  # noqa: F401

pytestmark = pytest.mark.gpu

# sequences, query heads (one kv head): 12, 24, 40, 100 and 180 rows
ROWS = [(6, 2), (6, 4), (10, 4), (25, 4), (45, 4)]
# own tokens: sequences that end on the shared pages (112 keys, one tile of 128) and behind them; all behind
ENDS = [[-20, 1, -50, 30], [1, 30]]


def _pages(c):
    return c["table"][0, :int(c["shared"][0])].long()


@pytest.mark.parametrize("m,hq", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("top", [2, 4, 100, 118])
def test_large_scale_out_of_sight(ga, m, hq, d, top):
    """Rows whose sequences end early see scales of 0 and 2^-126 only, the others a scale of 2^top in the same tile."""
    c = _case([m], [7], ENDS[0], 1, hq, 1, d, 16, seed=d + top)
    ids = _pages(c)
    c["vs"][ids[::2], 0] = 2.0 ** -126
    c["vs"][ids[1::2], 0] = 0.0
    c["vs"][ids[6], 0] = 2.0 ** top
    check(_run(ga, c, -1, 0, out_fp32=True), _want(c, -1, 0), floor(c, -1, 0))


@pytest.mark.parametrize("m,hq", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lower,top,rest", [(100, 10, 0.0), (100, 27, 0.0), (158, 4, 2.0 ** -126), (158, 100, 0.0)])
@pytest.mark.parametrize("tiles", [1, 3])
def test_large_scale_of_little_weight(ga, m, hq, d, lower, top, rest, tiles):
    """The last shared page's keys have 2^-lower of the others' weight and a scale of V of 2^top; the others' is
    `rest`.  A weight below 2^-126 is zero in 32 bits: at most the page's 16 keys times 2^(top - lower) times their
    code, 448, is then left out."""
    shared = 8 * tiles
    c = _case([m], [shared], [1], 1, hq, 1, d, 16, seed=d)
    used = ~torch.isnan(c["ks"][:, 0])
    ids = _pages(c)
    c["q"].fill_(1.0)
    c["ks"][used] = 1.0
    c["k"][used] = torch.where(c["k"][used] == 0x7f, c["k"][used], torch.zeros_like(c["k"][used]))
    c["k"][ids[-1]] = 0xb8  # -1
    c["vs"][used] = rest
    c["vs"][ids[-1]] = 2.0 ** top
    scale = lower * math.log(2.0) / d
    want = paged.decode(paged.np64(c["q"]), paged.raw(c["k"]), paged.raw(c["v"]), c["ks"].numpy(), c["vs"].numpy(),
                        c["table"].numpy(), c["lens"].numpy(), -1, 0, scale)
    # (weights that are next to nothing: P * v_scale goes by the page's own, not by its scale)
    least = floor(dict(c, vs=torch.clamp(c["vs"], max=2.0 ** (top - lower))), -1, 0)
    if lower > 126:
        least = least + 16 * 448 * 2.0 ** (top - lower)
    check(_run(ga, c, -1, 0, out_fp32=True, scale=scale), want, least)


@pytest.mark.parametrize("m,hq", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("low", [-112, -119, -126, -133])
@pytest.mark.parametrize("ends,shared", [(ENDS[0], 7), (ENDS[1], 7), (ENDS[1], 24)])
def test_small_values(ga, m, hq, d, low, ends, shared):
    c = _case([m], [shared], ends, 1, hq, 1, d, 16, seed=d - low)
    c["vs"] = torch.where(torch.isnan(c["vs"]), c["vs"], torch.full_like(c["vs"], 2.0 ** low))
    check(_run(ga, c, -1, 0, out_fp32=True), _want(c, -1, 0), floor(c, -1, 0))


@pytest.mark.parametrize("m,hq", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("low,high", [(-126, 0), (-40, 40), (-20, 100)])
def test_scales_apart_from_tile_to_tile(ga, m, hq, d, low, high):
    """Tiles that every row sees, of small and of large V in turn: the references rise and stay."""
    c = _case([m], [40], ENDS[1], 1, hq, 1, d, 16, seed=d + high)
    ids = _pages(c)
    for x, pid in enumerate(ids):
        c["vs"][pid] = 2.0 ** (high if (x // 8) % 2 else low)
    check(_run(ga, c, -1, 0, out_fp32=True), _want(c, -1, 0), floor(c, -1, 0))
