"""Decoding where the list of blocks cuts the work although a window bounds what is seen, long
sequences in many pieces, more sequences than a CTA has threads, and captured calls.  The size of
the workspace (256 bytes: none) shows that the list was taken.  Tolerances: tests/decode_tol.py."""
import ctypes

import pytest
import torch

from tests.decode_tol import check, floor
from tests.test_gpu_decode import DEV, INT, _case, _want, _wide, ga  # noqa: F401

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _args(c):
    return [c["q"].to(DEV), c["k"].to(DEV).view(F8), c["v"].to(DEV).view(F8), c["ks"].to(DEV), c["vs"].to(DEV),
            c["table"].to(DEV), c["lens"].to(DEV)]


def _by_list(ga, args, window, sink):
    p, _, _, _ = ga._decode_params(*args, window, sink, None, None, None, True)
    return ga.lib().attn_decode_workspace_bytes(ctypes.byref(p)) > 256


def _hide(c, window, sink):
    """What no query sees: NaN codes in K and V on pages that stay, and the other pages given back."""
    n, sq = c["q"].shape[:2]
    size = c["k"].shape[2]
    for i in range(n):
        lo = max(0, int(c["lens"][i]) - sq - window)  # the first query's first key in the window
        for key in range(min(sink, lo), lo):
            page = int(c["table"][i, key // size])
            for x in ("k", "v"):
                c[x][page, :, key % size] = 0x7f
        c["table"][i, -(-sink // size):lo // size] = -1
    return c


WINDOWED = [
    # n, sq, hq, hkv, d, size, longest, window, sink
    # at most 16 rows, more items than CTAs on the GPU
    (80, 1, 32, 8, 64, 16, 1500, 700, 5),
    (80, 1, 16, 8, 128, 64, 1400, 777, 40),
    (80, 1, 8, 8, 256, 32, 1200, 600, 33),
    (60, 2, 64, 8, 128, 16, 1300, 650, 17),
    (60, 3, 32, 8, 64, 128, 1300, 650, 0),
    (60, 1, 96, 8, 256, 16, 1100, 530, 100),
    # 17 to 32 rows
    (40, 2, 128, 8, 64, 32, 1500, 700, 77),
    (40, 7, 32, 8, 128, 16, 1400, 650, 1),
    (40, 5, 32, 8, 256, 64, 1200, 600, 45),
    # 33 to 64 rows
    (42, 3, 64, 4, 64, 16, 1300, 700, 40),
    (42, 8, 32, 4, 128, 32, 1500, 650, 16),
    (42, 5, 44, 4, 256, 128, 1200, 600, 130),
    (42, 33, 4, 4, 128, 16, 1400, 800, 3),
    # 65 and more rows
    (16, 8, 64, 4, 64, 32, 1600, 700, 45),
    (16, 9, 56, 4, 128, 16, 1500, 900, 7),
    (16, 16, 32, 4, 128, 64, 1300, 640, 0),
    (25, 8, 64, 4, 256, 16, 1300, 600, 20),
    (8, 40, 24, 4, 128, 64, 1500, 1100, 65),
    # windows beyond what a cluster takes, few sequences
    (2, 5, 32, 2, 64, 64, 21000, 17000, 50),
    (2, 3, 32, 2, 128, 32, 10500, 8500, 20),
    (1, 9, 8, 1, 256, 64, 6000, 4300, 70),
    (1, 6, 16, 1, 128, 16, 10500, 8600, 9),
]


@pytest.mark.parametrize("n,sq,hq,hkv,d,size,longest,window,sink", WINDOWED)
def test_windows_by_the_list(ga, n, sq, hq, hkv, d, size, longest, window, sink):
    """Kept tokens, a gap whose pages are given back and whose other keys are NaN, and the window."""
    lens = [longest - (i * 337) % longest if i % 7 else longest for i in range(n)]
    lens[n // 2] = max(lens[n // 2] if n > 2 else longest - 1, 1)
    c = _hide(_case(n, sq, hq, hkv, d, size, lens, seed=d + sq + n), window, sink)
    args = _args(c)
    assert _by_list(ga, args, window, sink)
    got = ga.attn_decode(*args, window_left=window, sink_tokens=sink, scale=d ** -0.5, out_fp32=True)
    check(got, _want(c, window, sink, d ** -0.5), floor(c, window, sink))


@pytest.mark.parametrize("n,sq,hq,hkv,d", [(80, 2, 16, 8, 64), (80, 2, 64, 8, 128), (42, 4, 44, 4, 128),
                                           (42, 4, 40, 4, 64), (16, 8, 64, 4, 128), (25, 8, 64, 4, 256)])
def test_nan_at_the_window_s_edge(ga, n, sq, hq, hkv, d):
    """A NaN in V of the last key that the first query's window holds, and of the first kept token's
    neighbour, which nobody sees: the first query has it, the others do not."""
    window, sink, size = 700, 6, 16
    lens = [1100 + 13 * i for i in range(n)]
    c = _case(n, sq, hq, hkv, d, size, lens, seed=n)
    ro, rl, mag = _want(c, window, sink, 0.1)
    least = floor(c, window, sink)
    for i, m in enumerate(lens):
        edge = m - sq - window
        c["v"][int(c["table"][i, edge // size]), :, edge % size, 9] = 0x7f
        c["v"][int(c["table"][i, sink // size]), :, sink % size] = 0xff
    args = _args(c)
    assert _by_list(ga, args, window, sink)
    out, lse = ga.attn_decode(*args, window_left=window, sink_tokens=sink, scale=0.1, out_fp32=True)
    check((out[:, 1:], lse[:, :, 1:]), (ro[:, 1:], rl[:, :, 1:], mag[:, 1:]), least[:, 1:])
    assert torch.isnan(out[:, 0, :, 9]).all()
    rest = [j for j in range(d) if j != 9]
    check((out[:, :1, :, rest], lse[:, :, :1]), (ro[:, :1, :, rest], rl[:, :, :1], mag[:, :1, :, rest]),
          least[:, :1, :, rest])


@pytest.mark.parametrize("sq,g,d", [(1, 8, 128), (4, 8, 64), (10, 5, 128), (16, 8, 128), (8, 16, 256)])
def test_one_sequence_in_many_pieces(ga, sq, g, d):
    """More pieces than the fold takes at a time, the largest scores in the last ones, then in the first."""
    n = 45000
    c = _case(1, sq, g, 1, d, 64, [n], seed=d + sq)
    c = _wide(c, 64)
    ids = c["table"][0, :-(-n // 64)].long()
    held = c["ks"].clone()
    for late in (True, False):
        steps = torch.linspace(-4, 2, len(ids)).round()
        c["ks"] = held.clone()
        c["ks"][ids, 0] *= torch.exp2(steps if late else steps.flip(0))
        args = _args(c)
        assert _by_list(ga, args, -1, 0)
        check(ga.attn_decode(*args, scale=0.05, out_fp32=True), _want(c, -1, 0, 0.05), floor(c, -1, 0))


@pytest.mark.parametrize("sq,hq,hkv,d", [(1, 4, 2, 64), (2, 16, 1, 128), (5, 16, 2, 64), (9, 8, 1, 128)])
def test_more_sequences_than_threads(ga, sq, hq, hkv, d):
    """300 ragged sequences, every third (and a run of forty) empty."""
    lens = [0 if i % 3 == 0 or 100 <= i < 140 else (i * 37) % 300 + 1 for i in range(300)]
    c = _wide(_case(300, sq, hq, hkv, d, 32, lens, seed=sq), 32)
    args = _args(c)
    assert _by_list(ga, args, -1, 0)
    check(ga.attn_decode(*args, scale=0.1, out_fp32=True), _want(c, -1, 0, 0.1), floor(c, -1, 0))


@pytest.mark.parametrize("sq,hq", [(1, 16), (4, 32), (8, 64)])
def test_captured_list(ga, sq, hq):
    """The list's two launches captured into one graph, twice beside each other with a workspace each,
    and replayed with other lengths: what an eager call gives, bit for bit."""
    n, hkv, d, size = 9, 4, 128, 32
    c = _wide(_case(n, sq, hq, hkv, d, size, [900 - 90 * i for i in range(n)], seed=3), size)
    args = _args(c)
    assert _by_list(ga, args, -1, 0)
    kw = dict(scale=0.09, out_fp32=True)
    other = torch.randn(args[0].shape, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    ga.attn_decode(*args, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = ga.attn_decode(*args, **kw)
        second = ga.attn_decode(other, *args[1:], **kw)
    for lens in (c["lens"].tolist(), [1, 0, 700, 33, 5, 64, 360, 2, 180], c["lens"].tolist()):
        args[6].copy_(torch.tensor([min(a, b) for a, b in zip(lens, c["lens"].tolist())], **INT))
        graph.replay()
        for q, got in ((args[0], first), (other, second)):
            want = ga.attn_decode(q, *args[1:], **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(first, _want(c, -1, 0, 0.09), floor(c, -1, 0))


def test_lists_on_two_streams(ga):
    """Two calls at once, each with its own workspace."""
    n, hkv, d, size = 12, 2, 64, 16
    both = []
    for k, (sq, hq) in enumerate(((1, 16), (7, 16))):
        c = _wide(_case(n, sq, hq, hkv, d, size, [150 * i + 3 for i in range(n)], seed=k), size)
        both.append((_args(c), _want(c, -1, 0, 0.1), floor(c, -1, 0)))
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for s, (args, _, _) in zip(streams, both):
            with torch.cuda.stream(s):
                got.append(ga.attn_decode(*args, scale=0.1, out_fp32=True))
        torch.cuda.synchronize()
        for g, (_, want, least) in zip(got, both):
            check(g, want, least)
