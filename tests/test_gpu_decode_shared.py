"""Decoding behind shared pages against the plain fp64 form, which knows nothing of them.

Tolerances as in test_gpu_decode: 2^-10 of sum P |v| (P and the scores round as there; the fold of partials adds
fp32 roundings of 2^-24 each), half a step of bf16 where out is bf16, 2e-4 for lse."""
import random

import numpy as np
import pytest
import torch

from tests import paged
from tests.paged import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
INT = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _case(sizes, shared, own, sq, hq, hkv, d, page, seed):
    """Groups of `sizes` sequences with `shared` pages each; `own`: tokens of each sequence behind them (negative:
    it is shorter than the shared part).  What no sequence has holds NaN codes, pages of nothing NaN scales."""
    g = torch.Generator().manual_seed(seed)
    of = [j for j, m in enumerate(sizes) for _ in range(m)]
    n = len(of)
    lens = [max(0, shared[of[i]] * page + own[i % len(own)]) for i in range(n)]
    need = [max(0, -(-m // page) - shared[of[i]]) for i, m in enumerate(lens)]
    pages = sum(shared) + sum(need) + 3
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((n, max([shared[j] for j in of] + [shared[of[i]] + m for i, m in enumerate(need)]) + 1), -1,
                       dtype=torch.int32)
    used, at, start = torch.zeros(pages, page, dtype=torch.bool), 0, [0]
    for j, m in enumerate(sizes):
        table[start[-1]:start[-1] + m, :shared[j]] = ids[at:at + shared[j]]
        if m:
            used[ids[at:at + shared[j]].long()] = True
        at += shared[j]
        start.append(start[-1] + m)
    for i, m in enumerate(need):
        table[i, shared[of[i]]:shared[of[i]] + m] = ids[at:at + m]
        for x in range(m):
            used[ids[at + x], :min(page, lens[i] - (shared[of[i]] + x) * page)] = True
        at += m
    cache = []
    for _ in range(2):
        x = torch.randn(pages, hkv, page, d, generator=g)
        x *= torch.exp2(torch.randint(-3, 4, (pages, hkv, 1, 1), generator=g).float())
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
        code = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        code[~used[:, None, :].expand(-1, hkv, -1)] = 0x7f
        scale[~used.any(1)] = float("nan")
        cache.append((code, scale))
    return dict(q=torch.randn(n, sq, hq, d, generator=g).to(torch.bfloat16), k=cache[0][0], ks=cache[0][1], v=cache[1][0],
                vs=cache[1][1], table=table, lens=torch.tensor(lens, dtype=torch.int32),
                shared=torch.tensor([shared[j] for j in of], dtype=torch.int32), start=torch.tensor(start, dtype=torch.int32),
                most=max(sizes))


def _args(c, wide=True):
    """The call's tensors; `wide`: with a page table for 256k tokens, by whose width the call takes the shared keys'
    kernels (small problems are attn_decode's)."""
    if wide:
        n, per = c["table"].shape
        more = torch.full((n, (1 << 18) // c["k"].shape[2] - per), -1, dtype=torch.int32)
        c = dict(c, table=torch.cat([c["table"], more], 1))
    return [c["q"].to(DEV), c["k"].to(DEV).view(torch.float8_e4m3fn), c["v"].to(DEV).view(torch.float8_e4m3fn),
            c["ks"].to(DEV), c["vs"].to(DEV), c["table"].to(DEV), c["lens"].to(DEV)]


def _run(ga, c, window, sink, wide=True, **kw):
    kw.setdefault("max_group", c["most"])
    return ga.attn_decode_shared(*_args(c, wide), c["shared"].to(DEV), c["start"].to(DEV), window_left=window, sink_tokens=sink,
                                 **kw)


def _want(c, window, sink):
    return paged.decode(np64(c["q"]), paged.raw(c["k"]), paged.raw(c["v"]), c["ks"].numpy(), c["vs"].numpy(),
                        c["table"].numpy(), c["lens"].numpy(), window, sink, c["q"].shape[3] ** -0.5)


def _check(got, want, bf16):
    (out, lse), (ro, rl, mag) = got, want
    out, lse = np64(out), np64(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(lse[fin] - rl[fin]) <= 2e-4)
    assert np.all(np.abs(out - ro) <= 2.0 ** -10 * mag + (2.0 ** -8 * np.abs(ro) if bf16 else 0))
    assert np.all(out[np.swapaxes(~fin, 1, 2)] == 0)


CASES = [
    # group sizes, shared pages, own tokens, sq, hq, hkv, d, page, window, sink
    ([2], [1], [1, 2], 1, 1, 1, 64, 16, -1, 0),                        # up to 8 rows
    ([4], [5], [7, 1, 90, 33], 1, 2, 1, 128, 64, -1, 0),
    ([3], [4], [5, 40, 300], 1, 8, 2, 256, 32, -1, 0),                 # 12 rows, the kernel of 16
    ([6], [9], [1, 70, 12], 1, 8, 2, 64, 16, -1, 0),                   # 24 rows, of 32
    ([5], [3], [1, 130, 77], 1, 16, 2, 128, 128, -1, 0),               # 40 rows, of 64
    ([7], [6], [10, 3, 200], 1, 8, 1, 256, 64, -1, 0),                 # 56 rows
    ([25], [8], [1, 17, 64, 150], 1, 4, 1, 128, 64, -1, 0),            # 100 rows, of 128
    ([70], [5], [1, 40, 2, 99, 64], 1, 4, 1, 64, 32, -1, 0),           # three tiles of 128, the last partly full
    ([33], [7], [1, 31, 200], 1, 8, 1, 128, 16, -1, 0),
    ([40], [3], [9, 100], 1, 4, 1, 256, 32, -1, 0),
    ([3, 1, 6], [4, 2, 9], [1, 20, 50], 1, 4, 2, 128, 16, -1, 0),      # groups of unlike sizes
    ([0, 5, 0, 2, 0], [3, 4, 2, 1, 7], [30, 1], 1, 4, 1, 64, 16, -1, 0),  # empty ones
    ([4, 3], [0, 3], [30, 1, 200], 1, 4, 2, 64, 32, -1, 0),            # nothing shared
    ([4], [6], [0, -1, 60, -90, -10000], 1, 4, 1, 64, 32, -1, 0),      # sequences that end with or inside the shared part
    ([3, 2], [4, 3], [-10000], 1, 4, 1, 64, 16, -1, 0),                # empty slots only
    ([5], [4], [3, 50, 1, 2, 8], 4, 4, 2, 128, 64, -1, 0),             # drafted tokens
    ([5, 2], [4, 5], [-125, 50, -64, 2, -200], 3, 4, 2, 64, 32, -1, 0),  # ... before the first position
    ([9], [5], [1, 100, 30], 5, 4, 1, 128, 32, -1, 0),                 # 180 rows
    ([6], [12], [1, 60, 200, 3], 1, 4, 2, 128, 16, 100, 0),            # windows: over part of the shared keys, or none
    ([6], [12], [1, 60, 200, 3], 1, 4, 2, 128, 16, 100, 5),
    ([6, 4], [12, 6], [1, 60, -30, 3], 2, 4, 2, 64, 16, 40, 37),
    ([40], [6], [1, 60, 200, 3, -70, -10000], 1, 4, 1, 128, 32, 90, 50),
    ([40], [6], [1, 60, 200, 3], 2, 4, 1, 64, 32, 0, 1),               # itself and the first token
    ([20], [4], [1, 60, 200, 3], 1, 8, 1, 256, 32, 33, 200),           # kept tokens past the shared ones
    ([20], [4], [1, 60, 200, 3], 1, 8, 1, 128, 32, 3, 10 ** 6),
]


@pytest.mark.parametrize("case", CASES)
def test_decode_shared(ga, case):
    *shape, window, sink = case
    c = _case(*shape, seed=len(shape[2]) + shape[6])
    want = _want(c, window, sink)
    _check(_run(ga, c, window, sink), want, True)
    _check(_run(ga, c, window, sink, out_fp32=True), want, False)
    # a bound above (other kernels) and below the groups' sizes, and the plain call
    _check(_run(ga, c, window, sink, out_fp32=True, max_group=len(c["lens"])), want, False)
    _check(_run(ga, c, window, sink, out_fp32=True, max_group=min(2, len(c["lens"]))), want, False)
    _check(_run(ga, c, window, sink, out_fp32=True, max_group=1), want, False)
    _check(_run(ga, c, window, sink, wide=False), want, True)


def test_one_group_without_an_array(ga):
    c = _case([5], [3], [9, 30, 1], 1, 4, 2, 64, 32, seed=1)
    want = _want(c, -1, 0)
    got = ga.attn_decode_shared(*_args(c), c["shared"].to(DEV), out_fp32=True)
    _check(got, want, False)


@pytest.mark.parametrize("d,rows", [(64, 4), (128, 4), (128, 12), (128, 24), (128, 48), (128, 200), (256, 12), (256, 130)])
def test_many_pieces(ga, d, rows):
    """A long shared part whose items are cut into as many pieces as there are CTAs, own parts of one page to many."""
    c = _case([rows], [400], [1, 30, 700, 2000] if rows < 50 else [1, 30, 90], 1, 1, 1, d, 32, seed=rows)
    want = _want(c, -1, 0)
    got = _run(ga, c, -1, 0, out_fp32=True)
    _check(got, want, False)
    again = _run(ga, c, -1, 0, out_fp32=True)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_many_groups(ga):
    """More groups and sequences than a CTA's threads sum up at once."""
    sizes = [1 + (7 * j) % 3 for j in range(300)]
    c = _case(sizes, [j % 4 for j in range(300)], [1, 9, 30, -3, 17], 1, 2, 1, 64, 16, seed=5)
    _check(_run(ga, c, -1, 0), _want(c, -1, 0), True)
    _check(_run(ga, c, 20, 3), _want(c, 20, 3), True)


@pytest.mark.parametrize("hq,m", [(2, 3), (8, 3), (4, 30)])
def test_nan_of_v_reaches_who_sees_it(ga, hq, m):
    """A NaN of V among the shared keys: rows whose window (or end) leaves it out have no trace of it."""
    c = _case([m], [6], [1, 40, 100, -20], 1, hq, 1, 128, 32, seed=3)
    table = c["table"].numpy()
    for key, d0 in ((5, 3), (150, 7), (170, 100), (190, 7)):
        c["v"][table[0, key // 32], 0, key % 32, d0] = 0x7f
    for window, sink in ((-1, 0), (60, 0), (60, 6)):
        ro, rl, mag = _want(c, window, sink)
        out, lse = _run(ga, c, window, sink, out_fp32=True)
        out = np64(out)
        assert np.array_equal(np.isnan(out), np.isnan(ro)) and np.isnan(ro).any()
        ok = ~np.isnan(ro)
        assert not ok.all() and np.all(np.abs(out - ro)[ok] <= 2.0 ** -10 * mag[ok])


@pytest.mark.parametrize("m", [3, 40])
def test_nan_of_a_query_stays_in_its_row(ga, m):
    c = _case([m], [6], [1, 40, 100], 1, 4, 1, 128, 32, seed=3)
    want = _want(c, -1, 0)
    c["q"][1, 0, 2, 5] = float("nan")
    out, lse = _run(ga, c, -1, 0, out_fp32=True)
    assert torch.isnan(out[1, 0, 2]).all() and torch.isnan(lse[1, 2, 0])
    out[1, 0, 2], lse[1, 2, 0] = torch.from_numpy(want[0][1, 0, 2]).float().to(DEV), float(want[1][1, 2, 0])
    _check((out, lse), want, False)


@pytest.mark.parametrize("rows", [4, 16, 60])
def test_one_key_outweighs_the_others(ga, rows):
    """Scores far apart: partials of the two parts and of pieces fold without loss.  The scores' fp32 sums are off by
    d 2^-24 of their terms' magnitudes, e; a weight then by 2 e of itself (its own score and the sum's), lse by e."""
    d = 64
    c = _case([rows], [40], [1, 40, 100], 1, 1, 1, d, 16, seed=3)
    c["q"] *= 60
    want = _want(c, -1, 0)
    k = np.abs(paged.from_e4m3(paged.raw(c["k"]))) * c["ks"].numpy()[:, :, None, None]
    e = d * 2.0 ** -24 * d ** -0.5 * (np.abs(np64(c["q"]))[:, 0, 0] @ np.nan_to_num(k).reshape(-1, d).T).max()
    assert e < 0.1
    out, lse = _run(ga, c, -1, 0, out_fp32=True)
    assert np.all(np.abs(np64(lse) - want[1]) <= 2e-4 + e)
    assert np.all(np.abs(np64(out) - want[0]) <= (2.0 ** -10 + 2 * e + 2 * e * e) * want[2])


@pytest.mark.parametrize("seed", range(24))
def test_random(ga, seed):
    r = random.Random(seed)
    d, page, hkv = r.choice([64, 128, 256]), r.choice([16, 32, 64, 128]), r.choice([1, 2, 3])
    sizes = [r.randrange(0, r.choice([3, 9, 40])) for _ in range(r.randrange(1, 5))]
    sizes[r.randrange(len(sizes))] += 2
    shared = [r.randrange(0, 1 + r.choice([2, 400]) // page + 1) for _ in sizes]
    own = [r.randrange(-60, r.choice([2, 90, 400])) for _ in range(7)]
    sq, g = r.choice([1, 1, 2, 5]), r.choice([1, 2, 3, 8])
    window = -1 if r.random() < 0.5 else r.randrange(0, 500)
    sink = r.choice([0, 1, 70])
    c = _case(sizes, shared, own, sq, hkv * g, hkv, d, page, seed)
    _check(_run(ga, c, window, sink, out_fp32=True), _want(c, window, sink), False)


def test_streams_workspaces_and_graphs(ga):
    c = _case([20, 3], [10, 4], [1, 60, 30], 1, 8, 2, 128, 32, seed=2)
    args, shared, start = _args(c), c["shared"].to(DEV), c["start"].to(DEV)
    want = ga.attn_decode_shared(*args, shared, start, max_group=20)
    need = ga.workspace_bytes_decode_shared(*args, shared, start, max_group=20)
    assert need > 256
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    with pytest.raises(ga.AttnError):
        ga.attn_decode_shared(*args, shared, start, max_group=20, workspace=ws[:need - 256])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ga.attn_decode_shared(*args, shared, start, max_group=20, workspace=ws, out=out, lse=lse)
    args[6].add_(-1)
    graph.replay()
    other = ga.attn_decode_shared(*args, shared, start, max_group=20)
    assert torch.equal(out, other[0]) and torch.equal(lse, other[1])
    args[6].add_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for s in (side, torch.cuda.current_stream()):  # two at once, a workspace each
        with torch.cuda.stream(s):
            got.append([ga.attn_decode_shared(*args, shared, start, max_group=20) for _ in range(5)])
    torch.cuda.synchronize()
    for o, l in got[0] + got[1]:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_pages_past_32_bits(ga):
    """Pages far apart in one buffer, so that offsets pass 2^32."""
    c = _case([12], [5], [1, 60, 30], 1, 4, 2, 128, 32, seed=2)
    want = _want(c, -1, 0)
    pages, hkv, page, d = c["k"].shape
    step = (1 << 32) // (pages - 3) // 16 * 16 + hkv * page * d
    big = torch.empty(step * (pages - 1) + 2 * hkv * page * d, dtype=torch.uint8, device=DEV)
    args = _args(c)
    for i in (1, 2):
        view = torch.as_strided(big, c["k"].shape, (step, page * d, d, 1), (i - 1) * hkv * page * d)
        view.copy_(args[i].view(torch.uint8))
        args[i] = view.view(torch.float8_e4m3fn)
    for most in (12, 2):
        got = ga.attn_decode_shared(*args, c["shared"].to(DEV), c["start"].to(DEV), max_group=most, out_fp32=True)
        _check(got, want, False)


def test_groups_that_are_no_groups_touch_no_other_memory(ga):
    """Bounds out of range, decreasing, and counts beyond the table: results of sequences in proper groups stay right."""
    c = _case([3, 3, 3], [2, 3, 1], [1, 40, 9], 1, 4, 1, 64, 16, seed=4)
    want = _want(c, -1, 0)
    c["start"] = torch.tensor([0, 3, 6, 1 << 30], dtype=torch.int32)
    got = _run(ga, c, -1, 0, out_fp32=True)
    _check(got, want, False)
    c["start"] = torch.tensor([0, 3, -7, 2, 6, 5, 9, 9], dtype=torch.int32)
    _run(ga, c, -1, 0)
    c["shared"] = torch.tensor([1 << 30, -5, 7, 2, 2, 2, -(1 << 31), 0, (1 << 31) - 1], dtype=torch.int32)
    _run(ga, c, -1, 0)
    torch.cuda.synchronize()
