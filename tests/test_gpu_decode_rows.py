"""Decoding of many rows per kv head (query tokens times the group), which takes a kernel of
its own from 33 rows on where the list of blocks cuts the work, with 64 or 128 rows per CTA.  Tolerances as
in test_gpu_decode."""
import numpy as np
import pytest
import torch

from tests.test_gpu_decode import DEV, INT, _case, _check, _run, _want, _wide, ga  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    # n, sq, hq, hkv, d, size, lens, window, sink
    (1, 5, 16, 1, 128, 64, [5], -1, 0),               # 80 rows, as many keys as tokens
    (3, 8, 32, 2, 128, 64, [0, 1, 900], -1, 0),       # 128 rows; fewer tokens than queries
    (4, 9, 16, 2, 64, 32, [300, 5, 33, 1290], 20, 3),
    (2, 16, 8, 2, 256, 32, [700, 90], 64, 5),         # 64 rows
    (3, 7, 14, 2, 256, 128, [129, 31, 1000], -1, 0),  # 49 rows
    (2, 60, 8, 2, 128, 16, [45, 700], -1, 0),         # 240 rows: a tile and most of another
    (2, 129, 1, 1, 64, 16, [513, 130], 0, 0),         # one row more than a tile, themselves only
    (1, 100, 8, 1, 128, 128, [2000], 1000, 10 ** 6),  # kept tokens: all
    (7, 10, 16, 2, 64, 16, [i * 97 for i in range(7)], 50, 40),
    (2, 1024, 1, 1, 128, 64, [1500, 300], -1, 0),     # the most rows
    (3, 11, 6, 2, 128, 16, [11, 500, 77], -1, 0),     # 33 rows
    (4, 4, 32, 2, 64, 64, [1, 130, 64, 2000], 100, 5),  # 64 rows
    (2, 13, 8, 2, 256, 64, [700, 14], 0, 2),          # 52 rows
    (2, 50, 1, 1, 128, 32, [2, 1000], 3, 10 ** 6),    # kept tokens: all
]


@pytest.mark.parametrize("n,sq,hq,hkv,d,size,lens,window,sink", CASES)
@pytest.mark.parametrize("bf16", [False, True])
def test_many_rows(ga, n, sq, hq, hkv, d, size, lens, window, sink, bf16):
    c = _case(n, sq, hq, hkv, d, size, lens, seed=d + sq)
    got = _run(ga, _wide(c, size), window, sink, d ** -0.5, out_fp32=not bf16)
    _check(got, _want(c, window, sink, d ** -0.5), bf16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [16, 6, 12])
def test_nan_of_a_later_token_stays_there(ga, d, g):
    """A NaN in a token's V reaches the queries that see it and no others, in both row tiles."""
    sq = 10
    c = _case(2, sq, g, 1, d, 64, [200, 77], seed=4)
    ro, rl, mag = _want(c, -1, 0, 0.1)
    at = lambda i, key: (int(c["table"][i, key // 64]), 0, key % 64)
    c["v"][at(0, 193)][5] = 0x7f   # token 3
    c["v"][at(0, 199)][d - 1] = 0xff  # token 9, rows 144 ..
    c["v"][at(1, 20)][7] = 0x7f    # all queries of the other sequence
    c["k"][at(0, 198)][3] = 0xff   # token 8
    out, lse = _run(ga, _wide(c, 64), -1, 0, 0.1, out_fp32=True)
    _check((out[:1, :3], lse[:1, :, :3]), (ro[:1, :3], rl[:1, :, :3], mag[:1, :3]), False)
    fine = [j for j in range(d) if j != 5]
    _check((out[:1, 3:8, :, fine], lse[:1, :, 3:8]), (ro[:1, 3:8, :, fine], rl[:1, :, 3:8], mag[:1, 3:8, :, fine]),
           False)
    assert torch.isnan(out[0, 3:, :, 5]).all()
    assert torch.isnan(out[0, 8:]).all() and torch.isnan(lse[0, :, 8:]).all()
    fine = [j for j in range(d) if j != 7]
    assert torch.isnan(out[1, :, :, 7]).all()
    _check((out[1:, :, :, fine], lse[1:]), (ro[1:, :, :, fine], rl[1:], mag[1:, :, :, fine]), False)


@pytest.mark.parametrize("top", [40, 110])
@pytest.mark.parametrize("g,d", [(16, 128), (8, 128), (8, 64), (8, 256)])
def test_scales_far_apart(ga, top, g, d):
    """Pages of V from 2^-top to 2^top, and of K that raise the maximum late."""
    c = _case(1, 6, g, 1, d, 16, [900], seed=5)
    n = 900 // 16 + 1
    ids = c["table"][0, :n].long()
    c["vs"][ids, 0] = torch.exp2(torch.linspace(-top, top, n).round())
    c["ks"][ids, 0] *= torch.exp2(torch.linspace(-3, 2, n).round())
    want = _want(c, -1, 0, 0.088)
    _check(_run(ga, _wide(c, 16), -1, 0, 0.088, out_fp32=True), want, False)
    c["vs"][ids, 0] = c["vs"][ids, 0].flip(0)
    c["vs"][ids[::3], 0] = 0.0
    c["ks"][ids[1::4], 0] = 0.0
    want = _want(c, 300, 2, 0.088)
    _check(_run(ga, _wide(c, 16), 300, 2, 0.088, out_fp32=True), want, False)


def test_pages_that_are_none(ga):
    c = _case(3, 12, 8, 1, 128, 32, [300, 200, 64], seed=1)
    c["table"][0, 1], c["table"][0, 4], c["table"][0, 9] = -1, 1 << 30, -(1 << 31)
    c["table"][2, :] = 10 ** 6
    want = _want(c, -1, 0, 0.125)
    _check(_run(ga, _wide(c, 32), -1, 0, 0.125, out_fp32=True), want, False)


def test_large_and_small_queries(ga):
    c = _case(1, 5, 16, 1, 64, 16, [100], seed=6)
    c["q"][:, 1] = 0
    for e, scale in ((60, 2.0 ** -63), (-120, 2.0 ** 57)):
        c["q"] *= 2.0 ** e
        _check(_run(ga, _wide(c, 16), -1, 0, scale, out_fp32=True), _want(c, -1, 0, scale), False)


def test_strided_pages_beside_other_work(ga):
    """K and V as halves of one pool; the kernel beside an attention on another stream, which
    holds tensor memory too.  Both results are what they are alone."""
    import workload
    c = _case(9, 8, 32, 2, 128, 32, [100 * i + 7 for i in range(9)], seed=9)
    pool = torch.stack([c["k"], c["v"]], 1).to(DEV).contiguous().view(torch.float8_e4m3fn)
    w = _wide(c, 32)
    args = [c["q"].to(DEV), pool[:, 0], pool[:, 1], c["ks"].to(DEV), c["vs"].to(DEV), w["table"].to(DEV),
            c["lens"].to(DEV)]
    ref = ga.attn_decode(*args, scale=0.09, out_fp32=True)
    _check(ref, _want(c, -1, 0, 0.09), False)
    q, k, v = workload.qkv(1, 2048, 8, 2, 128, seed=3, device=DEV)
    ids, pos = ga.segments_from_seqlens(torch.tensor([[2048]], **INT), 2048)
    alone, _ = ga.attn_fwd(q, k, v, ids, pos)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            there, _ = ga.attn_fwd(q, k, v, ids, pos)
        here = ga.attn_decode(*args, scale=0.09, out_fp32=True)
        torch.cuda.synchronize()
        assert torch.equal(there, alone) and torch.equal(here[0], ref[0]) and torch.equal(here[1], ref[1])


def test_offsets_past_32_bits(ga):
    """Pages whose bytes lie beyond 4 GB of the cache, and lengths behind the table."""
    size, hkv, d, pages = 128, 8, 128, 36000  # of 128 KB
    c = _case(2, 9, 64, hkv, d, size, [500, 130], seed=8)
    k = torch.empty(pages, hkv, size, d, dtype=torch.uint8, device=DEV)
    v = torch.empty(pages, hkv, size, d, dtype=torch.uint8, device=DEV)
    ks = torch.empty(pages, hkv, device=DEV)
    vs = torch.empty(pages, hkv, device=DEV)
    at = torch.tensor([pages - 1 - 100 * i for i in range(c["k"].shape[0])])
    for big, small in ((k, c["k"]), (v, c["v"]), (ks, c["ks"]), (vs, c["vs"])):
        big[at.to(DEV)] = small.to(DEV)
    want = _want(c, -1, 0, 0.09)
    table = torch.where(c["table"] >= 0, at[c["table"].clamp_min(0).long()].int(), c["table"])
    table = _wide(dict(table=table), size)["table"]
    f8 = torch.float8_e4m3fn
    got = ga.attn_decode(c["q"].to(DEV), k.view(f8), v.view(f8), ks, vs, table.to(DEV), c["lens"].to(DEV),
                         scale=0.09, out_fp32=True)
    _check(got, want, False)


def test_length_behind_the_table(ga):
    """Positions go by the length, keys end with the table (here all of its 4096 tokens hold)."""
    c = _case(2, 9, 8, 1, 64, 16, [4096, 4096], seed=3)
    c["table"] = c["table"][:, :256].contiguous()
    c["lens"] = torch.tensor([4100, 2 ** 31 - 1], dtype=torch.int32)
    for window, sink in ((-1, 0), (50, 3), (2 ** 31 - 1, 1)):
        _check(_run(ga, c, window, sink, 0.125, out_fp32=True), _want(c, window, sink, 0.125), False)


@pytest.mark.parametrize("seed", range(16))
def test_random_configurations(ga, seed):
    rng = np.random.default_rng(7000 + seed)
    d, size = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128]))
    n, sq, hkv = int(rng.integers(1, 9)), int(rng.integers(7, 25)), int(rng.integers(1, 4))
    g = int(rng.choice([9, 10, 16, 20]))
    lens = [int(m) for m in rng.integers(0, int(rng.choice([20, 200, 900])), n)]
    window = -1 if rng.random() < 0.4 else int(rng.integers(0, 200))
    sink = int(rng.choice([0, 1, 17, 40]))
    c = _case(n, sq, hkv * g, hkv, d, size, lens, seed=seed)
    if rng.random() < 0.5:
        gone = torch.from_numpy(rng.random(c["table"].shape) < 0.2)
        c["table"][gone] = int(rng.choice([-1, 1 << 20]))
    want = _want(c, window, sink, d ** -0.5)
    _check(_run(ga, _wide(c, size), window, sink, d ** -0.5, out_fp32=True), want, False)


@pytest.mark.parametrize("seed", range(16))
def test_random_configurations_of_fewer_rows(ga, seed):
    """33 to 64 rows."""
    rng = np.random.default_rng(8000 + seed)
    d, size = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128]))
    n, hkv, g = int(rng.integers(1, 9)), int(rng.integers(1, 4)), int(rng.choice([1, 2, 5, 8, 16]))
    sq = int(rng.integers(33 // g + 1, 64 // g + 1))
    lens = [int(m) for m in rng.integers(0, int(rng.choice([20, 200, 1500])), n)]
    window = -1 if rng.random() < 0.4 else int(rng.integers(0, 200))
    sink = int(rng.choice([0, 1, 17, 40]))
    c = _case(n, sq, hkv * g, hkv, d, size, lens, seed=seed)
    if rng.random() < 0.5:
        gone = torch.from_numpy(rng.random(c["table"].shape) < 0.2)
        c["table"][gone] = int(rng.choice([-1, 1 << 20]))
    want = _want(c, window, sink, d ** -0.5)
    _check(_run(ga, _wide(c, size), window, sink, d ** -0.5, out_fp32=True), want, False)
