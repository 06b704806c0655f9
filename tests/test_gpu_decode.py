"""Attention over the paged 8-bit cache against the plain fp64 form.

Tolerances.  P enters the second product as f16, off by at most 2^-11 of itself; scores
are fp32 sums of d products and differ from fp64 by at most d 2^-24 of the sum of the
products' magnitudes (under 1.5e-4 for normal q and k at d = 256, and that moves P by
the same share); together under 2^-10 of sum P |v| (fp32 outputs).  A bf16 output is off by
half a step, 2^-8 of its value, more.  lse moves with the scores: 2e-4."""
import numpy as np
import pytest
import torch

from tests import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"
INT = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _case(n, sq, hq, hkv, d, size, lens, seed, extra=3):
    """Normal values in e4m3 with a scale per page and head; unused slots and pages hold NaN codes."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-m // size) for m in lens]
    pages = sum(need) + extra
    per = max(need) + 1
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((n, per), -1, dtype=torch.int32)
    cache = []
    for _ in range(2):
        x = torch.randn(pages, hkv, size, d, generator=g)
        x *= torch.exp2(torch.randint(-3, 4, (pages, hkv, 1, 1), generator=g).float())
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
        cache.append([(x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale])
    used, at = torch.zeros(pages, size, dtype=torch.bool), 0
    for i, m in enumerate(lens):
        table[i, :need[i]] = ids[at:at + need[i]]
        for j in range(need[i]):
            used[table[i, j], :min(size, m - j * size)] = True
        at += need[i]
    for c in cache:
        c[0][~used[:, None, :].expand(-1, hkv, -1)] = 0x7f
        c[1][~used.any(1)] = float("nan")
    q = torch.randn(n, sq, hq, d, generator=g).to(torch.bfloat16)
    return dict(q=q, k=cache[0][0], ks=cache[0][1], v=cache[1][0], vs=cache[1][1], table=table,
                lens=torch.tensor(lens, dtype=torch.int32))


def _run(ga, c, window, sink, scale, **kw):
    args = [c["q"].to(DEV), c["k"].to(DEV).view(torch.float8_e4m3fn), c["v"].to(DEV).view(torch.float8_e4m3fn),
            c["ks"].to(DEV), c["vs"].to(DEV), c["table"].to(DEV), c["lens"].to(DEV)]
    return ga.attn_decode(*args, window_left=window, sink_tokens=sink, scale=scale, **kw)


def _want(c, window, sink, scale):
    return paged.decode(paged.np64(c["q"]), paged.raw(c["k"]), paged.raw(c["v"]), c["ks"].numpy(), c["vs"].numpy(),
                        c["table"].numpy(), c["lens"].numpy(), window, sink, scale)


def _check(got, want, bf16):
    (out, lse), (ro, rl, mag) = got, want
    out, lse = paged.np64(out), paged.np64(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(lse[fin] - rl[fin]) <= 2e-4)
    assert np.all(np.abs(out - ro) <= 2.0 ** -10 * mag + (2.0 ** -8 * np.abs(ro) if bf16 else 0))
    assert np.all(out[np.swapaxes(~fin, 1, 2)] == 0)


CASES = [
    # n, sq, hq, hkv, d, size, lens, window, sink
    (1, 1, 1, 1, 64, 16, [1], -1, 0),
    (3, 1, 2, 2, 128, 64, [0, 1, 64], -1, 0),
    (4, 1, 16, 1, 128, 64, [31, 32, 33, 700], -1, 0),
    (2, 1, 32, 1, 128, 32, [129, 1000], -1, 0),
    (2, 1, 15, 3, 64, 16, [17, 530], -1, 0),
    (2, 1, 8, 1, 256, 128, [127, 400], -1, 0),
    (2, 1, 24, 2, 256, 16, [5, 250], -1, 0),
    (2, 1, 64, 1, 64, 64, [65, 300], -1, 0),
    (1, 1, 40, 1, 128, 64, [333], -1, 0),          # two row tiles, the second partly empty
    (5, 1, 8, 2, 128, 64, [1, 40, 200, 641, 1500], 100, 0),
    (5, 1, 8, 2, 128, 16, [1, 40, 200, 641, 1500], 100, 5),
    (3, 1, 4, 1, 64, 32, [300, 33, 2], 0, 1),      # itself and the first token
    (3, 1, 4, 1, 64, 32, [300, 33, 2], 0, 0),
    (2, 1, 4, 2, 128, 32, [500, 130], 50, 10 ** 6),  # kept tokens: all
    (3, 4, 8, 2, 128, 64, [2, 4, 333], -1, 0),     # fewer tokens than queries
    (3, 3, 8, 2, 256, 32, [90, 1, 700], 40, 7),
    (2, 8, 16, 2, 64, 16, [3, 513], 5, 2),
    (1, 33, 2, 1, 128, 64, [100], 20, 0),          # many tokens: three row tiles
]


def _wide(c, size, keys=1 << 18):
    """The same with a table for 256k tokens: the work is then cut by the list of blocks, not
    given to a cluster of CTAs per item."""
    more = torch.full((c["table"].shape[0], keys // size - c["table"].shape[1]), -1, dtype=torch.int32)
    return dict(c, table=torch.cat([c["table"], more], 1))


@pytest.mark.parametrize("n,sq,hq,hkv,d,size,lens,window,sink", CASES)
@pytest.mark.parametrize("bf16,wide", [(False, False), (True, False), (False, True)])
def test_decode(ga, n, sq, hq, hkv, d, size, lens, window, sink, bf16, wide):
    c = _case(n, sq, hq, hkv, d, size, lens, seed=d + sq)
    got = _run(ga, _wide(c, size) if wide else c, window, sink, d ** -0.5, out_fp32=not bf16)
    _check(got, _want(c, window, sink, d ** -0.5), bf16)


@pytest.mark.parametrize("wide", [False, True])
def test_pages_that_are_none(ga, wide):
    """Entries outside the pool hide their tokens, whole sequences among them."""
    c = _case(3, 2, 4, 2, 64, 32, [300, 200, 64], seed=1)
    c["table"][0, 1], c["table"][0, 4], c["table"][0, 9] = -1, 1 << 30, -(1 << 31)
    c["table"][2, :] = 10 ** 6
    want = _want(c, -1, 0, 0.125)
    _check(_run(ga, _wide(c, 32) if wide else c, -1, 0, 0.125, out_fp32=True), want, False)


def test_pages_behind_the_window_are_not_needed(ga):
    c = _case(2, 2, 4, 2, 64, 16, [400, 333], seed=2)
    want = _want(c, 60, 20, 0.125)
    for i, n in enumerate((400, 333)):
        c["table"][i, 2:(n - 2 - 60) // 16] = -1
    _check(_run(ga, c, 60, 20, 0.125, out_fp32=True), want, False)


def test_length_behind_the_table(ga):
    """Positions go by the length, keys end with the table."""
    c = _case(2, 1, 4, 2, 64, 16, [64, 64], seed=3)
    c["lens"] = torch.tensor([100, 2 ** 31 - 1], dtype=torch.int32)
    _check(_run(ga, c, -1, 0, 0.125, out_fp32=True), _want(c, -1, 0, 0.125), False)
    _check(_run(ga, c, 50, 3, 0.125, out_fp32=True), _want(c, 50, 3, 0.125), False)


@pytest.mark.parametrize("wide", [False, True])
def test_nan_of_a_later_token_stays_there(ga, wide):
    """A NaN in a drafted token's V reaches the queries that see it and no others."""
    c = _case(1, 4, 4, 1, 128, 64, [200], seed=4)
    want = _want(c, -1, 0, 0.1)
    pid = int(c["table"][0, 198 // 64])
    c["v"][pid, 0, 198 % 64, 5] = 0x7f
    c["k"][int(c["table"][0, 199 // 64]), 0, 199 % 64, 3] = 0xff
    out, lse = _run(ga, _wide(c, 64) if wide else c, -1, 0, 0.1, out_fp32=True)
    ro, rl, mag = want
    _check((out[:, :2], lse[:, :, :2]), (ro[:, :2], rl[:, :, :2], mag[:, :2]), False)
    assert torch.isnan(out[:, 2, :, 5]).all() and not torch.isnan(out[:, 2, :, 6]).any()
    assert torch.isnan(out[:, 3]).all() and torch.isnan(lse[:, :, 3]).all()


@pytest.mark.parametrize("wide", [False, True])
def test_scales_far_apart(ga, wide):
    """Pages of V from 2^-40 to 2^40 and of K that raise the maximum late."""
    c = _case(1, 1, 8, 1, 128, 16, [600], seed=5)
    n = 600 // 16 + 1
    ids = c["table"][0, :n].long()
    c["vs"][ids, 0] = torch.exp2(torch.linspace(-40, 40, n).round())
    c["ks"][ids, 0] *= torch.exp2(torch.linspace(-3, 2, n).round())
    want = _want(c, -1, 0, 0.088)
    _check(_run(ga, _wide(c, 16) if wide else c, -1, 0, 0.088, out_fp32=True), want, False)


def test_zero_scales_and_large_queries(ga):
    c = _case(1, 1, 8, 1, 128, 16, [100], seed=6)
    ids = c["table"][0, :7].long()
    c["vs"][ids[::2], 0] = 0.0
    c["ks"][ids[1::3], 0] = 0.0
    c["q"] *= 2.0 ** 60
    _check(_run(ga, c, -1, 0, 2.0 ** -63, out_fp32=True), _want(c, -1, 0, 2.0 ** -63), False)
    c["q"] *= 2.0 ** -120
    _check(_run(ga, c, -1, 0, 2.0 ** 57, out_fp32=True), _want(c, -1, 0, 2.0 ** 57), False)


def test_partials_merge_to_the_whole(ga):
    """Two tables that hold the even and the odd pages: their merged partials are the whole."""
    c = _case(2, 1, 8, 2, 128, 32, [700, 45], seed=7)
    want = _want(c, -1, 0, 0.09)
    parts = []
    for k in (0, 1):
        half = dict(c, table=c["table"].clone())
        half["table"][:, k::2] = -1
        parts.append(_run(ga, half, -1, 0, 0.09, out_fp32=True))
    (oa, la), (ob, lb) = parts
    ga.attn_merge_partial(oa, la, ob, lb)
    _check((oa, la), want, False)


def test_offsets_past_32_bits(ga):
    """Pages whose bytes lie beyond 4 GB of the cache."""
    size, hkv, d = 128, 8, 128
    pages = 36000  # of 128 KB
    c = _case(2, 1, 16, hkv, d, size, [500, 130], seed=8)
    k = torch.empty(pages, hkv, size, d, dtype=torch.uint8, device=DEV)
    v = torch.empty(pages, hkv, size, d, dtype=torch.uint8, device=DEV)
    ks = torch.empty(pages, hkv, device=DEV)
    vs = torch.empty(pages, hkv, device=DEV)
    at = torch.tensor([pages - 1 - 100 * i for i in range(c["k"].shape[0])])
    for big, small in ((k, c["k"]), (v, c["v"]), (ks, c["ks"]), (vs, c["vs"])):
        big[at.to(DEV)] = small.to(DEV)
    want = _want(c, -1, 0, 0.09)
    table = torch.where(c["table"] >= 0, at[c["table"].clamp_min(0).long()].int(), c["table"])
    f8 = torch.float8_e4m3fn
    got = ga.attn_decode(c["q"].to(DEV), k.view(f8), v.view(f8), ks, vs, table.to(DEV), c["lens"].to(DEV),
                         scale=0.09, out_fp32=True)
    _check(got, want, False)


def test_ragged_batch_is_repeatable_on_any_stream(ga):
    c = _case(40, 1, 8, 2, 64, 16, [(i * 53) % 700 for i in range(40)], seed=9)
    first = _run(ga, c, -1, 0, 0.125, out_fp32=True)
    _check(first, _want(c, -1, 0, 0.125), False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = _run(ga, c, -1, 0, 0.125, out_fp32=True)
    side.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("n,hkv,lens_of", [(70, 8, lambda i: (i * 37) % 257), (40, 8, lambda i: (i * 131) % 513),
                                           (25, 2, lambda i: (i * 331) % 4000)])
def test_many_items(ga, n, hkv, lens_of):
    """More items than the GPU holds CTAs (one CTA each), as many (one each, or a pair), and
    few long ones (a cluster of eight)."""
    c = _case(n, 1, 4 * hkv, hkv, 64, 32, [lens_of(i) for i in range(n)], seed=n)
    _check(_run(ga, c, -1, 0, 0.125), _want(c, -1, 0, 0.125), True)


def test_captured_steps_follow_the_lengths(ga):
    """A graph of append and decode, replayed step by step with lengths on the device."""
    n, hq, hkv, d, size = 3, 8, 2, 128, 32
    g = torch.Generator().manual_seed(11)
    lens = [1, 31, 64]
    cache = [torch.zeros(12, hkv, size, d, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    cache += [torch.zeros(12, hkv, device=DEV) for _ in range(2)]
    table = torch.randperm(12, generator=g).reshape(3, 4).to(torch.int32)
    before = torch.tensor(lens, **INT)
    prompt = [torch.randn(n, 64, hkv, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    dt = table.to(DEV)
    ga.kv_cache_append(*prompt, *cache, dt, torch.zeros(n, **INT), lens=before)
    q = torch.zeros(n, 1, hq, d, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(n, 1, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    after = before + 1

    def step():
        ga.kv_cache_append(k, v, *cache, dt, before)
        got = ga.attn_decode(q, *cache, dt, after, window_left=40, sink_tokens=3, scale=0.09, out_fp32=True)
        before.add_(1)
        after.add_(1)
        return got

    held = [t.clone() for t in (*cache[:2], *cache[2:], before, after)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, h in zip((*cache, before, after), held):
        t.copy_(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for i in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = paged.decode(paged.np64(q), *(paged.raw(x) for x in cache[:2]), *(x.cpu().numpy() for x in cache[2:]),
                            table.numpy(), np.array(lens) + i + 1, 40, 3, 0.09)
        _check((out, lse), want, False)


def test_prompt_fork_and_decode_together(ga):
    """As a server uses them: attention over packed prompts with kept first tokens, their tokens
    into the cache, one sequence forked (its last page copied), then decoding steps of both."""
    import workload
    hq, hkv, d, size, window, sink = 8, 2, 128, 32, 70, 4
    lens = [150, 77]
    begin = [0, 160]
    q, k, v = workload.qkv(1, 240, hq, hkv, d, seed=3, device=DEV)
    i32 = lambda x: torch.tensor(x, **INT)
    ids, pos = ga.segments_from_seqlens(i32([lens]), 240, offsets=i32([begin]))
    kw = dict(window_left=window, sink_tokens=sink, scale=0.09)
    out, lse = ga.attn_fwd(q, k, v, ids, pos, **kw)
    cache = [torch.empty(20, hkv, size, d, dtype=torch.uint8, device=DEV).fill_(0x7f).view(torch.float8_e4m3fn)
             for _ in range(2)] + [torch.full((20, hkv), float("nan"), device=DEV) for _ in range(2)]
    table = torch.full((3, 8), -1, **INT)
    table[0, :7], table[1, :4] = torch.arange(7, **INT), torch.arange(7, 11, **INT)
    ga.kv_cache_append(k, v, *cache, table[:2], i32([0, 0]), lens=i32(lens), tok_start=i32(begin), max_new=150)
    # the prompt's last tokens through the cache: e4m3 moves q.k and v by 2^-4 of their terms at most,
    # each the other way, so the two outputs agree to a tenth of the values' size
    last = torch.stack([q[0, begin[i] + lens[i] - 1] for i in range(2)])[:, None].contiguous()
    got, _ = ga.attn_decode(last, *cache, table[:2].contiguous(), i32(lens), **kw)
    for i in range(2):
        ref = out[0, begin[i] + lens[i] - 1].float()
        assert (got[i, 0].float() - ref).norm() <= 0.1 * ref.norm()
    # fork sequence 0: full pages shared, the last one copied
    table[2, :4] = table[0, :4]
    table[2, 4] = 12
    table[2, 5] = 13
    ga.kv_cache_copy_pages(*cache, table[0, 4:5].contiguous(), table[2, 4:5].contiguous())
    n = [150, 77, 150]
    for step in range(12):
        qs, ks, vs = workload.qkv(3, 1, hq, hkv, d, seed=50 + step, device=DEV)
        ga.kv_cache_append(ks, vs, *cache, table, i32(n))
        n = [m + 1 for m in n]
        res = ga.attn_decode(qs, *cache, table, i32(n), out_fp32=True, **kw)
        want = paged.decode(paged.np64(qs), *(paged.raw(x) for x in cache[:2]), *(x.cpu().numpy() for x in cache[2:]),
                            table.cpu().numpy(), n, window, sink, 0.09)
        _check(res, want, False)


@pytest.mark.parametrize("wide", [False, True])
def test_partials_of_many_ctas_with_nan_and_empty_rows(ga, wide):
    """One long sequence over many CTAs: a NaN key reaches the row's whole result, and a
    query before the sequence's first token stays empty beside it."""
    c = _case(2, 2, 4, 1, 64, 64, [5000, 1], seed=12)
    ro, rl, mag = _want(c, -1, 0, 0.125)
    c = _wide(c, 64) if wide else c
    out, lse = _run(ga, c, -1, 0, 0.125, out_fp32=True)
    _check((out, lse), (ro, rl, mag), False)
    c["k"][int(c["table"][0, 40]), 0, 3, 7] = 0x7f
    out, lse = _run(ga, c, -1, 0, 0.125, out_fp32=True)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    _check((out[1:], lse[1:]), (ro[1:], rl[1:], mag[1:]), False)


def test_tensors_in_place_of_allocations(ga):
    c = _case(3, 1, 8, 2, 128, 32, [70, 0, 900], seed=13)
    want = _want(c, -1, 0, 0.09)
    c = _wide(c, 32)  # (small problems take no scratch)
    out = torch.full((3, 1, 8, 128), float("nan"), device=DEV)
    lse = torch.full((3, 8, 1), float("nan"), device=DEV)
    f8 = torch.float8_e4m3fn
    args = [c["q"].to(DEV), c["k"].to(DEV).view(f8), c["v"].to(DEV).view(f8), c["ks"].to(DEV), c["vs"].to(DEV),
            c["table"].to(DEV), c["lens"].to(DEV)]
    need = ga.workspace_bytes_decode(*args)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    got = ga.attn_decode(*args, scale=0.09, out=out, lse=lse, out_fp32=True, workspace=ws)
    assert got[0] is out and got[1] is lse
    _check(got, want, False)
    assert need > 256
    with pytest.raises(ga.AttnError):
        ga.attn_decode(*args, scale=0.09, workspace=ws[:need - 256])


def test_binding_refusals(ga):
    f8 = torch.float8_e4m3fn
    c = _case(2, 1, 8, 2, 64, 16, [40, 3], seed=14)
    good = dict(q=c["q"].to(DEV), k_cache=c["k"].to(DEV).view(f8), v_cache=c["v"].to(DEV).view(f8),
                k_scale=c["ks"].to(DEV), v_scale=c["vs"].to(DEV), page_table=c["table"].to(DEV),
                seqlens=c["lens"].to(DEV))
    ga.attn_decode(**good)
    bad = [dict(q=good["q"].half()), dict(q=good["q"][..., :32].contiguous()), dict(q=good["q"].transpose(1, 2)),
           dict(k_cache=good["k_cache"].view(torch.uint8).short()), dict(v_cache=good["v_cache"][:-1]),
           dict(k_cache=good["k_cache"].view(torch.uint8).transpose(1, 2).view(f8)),
           dict(k_scale=good["k_scale"].double()), dict(v_scale=good["v_scale"][:, :1]),
           dict(page_table=good["page_table"].long()), dict(page_table=good["page_table"][:1]),
           dict(page_table=good["page_table"][:, ::2]), dict(seqlens=good["seqlens"][:1]),
           dict(seqlens=good["seqlens"].cpu()), dict(q=good["q"].cpu()), dict(v_scale=good["v_scale"].cpu())]
    for kw in bad:
        with pytest.raises((ValueError, RuntimeError)):
            ga.attn_decode(**{**good, **kw})
    for kw, code in ((dict(window_left=-2), 1), (dict(sink_tokens=-1), 1), (dict(scale=-1.0), 1)):
        with pytest.raises(ga.AttnError) as err:
            ga.attn_decode(**good, **kw)
        assert err.value.code == code
    cache = [good[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    kv = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    start = torch.zeros(2, **INT)
    before = [t.clone() for t in cache]
    for args, kw in (((kv.float(), kv), {}), ((kv, kv[:1]), {}), ((kv[:, :, :1], kv[:, :, :1]), {}),
                     ((kv, kv), dict(start=start[:1])), ((kv, kv), dict(lens=start.long())),
                     ((kv[:1], kv[:1]), {}), ((kv, kv), dict(tok_start=start.cpu()))):
        with pytest.raises((ValueError, RuntimeError)):
            ga.kv_cache_append(*args, *cache, good["page_table"], **{"start": start, **kw})
    with pytest.raises((ValueError, RuntimeError)):
        ga.kv_cache_copy_pages(*cache, start, start[:1])
    torch.cuda.synchronize()
    for t, u in zip(cache, before):
        assert torch.equal(t.view(torch.uint8) if t.dtype == f8 else t.nan_to_num(9),
                           u.view(torch.uint8) if u.dtype == f8 else u.nan_to_num(9))


@pytest.mark.parametrize("seed", range(24))
def test_random_configurations(ga, seed):
    """Any mix of lengths, query tokens, groups, page sizes, windows, kept tokens and missing pages,
    by clusters and by the list."""
    rng = np.random.default_rng(9000 + seed)
    d, size = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128]))
    n, sq = int(rng.integers(1, 9)), int(rng.choice([1, 1, 2, 3, 5]))
    hkv, g = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 7, 8, 16, 20]))
    lens = [int(m) for m in rng.integers(0, int(rng.choice([20, 200, 900])), n)]
    window = -1 if rng.random() < 0.4 else int(rng.integers(0, 200))
    sink = int(rng.choice([0, 1, 17, 40]))
    c = _case(n, sq, hkv * g, hkv, d, size, lens, seed=seed)
    if rng.random() < 0.5:
        gone = torch.from_numpy(rng.random(c["table"].shape) < 0.2)
        c["table"][gone] = int(rng.choice([-1, 1 << 20]))
    want = _want(c, window, sink, d ** -0.5)
    _check(_run(ga, _wide(c, size) if seed % 2 else c, window, sink, d ** -0.5, out_fp32=True), want, False)
