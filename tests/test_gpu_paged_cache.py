"""The paged 8-bit cache: append and page copies, byte for byte against the plain forms."""
import numpy as np
import pytest
import torch

from tests import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _cache(pages, h, size, d, seed, halves=False):
    """Random finite codes and power-of-two scales (as one buffer's halves on request)."""
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (pages, 2, h, size, d), generator=g, dtype=torch.int32).to(torch.uint8)
    raw[(raw & 0x7f) == 0x7f] = 0x33
    both = raw.to(DEV)
    k, v = both[:, 0], both[:, 1]
    if not halves:
        k, v = k.contiguous(), v.contiguous()
    scales = [torch.exp2(torch.randint(-9, 2, (pages, h), generator=g).float()).to(DEV) for _ in range(2)]
    return [k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), *scales]


def _tables(n, per, pages, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[:n * per].reshape(n, per).to(torch.int32)


def _expect(k, v, cache, table, start, lens, tok_start):
    out = []
    for x, codes, scale in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        c, s = paged.raw(codes).copy(), scale.cpu().numpy().copy()
        paged.append(paged.np64(x).reshape(-1, *x.shape[2:]), c, s, table.numpy(), start, lens, tok_start)
        out.append((c, s))
    return out


def _same(cache, want):
    for (codes, scale), (c, s) in zip(((cache[0], cache[2]), (cache[1], cache[3])), want):
        np.testing.assert_array_equal(paged.raw(codes), c)
        np.testing.assert_array_equal(scale.cpu().numpy(), s)


def _new(b, s, h, d, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-6, 7, (1, 1, h, 1), generator=g).float())
    kv = (torch.randn(b, s, 2, h, d, generator=g) * size[:, :, None]).to(torch.bfloat16).to(DEV)
    return (kv[:, :, 0], kv[:, :, 1]) if packed else (kv[:, :, 0].contiguous(), kv[:, :, 1].contiguous())


@pytest.mark.parametrize("size,d,h", [(16, 64, 1), (32, 128, 3), (64, 128, 2), (128, 256, 1), (16, 256, 2)])
@pytest.mark.parametrize("s,starts", [(1, (0, 15, 16)), (5, (0, 30, 127)), (150, (0, 1, 129))])
def test_append_rows(ga, size, d, h, s, starts):
    per = (max(starts) + s) // size + 1
    cache = _cache(3 * per + 2, h, size, d, seed=s + d, halves=s == 5)
    table = _tables(3, per, 3 * per + 2, seed=s)
    k, v = _new(3, s, h, d, seed=size, packed=s != 1)
    lens = [s, max(1, s - 2), s]
    want = _expect(k, v, cache, table, starts, lens, [0, s, 2 * s])
    ga.kv_cache_append(k, v, *cache, table.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV),
                       lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    _same(cache, want)


def test_append_packed_prompts_and_dropped_tokens(ga):
    """Packed rows with gaps; an empty sequence, an inactive one, lengths over max_new, tokens
    outside the rows, positions behind the table, entries that are no page."""
    size, h, d = 16, 2, 64
    cache = _cache(20, h, size, d, seed=5)
    table = _tables(6, 3, 20, seed=1)
    table[3, 1], table[3, 2] = -1, 20
    k, v = _new(2, 60, h, d, seed=9, packed=True)
    start, lens, tok = [3, 0, -1, 4, 40, 7], [20, 0, 9, 40, 30, 25], [2, 5, 30, 40, 70, 110]
    want = _expect(k, v, cache, table, start, [min(n, 33) for n in lens], tok)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ga.kv_cache_append(k, v, *cache, table.to(DEV), i32(start), lens=i32(lens), tok_start=i32(tok), max_new=33)
    _same(cache, want)


def test_append_token_rows_outside_the_tensor(ga):
    """Rows before the first and behind the last are dropped, however far: what stays of a
    page's new tokens counts, and the slots before them are the page's older tokens."""
    size, h, d = 16, 1, 64
    tok = [-3, -(1 << 31), (1 << 31) - 1, 25, -40, 20]
    start, lens = [5, 0, 0, 3, 9, 30], [30, 40, 40, 40, 40, 2]
    cache = _cache(20, h, size, d, seed=8)
    table = _tables(6, 3, 20, seed=8)
    k, v = _new(1, 30, h, d, seed=8)
    want = _expect(k, v, cache, table, start, lens, tok)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ga.kv_cache_append(k, v, *cache, table.to(DEV), i32(start), lens=i32(lens), tok_start=i32(tok), max_new=40)
    _same(cache, want)


@pytest.mark.parametrize("fill", ["zero", "inf", "nan", "tiny", "huge", "border"])
def test_append_values_at_the_borders(ga, fill):
    size, h, d = 32, 1, 64
    cache = _cache(4, h, size, d, seed=2)
    table = _tables(1, 3, 4, seed=2)
    k, v = _new(1, 40, h, d, seed=3)
    if fill == "zero":
        k.zero_()
    elif fill in ("inf", "nan"):
        k[0, 7, 0, 5], v[0, 30, 0, 1] = float(fill), -float(fill)
        k[0, 35:] = float(fill)  # a page with nothing finite
    elif fill == "tiny":
        k.copy_(torch.full_like(k, 1e-40))
    elif fill == "huge":
        k.copy_(torch.full_like(k, torch.finfo(torch.bfloat16).max))
    else:  # the largest magnitude exactly 448 * 2^n, and the next value above it
        k.clamp_(-3, 3)[0, 0, 0, 0], v.clamp_(-3, 3)[0, 1, 0, 3] = 3.5, -3.515625
    want = _expect(k, v, cache, table, [30], [40], [0])
    ga.kv_cache_append(k, v, *cache, table.to(DEV), torch.tensor([30], dtype=torch.int32, device=DEV))
    _same(cache, want)


def test_append_token_by_token_grows_the_scale(ga):
    """Forty single tokens, each larger than the last: every growth requantises the page's
    older tokens, as the plain form does."""
    size, h, d = 16, 2, 64
    cache = _cache(5, h, size, d, seed=4)
    table = _tables(1, 3, 5, seed=4)
    for t in range(40):
        k, v = _new(1, 1, h, d, seed=100 + t)
        k, v = (k.float() * 1.25 ** t).to(torch.bfloat16), v
        want = _expect(k, v, cache, table, [t], [1], [0])
        ga.kv_cache_append(k, v, *cache, table.to(DEV), torch.tensor([t], dtype=torch.int32, device=DEV))
        _same(cache, want)


@pytest.mark.parametrize("h,size,d,halves", [(1, 16, 64, False), (3, 32, 128, True), (8, 128, 256, False)])
def test_copy_pages(ga, h, size, d, halves):
    cache = _cache(12, h, size, d, seed=6, halves=halves)
    want = [paged.raw(cache[0]).copy(), paged.raw(cache[1]).copy(), cache[2].cpu().numpy(), cache[3].cpu().numpy()]
    src, dst = [3, 3, 7, -1, 5, 2, 12], [4, 0, 11, 6, 5, 12, 1]  # a source twice, no pages, itself
    for s, t in [(3, 4), (3, 0), (7, 11)]:
        for x in want:
            x[t] = x[s]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ga.kv_cache_copy_pages(*cache, i32(src), i32(dst))
    got = [paged.raw(cache[0]), paged.raw(cache[1]), cache[2].cpu().numpy(), cache[3].cpu().numpy()]
    for x, y in zip(got, want):
        np.testing.assert_array_equal(x, y)


def test_copy_no_pairs(ga):
    cache = _cache(3, 1, 16, 64, seed=0)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    ga.kv_cache_copy_pages(*cache, none, none)


@pytest.mark.parametrize("seed", range(16))
def test_random_appends(ga, seed):
    """Three calls in a row on one cache with any starts, lengths, page sizes and heads."""
    rng = np.random.default_rng(8000 + seed)
    d, size, h = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 4))
    n, per = int(rng.integers(1, 5)), int(rng.integers(1, 5))
    cache = _cache(n * per + 2, h, size, d, seed=seed, halves=bool(seed & 1))
    table = _tables(n, per, n * per + 2, seed=seed)
    if seed % 3 == 0:
        table[rng.integers(0, n), rng.integers(0, per)] = -1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    at = [int(x) for x in rng.integers(0, size, n)]
    for call in range(3):
        s = int(rng.choice([1, 2, 17, 40]))
        k, v = _new(n, s, h, d, seed=100 * seed + call, packed=bool(seed & 2))
        lens = [int(x) for x in rng.integers(0, s + 1, n)]
        want = _expect(k, v, cache, table, at, lens, [i * s for i in range(n)])
        ga.kv_cache_append(k, v, *cache, table.to(DEV), i32(at), lens=i32(lens))
        _same(cache, want)
        at = [a + m for a, m in zip(at, lens)]
