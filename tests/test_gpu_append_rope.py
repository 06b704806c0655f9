"""Appending to the paged 8-bit cache with the rotation on the way, against the plain fp64 forms.

Tolerance.  K turned is off by 2^-20 of the pair's magnitudes (test_gpu_rope), then rounded to e4m3: by half
a step, 2^-4 of the value or, where codes are subnormal, 2^-10 of the page's scale.  The scale is the plain
form's unless the largest magnitude lies within 2^-19 of a border between two.  V and older slots are those
of the plain form byte for byte, and q as in test_gpu_rope."""
import numpy as np
import pytest
import torch

from tests import paged, rotation
from tests.paged import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
INT = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _cache(pages, h, size, d, seed):
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (pages, 2, h, size, d), generator=g, dtype=torch.int32).to(torch.uint8)
    raw[(raw & 0x7f) == 0x7f] = 0x33
    both = raw.to(DEV)
    scales = [torch.exp2(torch.randint(-9, 2, (pages, h), generator=g).float()).to(DEV) for _ in range(2)]
    return [both[:, 0].contiguous().view(torch.float8_e4m3fn), both[:, 1].contiguous().view(torch.float8_e4m3fn), *scales]


def _rows(b, s, hq, h, d, seed):
    """Columns of one [b, s, hq + 2 h, d], each head of its own size."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-6, 7, (1, 1, hq + 2 * h, 1), generator=g).float())
    x = (torch.randn(b, s, hq + 2 * h, d, generator=g) * size).to(torch.bfloat16).to(DEV)
    return x[:, :, :hq], x[:, :, hq:hq + h], x[:, :, hq + h:]


def _positions(shape, start, lens, tok):
    """Position of every flat token row, -1 where it is no sequence's."""
    pos = np.full(shape[0] * shape[1], -1, dtype=np.int64)
    for i, (a, n, t) in enumerate(zip(start, lens, tok)):
        for j in range(n if a >= 0 else 0):
            if 0 <= t + j < pos.size:
                pos[t + j] = a + j
    return pos


def _check(ga, q, k, v, cache, table, start, news, tok, f, how, **kw):
    """Runs the call (q into a buffer of 7's) and compares everything."""
    width = table.shape[1]
    pos = _positions(q.shape, start, news, tok)
    flat = lambda x: np64(x.flatten(0, 1))
    freqs = f.cpu().numpy()
    turned, mag = rotation.turn(flat(k), pos, freqs, **how)
    want = []
    for x, codes, scale in ((turned, cache[0], cache[2]), (flat(v), cache[1], cache[3])):
        c, s = paged.raw(codes).copy(), scale.cpu().numpy().copy()
        paged.append(x, c, s, table.numpy(), start, news, tok)
        want.append((c, s))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    got = ga.kv_cache_append_rope(q, k, v, *cache, table.to(DEV), torch.tensor(start, **INT), f, q_out=out, **how, **kw)
    assert got is out
    # V as without a rotation
    np.testing.assert_array_equal(paged.raw(cache[1]), want[1][0])
    np.testing.assert_array_equal(cache[3].cpu().numpy(), want[1][1])
    # K: every slot of a new token against its exact value; all others byte for byte
    size = cache[0].shape[2]
    codes, scale = paged.raw(cache[0]), cache[2].cpu().numpy().astype(np.float64)
    other = np.ones(codes.shape, dtype=bool)
    near = np.zeros(scale.shape, dtype=bool)  # pages whose scale may be the next
    for i, (a, n, t) in enumerate(zip(start, news, tok)):
        tops = {}
        for j in range(n if a >= 0 else 0):
            p, row = a + j, t + j
            pid = table[i, p // size] if p // size < width and 0 <= row < turned.shape[0] else -1
            if not 0 <= pid < codes.shape[0]:
                continue
            val, pid = np.where(np.isfinite(turned[row]), np.abs(turned[row]), 0).max(-1), int(pid)
            tops[pid] = np.maximum(tops.get(pid, 0), val)
            exact, sc = turned[row], scale[pid][:, None]
            back = paged.from_e4m3(codes[pid, :, p % size]) * sc
            fin = np.isfinite(exact)
            tol = np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * sc) + 2.0 ** -20 * mag[row]
            assert np.all(np.abs(back - exact)[fin] <= tol[fin])
            assert np.all(np.isnan(back[np.isnan(exact)]))
            other[pid, :, p % size] = False
        for pid, top in tops.items():
            m = np.where(top > 0, np.frexp(top / 448.0)[0] * 2, 1.5)  # [1, 2): 1 at a border
            near[pid] |= (m < 1 + 2.0 ** -19) | (m > 2 - 2.0 ** -19)
    same = scale == want[0][1]
    assert np.all(same | near)
    other &= same[:, :, None, None]
    np.testing.assert_array_equal(codes[other], want[0][0][other])
    # q
    y, mag = rotation.turn(flat(q), pos, freqs, **how)
    o = flat(out)
    mine = pos >= 0
    assert np.all(np.abs(o - y)[mine] <= (2.0 ** -20 * mag + 2.0 ** -8 * np.abs(y))[mine])
    assert np.all(o[~mine] == 7.0)


CASES = [
    # page, d, hq, h, rot, offset, interleaved, amplitude
    (16, 64, 3, 1, 64, 0, False, 1.0),
    (32, 128, 8, 2, 128, 0, False, 1.25),
    (64, 128, 4, 2, 64, 0, True, 1.0),
    (64, 128, 0, 3, 96, 24, False, 0.9),
    (128, 256, 2, 1, 256, 0, False, 1.0),
    (16, 256, 6, 2, 48, 208, True, 1.0),
    (128, 64, 1, 1, 16, 8, False, 1.0),
]


@pytest.mark.parametrize("s,starts", [(1, (0, 15, 100016)), (5, (0, 30, 127)), (150, (0, 1, 129))])
@pytest.mark.parametrize("case", CASES)
def test_rows(ga, case, s, starts):
    size, d, hq, h, rot, offset, inter, amp = case
    first = [a // size for a in starts]
    per = max((s + size - 2) // size + 1, 2)
    cache = _cache(3 * per + 2, h, size, d, seed=s + d)
    ids = torch.randperm(3 * per + 2, generator=torch.Generator().manual_seed(s)).to(torch.int32)
    table = torch.full((3, max(first) + per), -1, dtype=torch.int32)
    for i in range(3):
        table[i, first[i]:first[i] + per] = ids[i * per:(i + 1) * per]
    q, k, v = _rows(3, s, hq, h, d, seed=size)
    lens = [s, max(1, s - 2), s]
    f = ga.rope_frequencies(rot, device=DEV)
    how = dict(offset=offset, interleaved=inter, amplitude=amp)
    _check(ga, q, k, v, cache, table, starts, lens, [0, s, 2 * s], f, how, lens=torch.tensor(lens, **INT))


def test_packed_prompts_and_dropped_tokens(ga):
    """Packed rows with gaps; an empty sequence, an inactive one, lengths over max_new, tokens outside the
    rows, positions behind the table (their q turns all the same), entries that are no page."""
    size, h, d = 16, 2, 64
    cache = _cache(20, h, size, d, seed=5)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1))[:18].reshape(6, 3).to(torch.int32)
    table[3, 1], table[3, 2] = -1, 20
    q, k, v = _rows(2, 60, 5, h, d, seed=9)
    start, lens, tok = [3, 0, -1, 4, 40, 7], [20, 0, 9, 40, 30, 25], [2, 5, 30, 40, 75, 110]
    cut = [min(n, 33) for n in lens]
    f = ga.rope_frequencies(32, device=DEV)
    _check(ga, q, k, v, cache, table, start, cut, tok, f, dict(offset=16, interleaved=True, amplitude=1.0),
           lens=torch.tensor(lens, **INT), tok_start=torch.tensor(tok, **INT), max_new=33)


@pytest.mark.parametrize("fill", ["zero", "inf", "nan", "tiny", "huge"])
@pytest.mark.parametrize("inter", [False, True])
def test_values_at_the_borders(ga, fill, inter):
    size, h, d = 32, 1, 64
    cache = _cache(4, h, size, d, seed=2)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    q, k, v = _rows(1, 40, 1, h, d, seed=3)
    if fill == "zero":
        k.zero_()
    elif fill in ("inf", "nan"):
        k[0, 7, 0, 5], k[0, 30, 0, 1] = float(fill), -float(fill)
        k[0, 35:] = float("nan")
    elif fill == "tiny":
        k.copy_(torch.full_like(k, 1e-40))
    else:  # (a pair's sum stays in range)
        k.copy_(torch.full_like(k, torch.finfo(torch.bfloat16).max / 4))
    if fill == "inf":
        # an infinite value makes infinities and, where a factor is 0 or both values of a pair are infinite, NaN:
        # compared are the finite ones and the scales
        f = ga.rope_frequencies(64, device=DEV)
        turned, _ = rotation.turn(np64(k)[0], np.arange(30, 70), f.cpu().numpy(), interleaved=inter)
        with np.errstate(invalid="ignore"):
            fine = np.isfinite(turned)
        ga.kv_cache_append_rope(None, k, v, *cache, table.to(DEV), torch.tensor([30], **INT), f, interleaved=inter)
        for pid, rows in ((2, slice(0, 2)), (0, slice(2, 34)), (3, slice(34, 40))):
            t, ok = turned[rows, 0], fine[rows, 0]
            slots = slice(30, 32) if pid == 2 else slice(0, t.shape[0])
            back = paged.from_e4m3(paged.raw(cache[0])[pid, 0, slots]) * float(cache[2][pid, 0])
            top = np.abs(t[ok]).max() if ok.any() else 0
            if pid != 2:
                assert top <= 448 * float(cache[2][pid, 0]) * (1 + 2.0 ** -19) and top > 223 * float(cache[2][pid, 0])
            tol = np.maximum(2.0 ** -4 * np.abs(t), 2.0 ** -10 * float(cache[2][pid, 0])) + 2.0 ** -19 * top
            assert np.all(np.abs(back - t)[ok] <= tol[ok])
            assert np.all(np.isnan(back[np.isnan(t)]))
            inf = np.isinf(t)
            assert np.all(back[inf] == np.sign(t[inf]) * 448 * float(cache[2][pid, 0]))
        return
    _check(ga, q, k, v, cache, table, [30], [40], [0], ga.rope_frequencies(64, device=DEV),
           dict(interleaved=inter))


def test_angles_of_zero_and_in_place(ga):
    """With angles of zero the cache is kv_cache_append's, bit for bit, and q stays; q in place beside k and v in
    one packed buffer is what another buffer gets."""
    table = torch.randperm(12, generator=torch.Generator().manual_seed(1))[:10].reshape(2, 5).to(torch.int32).to(DEV)
    start = torch.tensor([0, 9], **INT)
    for inter in (False, True):
        q, k, v = _rows(2, 70, 4, 2, 64, seed=21)
        keep = [t.clone() for t in (q, k, v)]
        plain, turned, again = (_cache(12, 2, 16, 64, seed=4) for _ in range(3))
        ga.kv_cache_append(k, v, *plain, table, start)
        zero = torch.zeros(32, dtype=torch.float64, device=DEV)
        assert ga.kv_cache_append_rope(q, k, v, *turned, table, start, zero, interleaved=inter) is q
        assert torch.equal(q, keep[0])
        for s, t in zip(plain, turned):
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
        f = ga.rope_frequencies(48, device=DEV)
        how = dict(interleaved=inter, offset=16)
        pos = (start[:, None] + torch.arange(70, device=DEV)).to(torch.int32)
        want, _ = ga.rope(q, None, pos, f, **how)
        assert ga.kv_cache_append_rope(None, k, v, *turned, table, start, f, **how) is None
        out = ga.kv_cache_append_rope(q, k, v, *again, table, start, f, q_out=torch.zeros_like(want), **how)
        assert torch.equal(out, want)
        assert ga.kv_cache_append_rope(q, k, v, *again, table, start, f, **how) is q
        assert torch.equal(q, want) and torch.equal(k, keep[1]) and torch.equal(v, keep[2])
        for s, t in zip(turned, again):
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_streams_and_graphs(ga):
    q, k, v = _rows(3, 1, 8, 2, 128, seed=31)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    f = ga.rope_frequencies(128, device=DEV)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], **INT)
    start = torch.tensor([0, 60, 100], **INT)
    first, second = _cache(6, 2, 64, 128, seed=6), _cache(6, 2, 64, 128, seed=6)
    out = torch.empty_like(q)
    for _ in range(3):
        want = ga.kv_cache_append_rope(q, k, v, *first, table, start, f, q_out=torch.empty_like(q))
        start.add_(1)
    start.sub_(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ga.kv_cache_append_rope(q, k, v, *second, table, start, f, q_out=out)
        start.add_(1)
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, want)
    for a, b in zip(first, second):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_rows_past_32_bits(ga):
    """Token rows of q, k and v 2^31 + 64 values apart."""
    step = (1 << 31) + 64
    far = torch.empty(2 * step + 256, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(far, (1, 3, 4, 64), (0, step, 64, 1))
    g = torch.Generator().manual_seed(8)
    x.copy_(torch.randn(1, 3, 4, 64, generator=g).to(torch.bfloat16))
    q, k, v = x[:, :, :2], x[:, :, 2:3], x[:, :, 3:]
    f = ga.rope_frequencies(64, device=DEV)
    table, start = torch.tensor([[1]], **INT), torch.tensor([7], **INT)
    a, b = _cache(2, 1, 16, 64, seed=1), _cache(2, 1, 16, 64, seed=1)
    want = ga.kv_cache_append_rope(q.contiguous(), k.contiguous(), v.contiguous(), *a, table, start, f)
    got = ga.kv_cache_append_rope(q, k, v, *b, table, start, f)
    assert torch.equal(got, want)
    for s, t in zip(a, b):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
