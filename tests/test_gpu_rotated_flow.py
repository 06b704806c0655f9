"""The rotation, the cache and the attention together, as a program uses them.

Serving: what is appended is compared with the rotation elsewhere; here every step's attention is compared with
the plain fp64 form over the cache's own contents (tolerances as in test_gpu_decode), and what lies in the cache
with the rotation of the inputs within its 8 bits.  Training: attn_fwd / attn_bwd against the oracle on the turned
q and k themselves (relative norms of 1e-2, as for the backward elsewhere), and rope_bwd of what they return
against the plain rotation (test_gpu_rope)."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from tests import paged, rotation
from tests.paged import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
INT = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _decode_close(got, cache, q, table, lens, window, sink):
    (out, lse) = got
    ro, rl, mag = paged.decode(np64(q), paged.raw(cache[0]), paged.raw(cache[1]), cache[2].cpu().numpy(),
                               cache[3].cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy(), window, sink,
                               q.shape[3] ** -0.5)
    assert np.all(np.abs(np64(lse) - rl) <= 2e-4)
    assert np.all(np.abs(np64(out) - ro) <= 2.0 ** -10 * mag + 2.0 ** -8 * np.abs(ro))


@pytest.mark.parametrize("n,window,sink", [(5, -1, 0), (20, -1, 0), (20, 100, 4)])
def test_a_prompt_and_its_continuations(ga, n, window, sink):
    """A prompt of 200 tokens goes to the cache, n continuations fork from it (full pages shared, the last copied) and
    take three steps; tables for 256k tokens, so that the shared keys' kernels run."""
    hq, hkv, d, size, prompt, steps = 8, 2, 128, 32, 200, 3
    g = torch.Generator().manual_seed(n)
    f = ga.rope_frequencies(64, device=DEV)
    how = dict(offset=32, interleaved=True, amplitude=1.1)
    per = -(-(prompt + steps) // size)
    pages = per + 2 * n
    cache = [torch.zeros(pages, hkv, size, d, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    cache += [torch.zeros(pages, hkv, device=DEV) for _ in range(2)]

    def rows(b, s):
        x = torch.randn(b, s, hq + 2 * hkv, d, generator=g).to(torch.bfloat16).to(DEV)
        return x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]

    table = torch.full((n, (1 << 18) // size), -1, **INT)
    full = prompt // size
    table[:, :per] = torch.arange(per, **INT)
    q, k, v = rows(1, prompt)
    keep, kept_q = np64(k), np64(q)
    ga.kv_cache_append_rope(q, k, v, *cache, table[:1], torch.zeros(1, **INT), f, **how)  # q in place
    want, mag = rotation.turn(kept_q[0], np.arange(prompt), f.cpu().numpy(), **how)
    assert np.all(np.abs(np64(q)[0] - want) <= 2.0 ** -20 * mag + 2.0 ** -8 * np.abs(want))
    turned, mag = rotation.turn(keep[0], np.arange(prompt), f.cpu().numpy(), **how)
    code = paged.from_e4m3(paged.raw(cache[0])[:per]) * cache[2].cpu().numpy()[:per, :, None, None]
    code = np.swapaxes(code, 1, 2).reshape(-1, hkv, d)[:prompt]
    step = np.repeat(cache[2].cpu().numpy()[:per], size, 0)[:prompt, :, None]
    assert np.all(np.abs(code - turned) <= np.maximum(2.0 ** -4 * np.abs(turned), 2.0 ** -10 * step) + 2.0 ** -20 * mag)
    # the forks: each its own copy of the page that the prompt ends in, and a page to go on
    for i in range(1, n):
        table[i, full], table[i, full + 1] = per + 2 * i - 2, per + 2 * i - 1
    src, dst = torch.full((n - 1,), full, **INT), table[1:, full].contiguous()
    ga.kv_cache_copy_pages(*cache, src, dst)
    shared, lens = torch.full((n,), full, **INT), torch.full((n,), prompt, **INT)
    for _ in range(steps):
        q, k, v = rows(n, 1)
        q = ga.kv_cache_append_rope(q.contiguous(), k, v, *cache, table, lens, f, **how)
        lens += 1
        got = ga.attn_decode_shared(q, *cache, table, lens, shared, window_left=window, sink_tokens=sink)
        _decode_close(got, cache, q, table, lens, window, sink)
        plain = ga.attn_decode(q, *cache, table, lens, window_left=window, sink_tokens=sink)
        _decode_close(plain, cache, q, table, lens, window, sink)


@pytest.mark.parametrize("inter", [False, True])
def test_a_training_step(ga, inter):
    b, s, hq, hkv, d, window = 2, 300, 4, 2, 64, 90
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(b, s, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (hq, hkv, hkv, hq))
    ids, pos = ga.segments_from_seqlens(torch.tensor([[170, 130], [300, 0]], **INT), s)
    f = ga.rope_frequencies(d, factor=4.0, method="parts", device=DEV)
    how = dict(interleaved=inter, amplitude=1.1386)
    q1, k1 = ga.rope(q, k, pos, f, **how)
    out, lse = ga.attn_fwd(q1, k1, v, ids, pos, window_left=window)
    dq1, dk1, dv = ga.attn_bwd(q1, k1, v, out, lse, do, ids, pos, window_left=window)
    dq, dk = ga.rope_bwd(dq1, dk1, pos, f, **how)
    cpu = [t.cpu() for t in (q1, k1, v, ids, pos)]
    ro, rl = A.attn_fwd(*cpu, cpu[3], cpu[4], window, d ** -0.5)
    assert np.linalg.norm(np64(out) - ro) <= 1e-2 * np.linalg.norm(ro)
    rq, rk, rv = A.attn_bwd(cpu[0], cpu[1], cpu[2], do.cpu(), cpu[3], cpu[4], cpu[3], cpu[4], window, d ** -0.5,
                            out=out.float().cpu())
    for got, want in ((dq1, rq), (dk1, rk), (dv, rv)):
        assert np.linalg.norm(np64(got) - want) <= 1e-2 * np.linalg.norm(want)
    for got, grad in ((dq, dq1), (dk, dk1)):
        want, mag = rotation.turn(np64(grad), pos.cpu().numpy(), f.cpu().numpy(), inverse=True, **how)
        assert np.all(np.abs(np64(got) - want) <= 2.0 ** -20 * mag + 2.0 ** -8 * np.abs(want))


def test_a_captured_decoding_step(ga):
    """Rotation, append and attention in one graph, replayed as the sequences grow, are what eager calls give."""
    n, hq, hkv, d, size = 16, 16, 2, 64, 16
    g = torch.Generator().manual_seed(5)
    f = ga.rope_frequencies(d, device=DEV)
    pages = 20 + 4 * n
    start = torch.randint(0, 256, (pages, hkv, size, d), generator=g, dtype=torch.int32).to(torch.uint8) & 0x6f
    table = torch.full((n, (1 << 18) // size), -1, **INT)
    table[:, :20] = torch.arange(20, **INT)
    table[:, 20:24] = 20 + torch.arange(4 * n, **INT).reshape(n, 4)
    shared = torch.full((n,), 20, **INT)
    steps = [torch.randn(n, 1, hq + 2 * hkv, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(20)]
    x = torch.empty_like(steps[0])

    def fresh():
        c = [start.to(DEV).view(torch.float8_e4m3fn).clone(), start.to(DEV).view(torch.float8_e4m3fn).clone()]
        return c + [torch.full((pages, hkv), 2.0 ** -9, device=DEV) for _ in range(2)], torch.full((n,), 20 * size, **INT)

    def step(cache, lens, q_out):
        q = ga.kv_cache_append_rope(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], *cache, table, lens, f,
                                    q_out=q_out)
        lens.add_(1)
        return ga.attn_decode_shared(q, *cache, table, lens, shared)

    cache, lens = fresh()
    q_out, want = torch.empty(n, 1, hq, d, dtype=torch.bfloat16, device=DEV), []
    for t in steps:
        x.copy_(t)
        want.append([y.clone() for y in step(cache, lens, q_out)])
    again, lens2 = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(again, lens2, q_out)
    for t, (out, lse) in zip(steps, want):
        x.copy_(t)
        graph.replay()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    for a, b in zip(cache, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
