"""Appending with the rotation on the CPU: host checks of the C ABI (fake pointers, nothing is launched),
the binding's refusals and what it makes of its tensors."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__
    __graft_entry__.build()
    import long_context_attention_attn_gb300 as pkg
    return pkg


@pytest.fixture
def ga(pkg, monkeypatch):
    """The tensors pass for a GPU's; the call notes its parameters and launches nothing."""
    calls = []

    def note(index, call, ref, *rest):
        calls.append((call.__name__, ref._obj, rest))
        return 0

    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(pkg, "_on_device", note)
    pkg.calls = calls
    yield pkg
    del pkg.calls


A = 1 << 40  # aligned non-null fake device addresses; never dereferenced


def _append(pkg, **kw):
    p = pkg.KvAppendRopeParams()
    a, c, r = p.append, p.append.cache, p.rotation
    c.k, c.v, c.k_scale, c.v_scale = A, 2 * A, 3 * A, 4 * A
    c.num_pages, c.h_kv, c.page_size, c.d = 100, 2, 64, 128
    a.k, a.v, a.tokens = 5 * A, 6 * A, 10
    a.page_table, a.n, a.max_pages, a.start, a.row_tokens, a.max_new = 7 * A, 3, 8, 8 * A, 4, 4
    r.freqs, r.rot = 9 * A, 128  # (amplitude 0: one)
    p.q, p.q_out, p.h_q = 10 * A, 11 * A, 8
    for n, v in kw.items():
        where = r if n in ("freqs", "rot", "offset", "amplitude") else p if hasattr(p, n) else a if hasattr(a, n) else c
        setattr(where, n, v)
    return pkg.lib().attn_kv_append_rope(ctypes.byref(p), None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(start=None), 1), (dict(n=0), 1), (dict(max_new=0), 1), (dict(token_stride=260), 1),
    (dict(page_size=48), 2), (dict(num_pages=0), 1),              # as attn_kv_append
    (dict(freqs=None), 1), (dict(rot=0), 1), (dict(rot=136), 1), (dict(rot=24), 2), (dict(rot=64, offset=72), 1),
    (dict(rot=64, offset=4), 2), (dict(amplitude=-1.0), 1),       # as attn_rope
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(q=10 * A + 2), 1), (dict(h_q=-1), 1), (dict(h_q=65536), 2),
    (dict(q_stride=1000), 1), (dict(q_stride=1028), 1), (dict(q_out_stride=-8), 1),
    (dict(q_out=10 * A + 2048), 1), (dict(q_out=10 * A, q_out_stride=2048), 1),  # q over its output
    (dict(q_out=5 * A), 1), (dict(q_out=6 * A + 256), 1), (dict(q_out=A), 1), (dict(q=2 * A), 1), (dict(q=3 * A), 1),
])
def test_refusals(pkg, kw, code):
    assert _append(pkg, **kw) == code


def test_refuses_no_parameters(pkg):
    assert pkg.lib().attn_kv_append_rope(None, None) == 1


def _cache(pages=4, h=2, size=16, d=64):
    return ([torch.zeros(pages, h, size, d, dtype=torch.uint8) for _ in range(2)]
            + [torch.zeros(pages, h) for _ in range(2)])


def test_binding(ga):
    qkv = torch.zeros(2, 5, 8, 64, dtype=torch.bfloat16)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    table, start = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    f = torch.ones(16, dtype=torch.float64)
    cache = _cache()
    got = ga.kv_cache_append_rope(q, k, v, *cache, table, start, f, max_new=3, offset=8, interleaved=True,
                                  amplitude=2.0)
    assert got is q
    name, p, _ = ga.calls.pop()
    assert name == "attn_kv_append_rope"
    a = p.append
    assert (a.k, a.v, a.tokens, a.token_stride, a.n, a.max_new, a.row_tokens) == (k.data_ptr(), v.data_ptr(), 10, 512, 2, 3, 5)
    assert (p.q, p.q_out, p.h_q, p.q_stride, p.q_out_stride) == (q.data_ptr(), q.data_ptr(), 4, 512, 512)
    r = p.rotation
    assert (r.freqs, r.rot, r.offset, r.interleaved, r.amplitude) == (f.data_ptr(), 32, 8, 1, 2.0)
    out = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16)
    assert ga.kv_cache_append_rope(q, k, v, *cache, table, start, f, q_out=out) is out
    assert ga.calls.pop()[1].q_out_stride == 256
    assert ga.kv_cache_append_rope(None, k, v, *cache, table, start, f) is None
    assert ga.calls.pop()[1].h_q == 0
    none = torch.zeros(0, 3, dtype=torch.int32)
    assert ga.kv_cache_append_rope(q[:0], k[:0], v[:0], *cache, none, start[:0], f).shape == (0, 5, 4, 64)
    assert ga.calls == []
    bad = [
        dict(q=q.float()), dict(q=q[:, :4]), dict(q=q[..., :32]), dict(q=None, q_out=out), dict(q_out=out[:, :, :2]),
        dict(q_out=out.float()), dict(freqs=f.float()), dict(amplitude=0.0), dict(k=k.float()), dict(start=start.long()),
        dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
    ]
    for kw in bad:
        args = dict(q=q, k=k, v=v, start=start, freqs=f)
        more = {n: kw.pop(n) for n in list(kw) if n not in args}
        args.update(kw)
        with pytest.raises(ValueError):
            ga.kv_cache_append_rope(args["q"], args["k"], args["v"], *cache, table, args["start"], args["freqs"], **more)
    assert ga.calls == []


def test_binding_refuses_host_tensors(pkg):
    kv, i32 = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.kv_cache_append_rope(kv, kv, kv, *_cache(), i32[None], i32, torch.ones(32, dtype=torch.float64))
