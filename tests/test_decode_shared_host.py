"""Decoding behind shared pages on the CPU: host checks of the C ABI (fake pointers, nothing is launched),
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


def _decode(pkg, **kw):
    p = pkg.DecodeSharedParams()
    b, c = p.base, p.base.cache
    c.k, c.v, c.k_scale, c.v_scale = A, 2 * A, 3 * A, 4 * A
    c.num_pages, c.h_kv, c.page_size, c.d = 100, 2, 64, 128
    b.q, b.page_table, b.seqlens, b.out, b.lse = 5 * A, 6 * A, 7 * A, 8 * A, 9 * A
    b.n, b.max_pages, b.s_q, b.h_q, b.window_left, b.scale = 3, 8, 1, 8, -1, 0.1
    b.workspace, b.workspace_bytes = 10 * A, 1 << 40
    p.shared_pages, p.group_start, p.n_groups, p.max_group = 11 * A, 12 * A, 2, 2
    for n, v in kw.items():
        setattr(p if hasattr(p, n) else b if hasattr(b, n) else c, n, v)
    rc = pkg.lib().attn_decode_shared(ctypes.byref(p), None)
    assert pkg.lib().attn_decode_shared_workspace_bytes(ctypes.byref(p)) == 0 or "workspace" in kw
    assert pkg.lib().attn_decode_shared_test_timeout(ctypes.byref(p), None) == rc
    return rc


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=48), 2), (dict(d=192), 2), (dict(q=None), 1), (dict(n=0), 1), (dict(s_q=300), 2),
    (dict(window_left=-2), 1), (dict(scale=0.0), 1), (dict(workspace=A + 128), 1),  # as attn_decode
    (dict(shared_pages=None), 1), (dict(shared_pages=A + 2), 1), (dict(group_start=A + 1), 1), (dict(n_groups=0), 1),
    (dict(n_groups=65536), 2), (dict(group_start=None), 1), (dict(max_group=0), 1), (dict(max_group=4), 1),
])
def test_refusals(pkg, kw, code):
    assert _decode(pkg, **kw) == code


def test_refuses_no_parameters(pkg):
    assert pkg.lib().attn_decode_shared(None, None) == 1
    assert pkg.lib().attn_decode_shared_workspace_bytes(None) == 0


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_binding(ga):
    cache = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8) for _ in range(2)] + [torch.zeros(4, 2) for _ in range(2)]
    q, table, lens = torch.zeros(3, 1, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int32), _i32(17, 18, 19)
    shared, groups, ws = _i32(1, 1, 0), _i32(0, 2, 3), torch.empty(4096, dtype=torch.uint8)
    ga.attn_decode_shared(q, *cache, table, lens, shared, groups, max_group=2, window_left=5, sink_tokens=3, workspace=ws)
    name, p, _ = ga.calls.pop()
    assert name == "attn_decode_shared"
    assert (p.shared_pages, p.group_start, p.n_groups, p.max_group) == (shared.data_ptr(), groups.data_ptr(), 2, 2)
    b = p.base
    assert (b.q, b.n, b.max_pages, b.window_left, b.sink_tokens) == (q.data_ptr(), 3, 2, 5, 3)
    assert (b.workspace, b.workspace_bytes) == (ws.data_ptr(), 4096)
    ga.attn_decode_shared(q, *cache, table, lens, shared, workspace=ws)
    p = ga.calls.pop()[1]
    assert (p.group_start, p.n_groups, p.max_group) == (None, 1, 3)
    out, lse = ga.attn_decode_shared(q[:0], *cache, table[:0], lens[:0], shared[:0])
    assert out.shape == (0, 1, 4, 64) and lse.shape == (0, 4, 0) or lse.shape == (0, 4, 1)
    assert ga.calls == []
    for kw in (dict(shared=shared[:2]), dict(shared=shared.long()), dict(groups=groups[None]), dict(groups=groups[:1]),
               dict(groups=groups.long())):
        with pytest.raises(ValueError):
            ga.attn_decode_shared(q, *cache, table, lens, kw.get("shared", shared), kw.get("groups", groups), workspace=ws)
    assert ga.calls == []


def test_binding_refuses_host_tensors(pkg):
    cache = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8) for _ in range(2)] + [torch.zeros(4, 2) for _ in range(2)]
    with pytest.raises(ValueError, match="CUDA"):
        pkg.attn_decode_shared(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), *cache, _i32(0)[None], _i32(1), _i32(1))
