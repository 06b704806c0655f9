"""The paged cache's operators on the CPU: host checks of the C ABI (fake pointers, nothing is
launched), the binding's refusals, and the tests' plain forms against torch's e4m3."""
import ctypes

import numpy as np
import pytest
import torch

from tests import paged


@pytest.fixture(scope="module")
def ga():
    import __graft_entry__
    __graft_entry__.build()
    import long_context_attention_attn_gb300 as pkg
    return pkg


A = 1 << 40  # aligned non-null fake device addresses; never dereferenced


def _fill(c, kw):
    c.k, c.v, c.k_scale, c.v_scale = A, 2 * A, 3 * A, 4 * A
    c.num_pages, c.h_kv, c.page_size, c.d = 100, 2, 64, 128
    for n in list(kw):
        if n.startswith("c_"):
            setattr(c, n[2:], kw.pop(n))


def _append(ga, **kw):
    p = ga.KvAppendParams()
    _fill(p.cache, kw)
    p.k, p.v, p.tokens = 5 * A, 6 * A, 10
    p.page_table, p.n, p.max_pages, p.start = 7 * A, 3, 8, 8 * A
    p.row_tokens, p.max_new = 4, 4
    for n, v in kw.items():
        setattr(p, n, v)
    return ga.lib().attn_kv_append(ctypes.byref(p), None)


def _decode(ga, **kw):
    p = ga.DecodeParams()
    _fill(p.cache, kw)
    p.q, p.page_table, p.seqlens, p.out, p.lse = 5 * A, 6 * A, 7 * A, 8 * A, 9 * A
    p.n, p.max_pages, p.s_q, p.h_q, p.window_left, p.scale = 3, 8, 1, 8, -1, 0.1
    p.workspace, p.workspace_bytes = 10 * A, 1 << 30
    for n, v in kw.items():
        setattr(p, n, v)
    rc = ga.lib().attn_decode(ctypes.byref(p), None)
    assert ga.lib().attn_decode_workspace_bytes(ctypes.byref(p)) == 0 or "workspace" in kw
    return rc


def _copy(ga, n=3, src=5 * A, dst=6 * A, **kw):
    c = ga.KvCache()
    _fill(c, kw)
    return ga.lib().attn_kv_copy_pages(ctypes.byref(c), src, dst, n, None)


CACHE = [
    (dict(c_k=None), 1), (dict(c_v_scale=None), 1), (dict(c_k=A + 8), 1), (dict(c_k_scale=A + 2), 1),
    (dict(c_num_pages=0), 1), (dict(c_h_kv=0), 1), (dict(c_num_pages=1 << 31), 2), (dict(c_h_kv=65536), 2),
    (dict(c_page_size=48), 2), (dict(c_page_size=256), 2), (dict(c_d=96), 2), (dict(c_d=192), 2),
    (dict(c_page_stride=2 * 64 * 128 - 16), 1), (dict(c_page_stride=2 * 64 * 128 + 8), 1),
    (dict(c_page_stride=-16), 1),
]


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_is_checked_by_every_call(ga, kw, code):
    assert _append(ga, **kw) == code
    assert _decode(ga, **kw) == code
    assert _copy(ga, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=6 * A + 2), 1), (dict(start=None), 1), (dict(lens=A + 2), 1), (dict(tok_start=A + 1), 1),
    (dict(page_table=None), 1), (dict(n=0), 1), (dict(n=65536), 2), (dict(max_pages=0), 1),
    (dict(max_pages=(1 << 24) + 1), 2), (dict(tokens=0), 1), (dict(max_new=0), 1), (dict(max_new=(1 << 30) + 1), 2),
    (dict(row_tokens=-1), 1), (dict(token_stride=128), 1), (dict(token_stride=260), 1),
    (dict(k=A + 4096), 1), (dict(v=4 * A), 1),  # inputs over the cache's pages or scales
])
def test_append_refusals(ga, kw, code):
    assert _append(ga, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(lse=None), 1), (dict(seqlens=None), 1), (dict(page_table=A + 2), 1),
    (dict(q=A + 8), 1), (dict(out=A + 8), 1), (dict(n=0), 1), (dict(n=65536), 2), (dict(s_q=0), 1), (dict(h_q=7), 1),
    (dict(h_q=0), 1), (dict(window_left=-2), 1), (dict(sink_tokens=-1), 1), (dict(sink_tokens=1 << 31), 2),
    (dict(scale=0.0), 1), (dict(scale=float("inf")), 1), (dict(s_q=300), 2), (dict(s_q=1025, h_q=2), 2),
    (dict(max_pages=(1 << 24) + 1), 2), (dict(workspace=10 * A + 128), 1),
])
def test_decode_refusals(ga, kw, code):
    assert _decode(ga, **kw) == code


def test_copy_refusals(ga):
    assert _copy(ga, n=0) == 1
    assert _copy(ga, src=None) == 1
    assert _copy(ga, dst=6 * A + 2) == 1
    assert _copy(ga, n=1 << 31) == 2
    assert ga.lib().attn_kv_copy_pages(None, A, A, 1, None) == 1
    assert ga.lib().attn_kv_append(None, None) == 1
    assert ga.lib().attn_decode(None, None) == 1


def test_binding_refuses_host_tensors(ga):
    cache = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8) for _ in range(2)] + [torch.zeros(4, 2) for _ in range(2)]
    kv = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda: ga.kv_cache_append(kv, kv, *cache, table, i32),
                 lambda: ga.attn_decode(kv, *cache, table, i32),
                 lambda: ga.kv_cache_copy_pages(*cache, i32, i32)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_plain_e4m3_matches_torch():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float())
    x = torch.cat([x.clamp(-448, 448), torch.from_numpy((paged.E4M3[1:] + paged.E4M3[:-1]) / 2).float()])
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(paged.to_e4m3(x.double().numpy()), want)
    codes = np.arange(256, dtype=np.uint8)
    back = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(paged.from_e4m3(codes), back)
