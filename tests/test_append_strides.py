"""Token rows far apart in what is appended: the host's limits (fake pointers, nothing is launched),
and one token of every row of a long batch, byte for byte."""
import ctypes

import pytest
import torch

from tests.test_gpu_paged_cache import DEV, _cache, _expect, _same, _tables, ga  # noqa: F401


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=2, token_stride=(1 << 40) + 8), 2),
    (dict(tokens=(1 << 16) + 1, token_stride=(1 << 30) + 8), 2),   # more than 2^46 values apart in all
    (dict(tokens=1 << 36, token_stride=1 << 24), 2),
    (dict(tokens=3, token_stride=1 << 25, k=64), 1),               # within the limits: over the cache's pages
])
def test_limits_of_the_rows_distance(kw, code):
    import __graft_entry__
    __graft_entry__.build()
    import long_context_attention_attn_gb300 as ga
    a = 1 << 24
    p = ga.KvAppendParams()
    c = p.cache
    c.k, c.v, c.k_scale, c.v_scale = a, 2 * a, 3 * a, 4 * a
    c.num_pages, c.h_kv, c.page_size, c.d = 100, 2, 64, 128
    p.k, p.v, p.page_table, p.start = 5 * a, 6 * a, 7 * a, 8 * a
    p.n, p.max_pages, p.row_tokens, p.max_new = 1, 8, 4, 4
    for n, v in kw.items():
        setattr(p, n, v)
    assert ga.lib().attn_kv_append(ctypes.byref(p), None) == code


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_one_token_of_every_row(ga, packed):
    """k[:, t:t+1] of rows of 20000 tokens: 2^24 values and more from row to row."""
    b, s, h, d, size = 3, 20000, 8, 128, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    if packed:
        kv = torch.randn(b, s // 2, 2, h, d, generator=g, device=DEV).to(torch.bfloat16)
        k, v = kv[:, 777:778, 0], kv[:, 777:778, 1]
    else:
        k, v = (torch.randn(b, s, h, d, generator=g, device=DEV).to(torch.bfloat16)[:, 777:778] for _ in range(2))
    assert k.stride(0) > 1 << 24
    cache = _cache(8, h, size, d, seed=3)
    table = _tables(b, 2, 8, seed=3)
    starts = [0, 7, 16]
    want = _expect(k, v, cache, table, starts, [1] * b, list(range(b)))
    ga.kv_cache_append(k, v, *cache, table.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
    _same(cache, want)
