"""What the paged cache's binding makes of its tensors, on the CPU: the tensors pass for a GPU's and
the library call is replaced by one that notes its parameters, so nothing is launched."""
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
    calls = []

    def note(index, call, ref, *rest):
        calls.append((call.__name__, ref._obj, rest))
        return 0

    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(pkg, "_on_device", note)
    pkg.calls = calls
    yield pkg
    del pkg.calls


def _cache(pages=4, h=2, size=16, d=64):
    return ([torch.zeros(pages, h, size, d, dtype=torch.uint8) for _ in range(2)]
            + [torch.zeros(pages, h) for _ in range(2)])


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def _kv(b, s, h=2, d=64):
    return torch.zeros(b, s, h, d, dtype=torch.bfloat16)


def test_rows_of_stride_zero_are_refused(ga):
    """One token (or row) broadcast to several has no stride that the library could take: 0 means
    contiguous there, and rows behind the tensor's end would be read."""
    table = torch.zeros(3, 2, dtype=torch.int32)
    start = _i32(0, 0, 0)
    for k in (_kv(1, 1).expand(3, 1, 2, 64), _kv(1, 1).expand(3, 5, 2, 64), _kv(3, 1).expand(3, 5, 2, 64)):
        for pair in ((k, k), (k, k.contiguous()), (k.contiguous(), k)):
            with pytest.raises(ValueError):
                ga.kv_cache_append(*pair, *_cache(), table, start)
    with pytest.raises(ValueError):
        ga.kv_cache_append(_kv(1, 1).expand(1, 5, 2, 64), _kv(1, 1).expand(1, 5, 2, 64), *_cache(), table[:1], start[:1])
    assert ga.calls == []
    # rows of a larger tensor are taken as they lie, and sizes of one have no stride
    kv = torch.zeros(3, 5, 2, 2, 64, dtype=torch.bfloat16)
    ga.kv_cache_append(kv[:, :, 0], kv[:, :, 1], *_cache(), table, start)
    ga.kv_cache_append(kv[:, 2:3, 0], kv[:, 2:3, 1], *_cache(), table, start)
    one = _kv(1, 1).as_strided((1, 1, 2, 64), (0, 0, 64, 1))
    ga.kv_cache_append(one, one, *_cache(), table[:1], start[:1])
    assert [c[1].token_stride for c in ga.calls] == [2 * 2 * 64, 5 * 2 * 2 * 64, 2 * 64]


def test_pages_of_stride_zero_are_refused(ga):
    wide = [t[:1].expand(4, -1, -1, -1) for t in _cache()[:2]]
    cache = (*wide, *_cache()[2:])
    table, one = torch.zeros(1, 2, dtype=torch.int32), _i32(0)
    with pytest.raises(ValueError):
        ga.kv_cache_append(_kv(1, 1), _kv(1, 1), *cache, table, one)
    with pytest.raises(ValueError):
        ga.kv_cache_copy_pages(*cache, one, one)
    with pytest.raises(ValueError):
        ga.attn_decode(_kv(1, 1), *cache, table, one)
    with pytest.raises(ValueError):
        ga.workspace_bytes_decode(_kv(1, 1), *cache, table, one)
    assert ga.calls == []


def test_packed_sequences_need_lengths(ga):
    """Without lengths each sequence would take all tokens from its first on, other sequences' too."""
    k, table, two = _kv(1, 40), torch.zeros(2, 2, dtype=torch.int32), _i32(0, 0)
    with pytest.raises(ValueError, match="lens"):
        ga.kv_cache_append(k, k, *_cache(), table, two, tok_start=_i32(0, 25))
    assert ga.calls == []
    ga.kv_cache_append(k, k, *_cache(), table, two, tok_start=_i32(0, 25), lens=_i32(25, 15))
    ga.kv_cache_append(k, k, *_cache(), table, two, tok_start=_i32(0, 20), max_new=20)
    ga.kv_cache_append(k, k, *_cache(), table[:1], two[:1], tok_start=_i32(5))  # the rest of the row
    assert [(c[1].max_new, bool(c[1].lens)) for c in ga.calls] == [(40, True), (20, False), (40, False)]


def test_no_tokens_and_no_sequences(ga):
    """Nothing to append is no error, as no pairs to copy are none; neither is an empty batch."""
    table, none = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    ga.kv_cache_append(_kv(2, 0), _kv(2, 0), *_cache(), table, _i32(0, 0))
    ga.kv_cache_append(_kv(0, 5), _kv(0, 5), *_cache(), table[:0], none)
    ga.kv_cache_append(_kv(1, 0), _kv(1, 0), *_cache(), table, _i32(0, 0), lens=_i32(0, 0), tok_start=_i32(0, 0))
    ga.kv_cache_append(_kv(1, 7), _kv(1, 7), *_cache(), table[:0], none, lens=none, tok_start=none)
    for q in (torch.zeros(0, 1, 4, 64, dtype=torch.bfloat16), torch.zeros(0, 3, 4, 64, dtype=torch.bfloat16)):
        out, lse = ga.attn_decode(q, *_cache(), table[:0], none)
        assert out.shape == q.shape and lse.shape == (0, 4, q.shape[1])
    assert ga.calls == []
    for bad in (lambda: ga.kv_cache_append(_kv(2, 0), _kv(2, 0), *_cache(), table, _i32(0)),
                lambda: ga.kv_cache_append(_kv(0, 5, d=128), _kv(0, 5, d=128), *_cache(), table[:0], none),
                lambda: ga.attn_decode(torch.zeros(0, 1, 4, 64), *_cache(), table[:0], none)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("given,held", [(5, 5), (-1, -1), ((1 << 31) - 1, (1 << 31) - 1), (1 << 31, (1 << 31) - 1),
                                        (1 << 32, (1 << 31) - 1), ((1 << 40) + 3, (1 << 31) - 1),
                                        (-(1 << 32), -(1 << 31))])
def test_windows_past_32_bits_do_not_wrap(ga, given, held):
    """The C struct holds 32 bits: a window beyond them is as good as the largest (positions are
    below it), and one far below zero stays a refusal."""
    import workload
    q, k, v = workload.qkv(1, 16, 2, 1, 64)
    ids, pos = workload.segments(1, 16, None)
    p = ga._fwd_params(q, k, v, ids, pos, ids, pos, given, 0.1, q, q, False)
    assert p.window_left == held
    dp, _, _, _ = ga._decode_params(_kv(1, 1), *_cache(), torch.zeros(1, 2, dtype=torch.int32), _i32(1), given, 0,
                                    None, None, None, False)
    assert dp.window_left == held


@pytest.mark.parametrize("given,code", [(1 << 32, 2), ((1 << 64) + 5, 2), (-(1 << 32), 1), (-(1 << 64), 1)])
def test_kept_tokens_past_the_field_are_refused(ga, given, code):
    import workload
    q, k, v = workload.qkv(1, 16, 2, 1, 64)
    ids, pos = workload.segments(1, 16, None)
    p = ga._fwd_params(q, k, v, ids, pos, ids, pos, 4, 0.1, q, q, False, given)
    assert ga.lib().attn_fwd(ctypes.byref(p), None) == code
    dp, _, _, _ = ga._decode_params(_kv(1, 1), *_cache(), torch.zeros(1, 2, dtype=torch.int32), _i32(1), 4, given,
                                    None, None, None, False)
    assert ga.lib().attn_decode(ctypes.byref(dp), None) == code
