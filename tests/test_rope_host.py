"""Position rotation on the CPU: host checks of the C ABI (fake pointers, nothing is launched), the
binding's refusals and what it makes of its tensors, and the frequencies."""
import ctypes
import math

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


def _rope(pkg, **kw):
    p = pkg.RopeParams()
    p.q, p.k, p.q_out, p.k_out, p.pos = A, 2 * A, 3 * A, 4 * A, 5 * A
    p.tokens, p.h_q, p.h_k, p.d = 100, 8, 2, 128
    p.rotation.freqs, p.rotation.rot, p.rotation.amplitude = 6 * A, 128, 1.0
    for n, v in kw.items():
        setattr(p.rotation if n in ("freqs", "rot", "offset", "amplitude") else p, n, v)
    return pkg.lib().attn_rope(ctypes.byref(p), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k_out=None), 1), (dict(pos=None), 1), (dict(freqs=None), 1), (dict(q=A + 8), 1),
    (dict(k_out=A + 2), 1), (dict(pos=A + 2), 1), (dict(freqs=A + 4), 1), (dict(tokens=0), 1), (dict(h_q=-1), 1),
    (dict(h_q=0, h_k=0), 1), (dict(d=0), 1), (dict(d=264), 2), (dict(d=136), 2), (dict(h_q=65536), 2),
    (dict(rot=0), 1), (dict(rot=144), 1), (dict(rot=8), 2), (dict(rot=72, d=128), 2), (dict(offset=-8), 1),
    (dict(rot=64, offset=72), 1), (dict(rot=64, offset=4), 2), (dict(amplitude=-1.0), 1),
    (dict(amplitude=math.inf), 1), (dict(amplitude=math.nan), 1), (dict(q_stride=1000), 1), (dict(k_stride=260), 1),
    (dict(q_out_stride=-8), 1), (dict(tokens=1 << 40), 2), (dict(tokens=1 << 30, q_stride=1 << 30), 2),
    (dict(q_out=A + 4096), 1),              # rows of q over other rows of its output
    (dict(q_out=A, q_out_stride=2048), 1),  # the same first row, others apart
    (dict(k_out=A + 2048), 1), (dict(q_out=2 * A), 1), (dict(k_out=3 * A + 256), 1),
])
def test_refusals(pkg, kw, code):
    assert _rope(pkg, **kw) == code


def test_refuses_no_parameters(pkg):
    assert pkg.lib().attn_rope(None, None) == 1


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


POS = torch.zeros(2, 5, dtype=torch.int32)
F = torch.ones(32, dtype=torch.float64)


def test_binding_refuses(ga):
    q, k = _bf16(2, 5, 4, 64), _bf16(2, 5, 2, 64)
    bad = [
        (None, None, POS, F, {}), (q[0], None, POS, F, {}), (q.half(), None, POS, F, {}), (q, k.float(), POS, F, {}),
        (q, k[:, :4], POS, F, {}), (q, k, POS.long(), F, {}), (q, k, POS[:, :4], F, {}), (q, k, POS, F.float(), {}),
        (q, k, POS, F[None], {}), (q, k, POS, F, dict(amplitude=0.0)), (q, k, POS, F, dict(amplitude=math.nan)),
        (q, None, POS, F, dict(k_out=k)), (q, k, POS, F, dict(q_out=q[:, :, :2])), (q, k, POS, F, dict(k_out=k.float())),
        (q[..., ::2], None, POS, F, {}), (q[:, :1].expand(2, 5, 4, 64), None, POS, F, {}),
        (q.transpose(1, 2).contiguous().transpose(1, 2), None, POS, F, {}),
    ]
    for x, y, pos, f, kw in bad:
        with pytest.raises(ValueError):
            ga.rope(x, y, pos, f, **kw)
    assert ga.calls == []


def test_binding_refuses_host_tensors(pkg):
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rope(_bf16(2, 5, 4, 64), None, POS, F)


def test_binding_passes_layouts(ga):
    qkv = _bf16(2, 5, 8, 64)
    q, k = qkv[:, :, :4], qkv[:, :, 4:6]
    got = ga.rope(q, k, POS, F[:16], offset=32, interleaved=True, amplitude=1.5, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    name, p, _ = ga.calls.pop()
    assert name == "attn_rope"
    assert (p.q, p.q_out, p.k, p.k_out) == (qkv.data_ptr(),) * 2 + (k.data_ptr(),) * 2
    assert (p.q_stride, p.q_out_stride, p.k_stride, p.k_out_stride) == (512,) * 4
    assert (p.tokens, p.h_q, p.h_k, p.d, p.fp32, p.inverse) == (10, 4, 2, 64, 0, 0)
    r = p.rotation
    assert (r.rot, r.offset, r.interleaved, r.amplitude) == (32, 32, 1, 1.5)
    ga.rope_bwd(None, k.float(), POS, F)
    _, p, _ = ga.calls.pop()
    assert (p.q, p.h_q, p.h_k, p.fp32, p.inverse, p.k_out_stride) == (None, 0, 2, 1, 1, 128)
    assert ga.rope(_bf16(2, 0, 4, 64), None, POS[:, :0], F)[0].shape == (2, 0, 4, 64)
    assert ga.calls == []


def test_frequencies(pkg):
    f = pkg.rope_frequencies(64, 500.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    want = [500.0 ** (-2 * i / 64) for i in range(32)]
    assert torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(pkg.rope_frequencies(64, 500.0, factor=8.0, device="cpu"), f / 8, rtol=1e-14)
    g = pkg.rope_frequencies(64, 500.0, factor=8.0, method="base", device="cpu")
    assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 8, rel_tol=1e-12)
    g = pkg.rope_frequencies(64, 500.0, factor=8.0, method="parts", trained=1000, fast=30.0, slow=2.0, device="cpu")
    for i in range(32):
        keep = min(max((want[i] * 1000 / (2 * math.pi) - 2) / 28, 0), 1)
        assert math.isclose(g[i], want[i] * keep + want[i] / 8 * (1 - keep), rel_tol=1e-12)
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / 8, rel_tol=1e-12)
    for kw in (dict(rot=7), dict(rot=0), dict(rot=64, factor=0.0), dict(rot=64, base=-1.0), dict(rot=64, method="x")):
        with pytest.raises(ValueError):
            pkg.rope_frequencies(device="cpu", **kw)
