"""Position rotation against the plain fp64 form.

Tolerance.  The kernel's cos and sin: the angle's rest is cut at 2^-32 of a turn (1.5e-9), its conversion
and the product with 2 pi / 2^32 round twice (2 * 2^-24 of at most pi / 4), the series' last steps and the
amplitude once each (3 * 2^-24), the term left out is below 2e-9: together under 2^-21 of the amplitude.
A product, a fused product and sum round by 2^-24 each.  So |y| is off by at most (2^-21 + 2^-23)
amplitude (|x1| + |x2|) < 2^-20 of that, and its rounding, 2^-24 of itself in fp32 and 2^-8 in bf16."""
import numpy as np
import pytest
import torch

from tests import rotation
from tests.paged import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _normal(*shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def _close(got, want, mag, dtype):
    got = np64(got)
    half = 2.0 ** (-8 if dtype == torch.bfloat16 else -24)
    assert np.all(np.abs(got - want) <= 2.0 ** -20 * mag + half * np.abs(want))


CASES = [
    # b, s, hq, hk, d, rot, offset, interleaved, amplitude, positions up to
    (1, 1, 1, 1, 64, 64, 0, False, 1.0, 0),
    (2, 3, 5, 1, 64, 16, 0, True, 1.0, 100),
    (3, 7, 4, 2, 128, 128, 0, False, 1.25, 1000003),
    (1, 33, 9, 3, 128, 128, 0, True, 1.0, (1 << 31) - 40),
    (1, 65, 2, 2, 192, 64, 128, True, 0.7, 5000),
    (2, 19, 7, 1, 192, 192, 0, False, 1.0, 70000),
    (1, 40, 3, 1, 256, 256, 0, False, 1.0, 4000),
    (1, 40, 6, 2, 256, 64, 24, False, 1.1, 4000),
    (1, 21, 3, 0, 256, 240, 8, True, 1.0, 4000),
    (1, 500, 40, 8, 128, 96, 16, False, 1.0, 131072),
    (5, 1001, 4, 2, 64, 48, 8, True, 1.0, 131072),
    (1, 30, 2, 1, 16, 16, 0, False, 1.0, 50),
    (32, 1, 32, 8, 128, 128, 0, False, 1.0, 1000000),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_rope(ga, case, dtype):
    b, s, hq, hk, d, rot, offset, inter, amp, top = case
    q, k = _normal(b, s, hq, d, seed=1, dtype=dtype), (_normal(b, s, hk, d, seed=2, dtype=dtype) if hk else None)
    g = torch.Generator().manual_seed(3)
    pos = (torch.randint(0, top + 1, (b, 1), generator=g) + torch.arange(s)).to(torch.int32)
    pos[0, s // 2] = -5 - top // 2
    f = ga.rope_frequencies(rot, 10000.0, device=DEV)
    how = dict(interleaved=inter, offset=offset, amplitude=amp)
    for call, inverse in ((ga.rope, False), (ga.rope_bwd, True)):
        got = call(q, k, pos.to(DEV), f, **how)
        for x, y in zip((q, k), got):
            if x is None:
                assert y is None
                continue
            want, mag = rotation.turn(np64(x), pos.numpy(), f.cpu().numpy(), inverse=inverse, **how)
            assert y.dtype == dtype
            _close(y, want, mag, dtype)
            other = [i for i in range(d) if not offset <= i < offset + rot]
            assert torch.equal(y[..., other], x[..., other])
        # in place the same, bit for bit
        out = ("q_out", "k_out") if call is ga.rope else ("dq_out", "dk_out")
        x, y = q.clone(), None if k is None else k.clone()
        kw = {out[0]: x} if y is None else {out[0]: x, out[1]: y}
        call(x, y, pos.to(DEV), f, **how, **kw)
        assert torch.equal(x, got[0]) and (y is None or torch.equal(y, got[1]))


def test_frequencies_at_their_borders(ga):
    """Frequencies of several turns a position, negative, tiny, zero and subnormal ones."""
    f = torch.tensor([100.0, 7.5, -3.0, 2 * np.pi, np.pi, 1e-9, 1e-300, 0.0, 5e-324, 1e6, 0.5, 1.0, 2.0 ** -30, 3e-5, -1e-3,
                      6.0], dtype=torch.float64)
    pos = torch.tensor([[0, 1, -1, 12345, (1 << 31) - 1, -(1 << 31), 65536]], dtype=torch.int32)
    x = _normal(1, 7, 2, 32, seed=4, dtype=torch.float32)
    got, _ = ga.rope(x, None, pos.to(DEV), f.to(DEV))
    # (numpy's long double carries 100 * 2^31 radians to 2^-26 of one, 1e6 * 2^31 to 2^-13: those pairs
    # are compared at the small positions only)
    want, mag = rotation.turn(np64(x), pos.numpy(), f.numpy())
    for i, top in ((0, 1 << 17), (9, 1 << 14)):
        far = np.abs(pos.numpy().astype(np.int64))[0] > top
        for j in (i, i + 16):
            mag[0, far, :, j] = np.inf
    got = np64(got)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= 2.0 ** -20 * mag + 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("inter", [False, True])
def test_values_that_are_not_finite_stay_in_their_pair(ga, inter):
    x = _normal(1, 4, 2, 64, seed=5, dtype=torch.bfloat16)
    bad = x.clone()
    bad[0, 1, 0, 3], bad[0, 2, 1, 40], bad[0, 3, 0, 60] = float("nan"), float("inf"), float("nan")
    pos = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    f = ga.rope_frequencies(32, device=DEV)  # the first 32 of 64 turn
    y, z = (ga.rope(t, None, pos, f, interleaved=inter)[0] for t in (x, bad))
    same = torch.ones_like(x, dtype=torch.bool)
    same[0, 1, 0, 3] = same[0, 1, 0, 2 if inter else 19] = same[0, 2, 1, 40] = same[0, 3, 0, 60] = False
    assert torch.equal(y[same], z[same])
    assert torch.isnan(z[0, 1, 0, 3]) and torch.isnan(z[0, 1, 0, 2 if inter else 19])
    assert z[0, 2, 1, 40] == float("inf") and torch.isnan(z[0, 3, 0, 60])


def test_packed_rows(ga):
    """q and k as columns of one [b, s, Hq + 2 Hkv, d]: in place, v untouched; and into another buffer's."""
    qkv = _normal(2, 37, 12, 128, seed=6, dtype=torch.bfloat16)
    before, other = qkv.clone(), torch.zeros_like(qkv)
    pos = torch.arange(37, dtype=torch.int32, device=DEV).repeat(2, 1)
    f = ga.rope_frequencies(128, device=DEV)
    want = ga.rope(qkv[:, :, :8].contiguous(), qkv[:, :, 8:10].contiguous(), pos, f)
    ga.rope(qkv[:, :, :8], qkv[:, :, 8:10], pos, f, q_out=other[:, :, 2:10], k_out=other[:, :, 10:])
    assert torch.equal(other[:, :, 2:10], want[0]) and torch.equal(other[:, :, 10:], want[1])
    assert torch.count_nonzero(other[:, :, :2]) == 0 and torch.equal(qkv, before)
    ga.rope(qkv[:, :, :8], qkv[:, :, 8:10], pos, f, q_out=qkv[:, :, :8], k_out=qkv[:, :, 8:10])
    assert torch.equal(qkv[:, :, :8], want[0]) and torch.equal(qkv[:, :, 8:10], want[1])
    assert torch.equal(qkv[:, :, 10:], before[:, :, 10:])


def test_rows_past_32_bits(ga):
    """Token rows 2^31 + 64 values apart: the third begins past 2^32."""
    far = torch.empty(2 * ((1 << 31) + 64) + 64, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(far, (1, 3, 1, 64), (0, (1 << 31) + 64, 64, 1))
    x.copy_(_normal(1, 3, 1, 64, seed=7, dtype=torch.bfloat16))
    pos = torch.tensor([[5, 6, 7]], dtype=torch.int32, device=DEV)
    f = ga.rope_frequencies(64, device=DEV)
    want, _ = ga.rope(x.contiguous(), None, pos, f)
    ga.rope(x, None, pos, f, q_out=x)
    assert torch.equal(x, want)


def test_gradient_against_differences(ga):
    """The map is linear: <g, rope(x + h) - rope(x)> = <rope_bwd(g), h>, for q and k at once.  fp32: each side's
    terms are off by 2^-20 of |g| |h| (and rope(x) by that of |x|, h being as large)."""
    for inter in (False, True):
        how = dict(interleaved=inter, offset=16, amplitude=1.3)
        f = ga.rope_frequencies(32, device=DEV)
        pos = torch.randint(0, 9000, (2, 50), dtype=torch.int32, device=DEV)
        q, h, g = (_normal(2, 50, 3, 64, seed=s, dtype=torch.float32) for s in (8, 9, 10))
        k, hk, gk = (_normal(2, 50, 1, 64, seed=s, dtype=torch.float32) for s in (11, 12, 13))
        y0, y1 = ga.rope(q, k, pos, f, **how), ga.rope(q + h, k + hk, pos, f, **how)
        b = ga.rope_bwd(g, gk, pos, f, **how)
        for y, z, grad, step, x, back in ((y0[0], y1[0], g, h, q, b[0]), (y0[1], y1[1], gk, hk, k, b[1])):
            left, right = (grad.double() * (z.double() - y.double())).sum(), (back.double() * step.double()).sum()
            size = 2 * 1.3 * (grad.abs().max() * (x.abs() + step.abs()).max()).double() * grad.numel()
            assert abs(left - right) <= 4 * 2.0 ** -20 * size


def test_streams_graphs_and_no_tokens(ga):
    x = _normal(2, 64, 4, 128, seed=14, dtype=torch.bfloat16)
    pos = torch.arange(64, dtype=torch.int32, device=DEV).repeat(2, 1)
    f = ga.rope_frequencies(128, device=DEV)
    want, _ = ga.rope(x, None, pos, f)
    out = torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ga.rope(x, None, pos, f, q_out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ga.rope(x, None, pos, f, q_out=out)
        ga.rope_bwd(out, None, pos, f, dq_out=out)
    out.zero_()
    pos.add_(77)
    graph.replay()
    back = ga.rope_bwd(ga.rope(x, None, pos, f)[0], None, pos, f)[0]
    assert torch.equal(out, back)
    empty, none = ga.rope(x[:, :0], None, pos[:, :0].contiguous(), f)
    assert empty.shape == (2, 0, 4, 128) and none is None
