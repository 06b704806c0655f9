"""What rope_frequencies refuses (CPU): arguments whose frequencies would be NaN, infinite or zero for all pairs."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def pkg():
    import long_context_attention_attn_gb300 as pkg
    return pkg


@pytest.mark.parametrize("kw", [
    dict(method="parts", fast=4.0, slow=4.0), dict(method="parts", fast=1.0, slow=32.0),
    dict(method="parts", fast=math.nan), dict(method="parts", slow=math.nan),
    dict(method="parts", slow=-math.inf), dict(method="parts", trained=0), dict(method="parts", trained=-4096),
    dict(method="parts", trained=math.inf), dict(method="parts", trained=math.nan),
    dict(factor=math.inf), dict(factor=math.nan), dict(factor=math.inf, method="parts"), dict(base=math.inf),
    dict(base=math.nan), dict(factor=1e300, method="base"), dict(factor=1e200, base=1e200, method="base"),
])
def test_refusals(pkg, kw):
    with pytest.raises(ValueError):
        pkg.rope_frequencies(32, device="cpu", **kw)


@pytest.mark.parametrize("kw", [
    dict(), dict(method="parts"), dict(method="parts", fast=4.0, slow=0.0), dict(method="parts", fast=math.inf),
    dict(method="parts", factor=8.0, trained=512.5),
    dict(method="base", factor=4.0), dict(factor=0.5), dict(fast=1.0, slow=1.0, trained=0),  # (not used)
])
def test_finite(pkg, kw):
    f = pkg.rope_frequencies(32, device="cpu", **kw)
    assert f.shape == (16,) and f.dtype == torch.float64 and bool((f.isfinite() & (f > 0)).all())


@pytest.mark.parametrize("rot", [2, 4, 256])
def test_parts_mixes_in_proportion(pkg, rot):
    kw = dict(base=10000.0, factor=4.0)
    plain = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    got = pkg.rope_frequencies(rot, method="parts", trained=4096, fast=32.0, slow=1.0, device="cpu", **kw).tolist()
    for f, g in zip(plain, got):
        keep = min(max((f * 4096 / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0)
        assert abs(g - (f * keep + f / 4.0 * (1.0 - keep))) <= 1e-14 * f
