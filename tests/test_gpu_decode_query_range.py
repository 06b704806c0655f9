"""Decoding with query rows at both ends of bf16's range (K's scales bring the scores back), rows of zeros among them,
and rows of one sequence that lie far apart from each other.  Tolerances as in test_gpu_decode_shared_outliers."""
import numpy as np
import pytest
import torch

from tests import test_gpu_decode as plain, test_gpu_decode_shared as shared
from tests.paged import np64
from tests.test_gpu_decode_shared import ga  # noqa: F401
from tests.test_gpu_decode_shared_outliers import _error_of_scores

pytestmark = pytest.mark.gpu


def _scale(c, power):
    """q times 2^power, K's scales by its inverse; every fifth row of q is zero, every seventh 2^-9 of that."""
    n, sq, hq, _ = c["q"].shape
    r = torch.arange(n * sq * hq).reshape(n, sq, hq, 1)
    q = c["q"].double() * 2.0 ** power
    q = torch.where(r % 7 == 3, q * 2.0 ** -9, torch.where(r % 5 == 2, q * 0.0, q))
    c["q"], c["ks"] = q.to(torch.bfloat16), (c["ks"].double() * 2.0 ** -power).float()
    assert bool(torch.isfinite(c["q"]).all())


def _check(got, want, e):
    ro, rl, mag = want
    out, lse = np64(got[0]), np64(got[1])
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert e < 0.02 and np.all(np.abs(lse[fin] - rl[fin]) <= 2e-4 + e)
    assert np.all(np.abs(out - ro) <= (2.0 ** -10 + 2 * e + 2 * e * e) * mag)


@pytest.mark.parametrize("power", [-110, -60, 60, 115])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m,sq,hq", [(4, 1, 2), (3, 2, 4), (5, 1, 8), (25, 1, 4), (30, 5, 2)])
def test_decode_shared(ga, power, d, m, sq, hq):
    c = shared._case([m], [6], [1, 40, -20, 100], sq, hq, 1, d, 32, seed=d + m)
    _scale(c, power)
    _check(shared._run(ga, c, -1, 0, out_fp32=True), shared._want(c, -1, 0), _error_of_scores(c))


@pytest.mark.parametrize("power", [-110, -60, 60, 115])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sq,hq", [(1, 4), (2, 12), (5, 8), (6, 20)])
@pytest.mark.parametrize("wide", [False, True])
def test_decode(ga, power, d, sq, hq, wide):
    c = plain._case(3, sq, hq, 1, d, 16, [70, 300, 1], seed=d + sq)
    _scale(c, power)
    want = plain._want(c, -1, 0, d ** -0.5)
    _check(plain._run(ga, plain._wide(c, 16) if wide else c, -1, 0, d ** -0.5, out_fp32=True), want, _error_of_scores(c))
