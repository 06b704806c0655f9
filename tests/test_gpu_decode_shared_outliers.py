"""Decoding behind shared pages where one value of each query row is far larger than the others and the keys are
zero, or next to it, in its channel, so that the small values alone decide the scores.

Tolerances, e being the error of a score:
* fp32 sums: d 2^-24 of their terms' magnitudes.
* q: at coarsest (the kernel of many rows) exact down to 2^-23 of the row's largest value, and below that off by
  no more than 2^-17 where the largest value is above 7 / 8 of 2^15: 2^-31 of it is a bound.
A weight is then off by 2 e of itself (its own score and the sum's), lse by e, beside 2^-10 of sum P |v| and 2e-4 for
everything else as in test_gpu_decode_shared."""
import numpy as np
import pytest
import torch

from tests import paged
from tests.paged import np64
from tests.test_gpu_decode_shared import _case, _run, _want, ga  # noqa: F401

pytestmark = pytest.mark.gpu


def _outliers(m, sq, hq, d, power, near, seed):
    c = _case([m], [6], [1, 40, 100], sq, hq, 1, d, 32, seed=seed)
    g = torch.Generator().manual_seed(seed)
    channel = 5 + 17 * (seed % 3)
    sign = torch.randint(0, 2, c["q"].shape[:3], generator=g) * 2 - 1
    c["q"][..., channel] = (sign * 2.0 ** power * 1.375).to(torch.bfloat16)
    unused = c["k"][..., channel] == 0x7f  # (slots that hold nothing keep their NaN)
    # zeros, or the four codes of least magnitude but for them, -2^-9 .. 2^-8
    small = torch.tensor([0x01, 0x81, 0x02, 0x82], dtype=torch.uint8)[torch.randint(0, 4, unused.shape, generator=g)]
    c["k"][..., channel] = torch.where(unused, torch.full_like(small, 0x7f), small if near else torch.zeros_like(small))
    return c


def _error_of_scores(c):
    d = c["q"].shape[3]
    q = np.abs(np64(c["q"])).reshape(-1, d)
    used = paged.from_e4m3(paged.raw(c["k"])) * c["ks"].numpy().astype(np.float64)[:, :, None, None]
    k = np.abs(np.nan_to_num(used)).reshape(-1, d)
    return d ** -0.5 * (d * 2.0 ** -24 * (q @ k.T).max() + 2.0 ** -31 * q.max() * k.sum(1).max())


# sequences, drafted tokens, query heads: 4, 24, 40, 100, 140 and 300 rows
ROWS = [(4, 1, 1), (3, 2, 4), (5, 1, 8), (25, 1, 4), (35, 1, 4), (30, 5, 2)]


@pytest.mark.parametrize("m,sq,hq", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [6, 10, 14])
@pytest.mark.parametrize("near", [False, True])
def test_values_far_below_their_rows_largest(ga, m, sq, hq, d, power, near):
    c = _outliers(m, sq, hq, d, power, near, seed=d + power + m)
    e = _error_of_scores(c)
    assert e < 0.02
    ro, rl, mag = _want(c, -1, 0)
    out, lse = _run(ga, c, -1, 0, out_fp32=True)
    assert np.all(np.abs(np64(lse) - rl) <= 2e-4 + e)
    assert np.all(np.abs(np64(out) - ro) <= (2.0 ** -10 + 2 * e + 2 * e * e) * mag)
