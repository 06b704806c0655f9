"""A query row that holds an infinity: its scores are infinities and NaN (0 * infinity), so every result of the row is
NaN where it sees a key, also where all of its scores are minus infinity, which looks like a row without keys.
Other rows have no trace of it, and rows without keys stay 0 and minus infinity."""
import numpy as np
import pytest
import torch

from tests import paged, test_gpu_decode as plain, test_gpu_decode_shared as shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ga():
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _one_sign(c, channel):
    """K positive in the channel, wherever a slot holds a token."""
    k = c["k"][..., channel]
    c["k"][..., channel] = torch.where(k == 0x7f, k, (k & 0x3f) | 0x20)


def _place(c, channel, value):
    """Infinities of one sign in every third row of q; their mask."""
    n, sq, hq, _ = c["q"].shape
    rows = (torch.arange(n * sq * hq) % 3 == 1).reshape(n, sq, hq)
    c["q"][..., channel] = torch.where(rows, torch.full_like(c["q"][..., channel], value), c["q"][..., channel])
    return rows.numpy()


def _check(got, want, rows):
    (out, lse), (ro, rl, mag) = got, want
    out, lse = paged.np64(out), np.swapaxes(paged.np64(lse), 1, 2)
    rl = np.swapaxes(rl, 1, 2)
    sees = ~np.isneginf(rl)
    assert (rows & sees).any() and (~rows & sees).any()
    assert np.isnan(out[rows & sees]).all() and np.isnan(lse[rows & sees]).all()
    assert (out[~sees] == 0).all() and np.isneginf(lse[~sees]).all()
    ok = ~rows & sees
    assert np.all(np.abs(lse[ok] - rl[ok]) <= 2e-4) and np.all(np.abs(out[ok] - ro[ok]) <= 2.0 ** -10 * mag[ok])


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
# query tokens, query heads: up to 8 and 16 rows, 24, 40 and 120
@pytest.mark.parametrize("sq,hq", [(1, 4), (1, 12), (2, 12), (5, 8), (6, 20)])
@pytest.mark.parametrize("wide", [False, True])
def test_decode(ga, value, d, sq, hq, wide):
    c = plain._case(5, sq, hq, 1, d, 16, [1, 2, 3, 70, 0], seed=d + sq)
    _one_sign(c, 3)
    want = plain._want(c, -1, 0, d ** -0.5)
    rows = _place(c, 3, value)
    _check(plain._run(ga, plain._wide(c, 16) if wide else c, -1, 0, d ** -0.5, out_fp32=True), want, rows)


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m,sq,hq", [(7, 1, 1), (7, 1, 4), (11, 1, 4), (30, 1, 4), (50, 1, 4)])
@pytest.mark.parametrize("most", [None, 1])
def test_decode_shared(ga, value, d, m, sq, hq, most):
    """Sequences that see one to three of the shared keys, all of them, or none."""
    c = shared._case([m], [4], [-63, -62, -61, 1, 40, -64], sq, hq, 1, d, 16, seed=d + m)
    _one_sign(c, 3)
    want = shared._want(c, -1, 0)
    rows = _place(c, 3, value)
    _check(shared._run(ga, c, -1, 0, out_fp32=True, max_group=most or m), want, rows)
