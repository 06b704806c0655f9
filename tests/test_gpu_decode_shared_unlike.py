"""Windows over groups whose members' lengths lie far apart: the keys that some member sees reach over far more than
one window, and are shared out to as many CTAs as without one."""
import pytest
import torch

from tests.test_gpu_decode_shared import DEV, INT, _case, _check, _run, _want, ga  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [2, 10, 40, 100])  # 8 and 16 rows, 64 and 128 rows a CTA
def test_the_span_of_a_group_is_shared_out(ga, m):
    """d 256: both lists take the same kernel for as many rows; a window of 12000 tokens bounds the
    runs that a sequence's own keys can be cut into, but not a group's."""
    page, table = 64, torch.zeros(m, 2048, **INT)
    q = torch.zeros(m, 1, 1, 256, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, 1, page, 256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scale = torch.ones(1, 1, device=DEV)
    lens, shared = torch.full((m,), 100000, **INT), torch.full((m,), 1500, **INT)
    lens[0] = 13000

    def need(window, most):
        return ga.workspace_bytes_decode_shared(q, k, k, scale, scale, table, lens, shared, max_group=most, window_left=window)

    whole, cut = need(-1, m), need(12000, m)
    # with a group of two at most both lists have items of up to 8 rows
    own = need(-1, 2) // 2
    assert whole > own and cut >= whole - own


@pytest.mark.parametrize("m", [2, 10, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sink", [0, 70])
def test_members_far_apart(ga, m, d, sink):
    c = _case([m], [300], [-9000, 1, -300, 60], 1, 1, 1, d, 32, seed=m + d)
    _check(_run(ga, c, 200, sink, out_fp32=True), _want(c, 200, sink), False)
