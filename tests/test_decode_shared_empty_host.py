"""Decoding of no sequences behind shared pages (CPU): outputs of the right shapes, and nothing is launched."""
import pytest
import torch

from tests.test_decode_shared_host import ga, pkg  # noqa: F401


@pytest.mark.parametrize("sq,hq", [(1, 4), (3, 2)])
def test_shapes_of_no_sequences(ga, sq, hq):
    cache = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8) for _ in range(2)] + [torch.zeros(4, 2) for _ in range(2)]
    q, none = torch.zeros(0, sq, hq, 64, dtype=torch.bfloat16), torch.zeros(0, dtype=torch.int32)
    out, lse = ga.attn_decode_shared(q, *cache, torch.zeros(0, 2, dtype=torch.int32), none, none)
    assert out.shape == (0, sq, hq, 64) and lse.shape == (0, hq, sq)
    assert ga.calls == []
