"""First tokens that stay visible behind the sliding window (sink_tokens), CPU side: the
oracle's mask against its definition and its gradient against differences, and the
library's host checks."""
import ctypes

import numpy as np
import pytest

import workload
from oracle import attention as A


@pytest.mark.parametrize("window,sink", [(-1, 3), (0, 0), (0, 1), (5, 2), (7, 100)])
def test_visible_follows_the_definition(window, sink):
    ids, pos = workload.random_segments(1, 40, seed=3)
    ids, pos = ids[0].numpy(), pos[0].numpy()
    got = A.visible(ids, pos, ids, pos, window, sink)
    for i in range(40):
        for j in range(40):
            near = window < 0 or pos[i] - pos[j] <= window or pos[j] < sink
            assert got[i, j] == (ids[i] == ids[j] != 0 and pos[j] <= pos[i] and near)


def test_oracle_gradient_matches_differences():
    """Central differences of vdot(out, dout) in fp64: with steps of 1e-5 the difference is
    off by its third derivative times 1e-10 and by rounding, 1e-16 / 1e-5; 1e-7 covers both."""
    rng = np.random.default_rng(0)
    s, hq, hkv, d = 13, 4, 2, 4
    ids, pos = workload.random_segments(1, s, seed=8, max_segments=2)
    x = [rng.standard_normal((1, s, h, d)) for h in (hq, hkv, hkv)]
    dout = rng.standard_normal((1, s, hq, d))
    kw = dict(sink_tokens=2)
    grads = A.attn_bwd(*x, dout, ids, pos, ids, pos, 3, 0.5, **kw)
    for which in range(3):
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in x[which].shape)
            loss = []
            for step in (1e-5, -1e-5):
                y = [t.copy() for t in x]
                y[which][at] += step
                out, _ = A.attn_fwd(*y, ids, pos, ids, pos, 3, 0.5, **kw)
                loss.append(float((out * dout).sum()))
            assert abs((loss[0] - loss[1]) / 2e-5 - grads[which][at]) < 1e-7


@pytest.fixture(scope="module")
def ga():
    import __graft_entry__
    __graft_entry__.build()
    import long_context_attention_attn_gb300 as pkg
    return pkg


@pytest.mark.parametrize("sink,code", [(-1, 1), ((1 << 30) + 1, 2)])
def test_sink_tokens_out_of_range_is_refused(ga, sink, code):
    p = ga.FwdParams()
    fake = 1 << 20  # aligned non-null fake device address; never dereferenced
    for f in ("q", "k", "v", "q_segment_ids", "q_segment_pos", "kv_segment_ids", "kv_segment_pos", "out",
              "lse", "workspace"):
        setattr(p, f, fake)
    p.b, p.s_q, p.s_kv, p.h_q, p.h_kv, p.d = 1, 256, 256, 4, 2, 64
    p.window_left, p.scale, p.workspace_bytes = 16, 0.125, 1 << 30
    p.sink_tokens = 1 << 30
    assert ga.lib().attn_fwd_workspace_bytes(ctypes.byref(p)) > 0
    p.sink_tokens = sink
    assert ga.lib().attn_fwd_workspace_bytes(ctypes.byref(p)) == 0
    assert ga.lib().attn_fwd(ctypes.byref(p), None) == code
    b = ga.BwdParams()
    b.fwd = p
    b.dout = b.dq = b.dk = b.dv = fake
    assert ga.lib().attn_bwd(ctypes.byref(b), None) == code


