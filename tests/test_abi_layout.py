"""Callers built against the header as it was before sink_tokens: the parameters that they pass lie
where the library reads them (CPU; fake pointers, nothing is launched)."""
import ctypes

import pytest

vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class Fwd(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("q", "k", "v", "q_segment_ids", "q_segment_pos", "kv_segment_ids",
                                  "kv_segment_pos")]
    _fields_ += [(n, i64) for n in ("b", "s_q", "s_kv", "h_q", "h_kv", "d")]
    _fields_ += [("window_left", i32), ("window_right", i32), ("scale", ctypes.c_float), ("out_fp32", i32),
                 ("out", vp), ("lse", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t),
                 ("merge_into_out", i32), ("out_final", vp), ("kv_token_stride", i64), ("d_v", i64)]


class Bwd(ctypes.Structure):
    _fields_ = [("fwd", Fwd), ("dout", vp), ("dq", vp), ("dk", vp), ("dv", vp), ("accumulate_fp32", i32),
                ("deterministic", i32), ("kernel_events", vp * 2), ("delta", vp)]


class Behind(ctypes.Structure):
    """What lies behind a caller's struct is not the library's to read."""
    _fields_ = [("fwd", Fwd), ("other", i64)]


@pytest.fixture(scope="module")
def ga():
    import __graft_entry__
    __graft_entry__.build()
    import long_context_attention_attn_gb300 as pkg
    return pkg


def _fill(p):
    fake = 1 << 20
    for f in ("q", "k", "v", "q_segment_ids", "q_segment_pos", "kv_segment_ids", "kv_segment_pos", "out", "lse",
              "workspace"):
        setattr(p, f, fake)
    p.b, p.s_q, p.s_kv, p.h_q, p.h_kv, p.d = 2, 4096, 4096, 16, 2, 128
    p.window_left, p.scale = 1024, 0.1


def test_forward(ga):
    old, new = Behind(other=-1), ga.FwdParams()
    _fill(old.fwd)
    _fill(new)
    size = lambda p: ga.lib().attn_fwd_workspace_bytes(ctypes.cast(ctypes.pointer(p), ctypes.POINTER(ga.FwdParams)))
    assert size(old) == size(new) > 0
    assert ctypes.sizeof(ga.FwdParams) == ctypes.sizeof(Fwd)
    for name, _ in Fwd._fields_:
        assert getattr(Fwd, name).offset == getattr(ga.FwdParams, name).offset


def test_backward(ga):
    size = lambda p: ga.lib().attn_bwd_workspace_bytes(ctypes.cast(ctypes.pointer(p), ctypes.POINTER(ga.BwdParams)))
    run = lambda p: ga.lib().attn_bwd(ctypes.cast(ctypes.pointer(p), ctypes.POINTER(ga.BwdParams)), None)
    for det in (0, 1):
        old, new = Bwd(), ga.BwdParams()
        for p in (old, new):
            _fill(p.fwd)
            p.fwd.workspace_bytes = 1 << 40
            p.dout, p.dq, p.dk, p.dv = 1 << 21, 1 << 22, 1 << 23, 1 << 24
            p.deterministic = det
        assert size(old) == size(new) > 0
        old.delta = (1 << 40) + 2  # misaligned
        assert run(old) == ga.ATTN_ERR_INVALID_ARG
        old.delta, old.dv = None, None
        assert run(old) == ga.ATTN_ERR_INVALID_ARG
    for name, _ in Bwd._fields_:
        assert getattr(Bwd, name).offset == getattr(ga.BwdParams, name).offset


def test_kept_tokens_reach_the_library(ga):
    """The field sits in what was padding: without it, none; out of range, refused; and the
    backward's scratch for key tiles that hold some."""
    b = ga.BwdParams()
    _fill(b.fwd)
    plain = ga.lib().attn_bwd_workspace_bytes(ctypes.byref(b))
    b.fwd.sink_tokens = 4
    assert ga.lib().attn_bwd_workspace_bytes(ctypes.byref(b)) > plain > 0
    b.fwd.sink_tokens = -1
    assert ga.lib().attn_bwd_workspace_bytes(ctypes.byref(b)) == 0
