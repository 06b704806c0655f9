"""First tokens that stay visible behind the sliding window, forward and backward, against
the fp64 oracle.  Tolerances: tests/parity.py (the hot path's)."""
import numpy as np
import pytest
import torch

import workload
from oracle import attention as A
from oracle import plan as P
from tests.parity import check_grad, check_lse, check_out

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(b, s, hq, hkv, d, dv, packing, seed):
    q, k, v, dout = workload.qkv(b, s, hq, hkv, d, seed=seed, with_dout=True, dv=dv)
    if packing == "one":
        ids, pos = workload.segments(b, s, None)
    else:
        ids, pos = workload.random_segments(b, s, seed=seed, max_segments=3)
    return dict(q=q, k=k, v=v, dout=dout, ids=ids, pos=pos)


def _gpu(ga, x, window, sink, scale, det=False):
    g = {n: t.to(DEV) for n, t in x.items()}
    kw = dict(window_left=window, sink_tokens=sink, scale=scale, check_status=True)
    out, lse = ga.attn_fwd(g["q"], g["k"], g["v"], g["ids"], g["pos"], **kw)
    grads = ga.attn_bwd(g["q"], g["k"], g["v"], out, lse, g["dout"], g["ids"], g["pos"], deterministic=det, **kw)
    return out, lse, grads


@pytest.mark.parametrize("b,s,hq,hkv,d,dv,window,sink,packing", [
    (1, 1, 2, 1, 64, 64, 0, 1, "one"),          # one token
    (1, 129, 2, 2, 64, 64, 0, 1, "one"),        # each token sees itself and the first
    (1, 700, 4, 2, 64, 64, 16, 4, "one"),       # tiles between the first and the window are skipped
    (1, 700, 4, 2, 128, 128, 100, 130, "one"),  # the kept tokens end inside the second tile
    (1, 900, 2, 1, 128, 128, 127, 128, "one"),  # a whole kept tile, seen without a mask
    (2, 640, 8, 2, 128, 128, 40, 7, "packed"),
    (1, 515, 5, 1, 64, 64, 3, 600, "packed"),   # more kept tokens than there are
    (1, 600, 4, 2, 256, 256, 50, 5, "packed"),
    (1, 600, 4, 2, 192, 128, 50, 5, "packed"),
])
@pytest.mark.parametrize("det", [False, True])
def test_forward_and_backward(b, s, hq, hkv, d, dv, window, sink, packing, det):
    import long_context_attention_attn_gb300 as ga
    x = _inputs(b, s, hq, hkv, d, dv, packing, seed=s + d)
    scale = d ** -0.5
    out, lse, grads = _gpu(ga, x, window, sink, scale, det)
    ro, rl = A.attn_fwd(x["q"], x["k"], x["v"], x["ids"], x["pos"], x["ids"], x["pos"], window, scale,
                        sink_tokens=sink)
    check_out(out.cpu(), ro)
    check_lse(lse.cpu(), rl)
    ref = A.attn_bwd(x["q"], x["k"], x["v"], x["dout"], x["ids"], x["pos"], x["ids"], x["pos"], window, scale,
                     sink_tokens=sink)
    for name, got, want in zip(("dq", "dk", "dv"), grads, ref):
        check_grad(got.cpu(), want, name)


@pytest.mark.parametrize("window,sink,same", [(40, 0, (40, 0)), (-1, 9, (-1, 0)), (40, 1 << 30, (-1, 0))])
def test_same_as_the_mask_it_amounts_to(window, sink, same):
    """No kept tokens is the window alone, any without a window and all of them is causal:
    the same tiles with the same visible keys, so the same bits (dq through the
    deterministic pair, whose sums have one order).  With all tokens kept the key tiles'
    dK and dV are summed in parts: fp32 sums of another order, rounded to bf16 once, so
    a step (2^-7 of the value) apart at most."""
    import long_context_attention_attn_gb300 as ga
    x = _inputs(1, 517, 4, 2, 128, 128, "packed", seed=4)
    a = _gpu(ga, x, window, sink, 0.1, det=True)
    b = _gpu(ga, x, *same, 0.1, det=True)
    for t, u in zip((a[0], a[1], a[2][0]), (b[0], b[1], b[2][0])):
        assert torch.equal(t, u)
    for t, u in zip(a[2][1:], b[2][1:]):
        if window >= 0 and sink:
            assert (t.double() - u.double()).norm() <= 2.0 ** -7 * u.double().norm()
        else:
            assert torch.equal(t, u)


@pytest.mark.parametrize("det,d,dv", [(False, 64, 64), (False, 128, 128), (True, 128, 128), (True, 256, 256),
                                      (True, 192, 128)])
def test_key_tiles_in_parts(det, d, dv):
    """Two long documents under a short window: the tiles of kept tokens see 15 and 5 query
    tiles and are cut; run to run the same bits in the deterministic pair, also on a
    workspace full of NaN, and with the gradients added to what is there."""
    import long_context_attention_attn_gb300 as ga
    s, hq, hkv, window, sink, scale = 2600, 6, 2, 100, 5, 0.1
    q, k, v, dout = (t.to(DEV) for t in workload.qkv(1, s, hq, hkv, d, seed=d, with_dout=True, dv=dv))
    ids = torch.ones(1, s, dtype=torch.int32)
    pos = torch.arange(s, dtype=torch.int32)[None].clone()
    ids[:, 1900:], pos[:, 1900:] = 2, pos[:, 1900:] - 1900
    ids[:, 1850:1900] = 0
    di, dp = ids.to(DEV), pos.to(DEV)
    kw = dict(window_left=window, sink_tokens=sink, scale=scale, check_status=True)
    out, lse = ga.attn_fwd(q, k, v, di, dp, **kw)
    need = ga.workspace_bytes_bwd(q, k, di, dp, window, v=v, deterministic=det, sink_tokens=sink)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    got = ga.attn_bwd(q, k, v, out, lse, dout, di, dp, deterministic=det, workspace=ws, **kw)
    ref = A.attn_bwd(*(t.cpu() for t in (q, k, v, dout)), ids, pos, ids, pos, window, scale, sink_tokens=sink)
    for name, g, r in zip(("dq", "dk", "dv"), got, ref):
        check_grad(g.cpu(), r, name)
    again = ga.attn_bwd(q, k, v, out, lse, dout, di, dp, deterministic=det, **kw)
    for n, (g, r) in enumerate(zip(got, again)):
        if det or n:  # (the fused kernel sums dq in hardware order)
            assert torch.equal(g, r)
    start = [torch.full(t.shape, 0.5, dtype=torch.float32, device=DEV) for t in (q, k, v)]
    ga.attn_bwd(q, k, v, out, lse, dout, di, dp, deterministic=det, dq=start[0], dk=start[1], dv=start[2],
                accumulate_fp32=True, **kw)
    for name, g, r in zip(("dq", "dk", "dv"), start, ref):
        check_grad(g.cpu() - 0.5, r, name)


def test_key_tiles_in_parts_of_packed_kv():
    """The same with K and V (and their gradients) as the halves of one tensor, and a batch."""
    import long_context_attention_attn_gb300 as ga
    b, s, hq, hkv, d = 2, 900, 4, 2, 64
    q, k, v, dout = workload.qkv(b, s, hq, hkv, d, seed=5, with_dout=True)
    ids, pos = workload.segments(b, s, 2)
    kv = torch.stack([k, v], dim=2).to(DEV)
    g = [t.to(DEV) for t in (q, dout, ids, pos)]
    kw = dict(window_left=30, sink_tokens=3, scale=0.125)
    out, lse = ga.attn_fwd(g[0], kv[:, :, 0], kv[:, :, 1], g[2], g[3], **kw)
    got = ga.attn_bwd(g[0], kv[:, :, 0], kv[:, :, 1], out, lse, g[1], g[2], g[3], **kw)
    ref = A.attn_bwd(q, k, v, dout, ids, pos, ids, pos, 30, 0.125, sink_tokens=3)
    for name, x, r in zip(("dq", "dk", "dv"), got, ref):
        check_grad(x.cpu(), r, name)


def test_many_kv_heads_take_no_parts():
    """With as many kv heads as parts in all, no key tile is cut."""
    import long_context_attention_attn_gb300 as ga
    x = _inputs(1, 400, 460, 460, 64, 64, "one", seed=6)
    out, lse, grads = _gpu(ga, x, 16, 3, 0.125)
    ro, _ = A.attn_fwd(x["q"], x["k"], x["v"], x["ids"], x["pos"], x["ids"], x["pos"], 16, 0.125, sink_tokens=3)
    check_out(out.cpu(), ro)
    ref = A.attn_bwd(x["q"], x["k"], x["v"], x["dout"], x["ids"], x["pos"], x["ids"], x["pos"], 16, 0.125,
                     sink_tokens=3)
    for name, got, want in zip(("dq", "dk", "dv"), grads, ref):
        check_grad(got.cpu(), want, name)


@pytest.mark.parametrize("s,window,sink,packing", [(1500, 100, 4, "one"), (1500, 100, 300, "one"),
                                                   (1300, 20, 5, "packed"), (9000, 1000, 140, "one")])
def test_tile_plan_covers_the_mask(s, window, sink, packing):
    """Tiles with a visible pair are not skipped, tiles taken without a mask are all visible."""
    import long_context_attention_attn_gb300 as ga
    x = _inputs(1, s, 2, 1, 64, 64, packing, seed=s)
    g = {n: t.to(DEV) for n, t in x.items()}
    cls, _ = ga.attn_tile_plan(g["q"], g["k"], g["ids"], g["pos"], window_left=window, sink_tokens=sink)
    got = cls.cpu().numpy()
    want = P.brute_classes(x["ids"].numpy(), x["pos"].numpy(), x["ids"].numpy(), x["pos"].numpy(), window,
                           sink_tokens=sink)
    assert not np.any((got == P.SKIP) & (want != P.SKIP))
    assert not np.any((got == P.FULL) & (want != P.FULL))
    if packing == "one":  # one segment: exact, the ragged last tile apart
        n = s // 128
        assert np.array_equal(got[:, :n, :n], want[:, :n, :n])


@pytest.mark.parametrize("batch_shards", [False, True])
def test_ring_and_allgather(batch_shards):
    from long_context_attention_attn_gb300 import ring
    x = _inputs(1, 768, 4, 2, 64, 64, "one", seed=11)
    g = {n: t.to(DEV) for n, t in x.items()}
    kw = dict(window_left=70, sink_tokens=6, scale=0.125)
    ro, rl = A.attn_fwd(x["q"], x["k"], x["v"], x["ids"], x["pos"], x["ids"], x["pos"], 70, 0.125, sink_tokens=6)
    ref = A.attn_bwd(x["q"], x["k"], x["v"], x["dout"], x["ids"], x["pos"], x["ids"], x["pos"], 70, 0.125,
                     sink_tokens=6)
    out, lse = ring.ring_attn_fwd(g["q"], g["k"], g["v"], g["ids"], g["pos"], 4, batch_shards=batch_shards, **kw)
    check_out(out.cpu(), ro)
    check_lse(lse.cpu(), rl)
    grads = [ring.ring_attn_bwd(g["q"], g["k"], g["v"], out, lse, g["dout"], g["ids"], g["pos"], 4,
                                batch_shards=batch_shards, **kw)]
    if not batch_shards:
        ag = dict(stripe_size=64, **kw)
        out2, lse2 = ring.allgather_attn_fwd(g["q"], g["k"], g["v"], g["ids"], g["pos"], 4, **ag)
        check_out(out2.cpu(), ro)
        grads.append(ring.allgather_attn_bwd(g["q"], g["k"], g["v"], out2, lse2, g["dout"], g["ids"], g["pos"], 4,
                                             **ag))
    for got3 in grads:
        for name, got, want in zip(("dq", "dk", "dv"), got3, ref):
            check_grad(got.cpu(), want, name)


LENGTHS = [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 383, 640, 1000, 1500]


@pytest.mark.parametrize("seed", range(16))
def test_random_configurations(seed):
    """Lengths around the tiles' edges, groups of one to five, any window and kept tokens, random
    packings, and queries of one block against the keys of an earlier one."""
    import long_context_attention_attn_gb300 as ga
    rng = np.random.default_rng(7000 + seed)
    d, dv = [(64, 64), (128, 128), (256, 256), (192, 128)][seed % 4]
    b, hkv, g = int(rng.integers(1, 3)), int(rng.integers(1, 3)), int(rng.integers(1, 6))
    s_q = int(rng.choice(LENGTHS))
    cross = bool(rng.random() < 0.3)
    s_kv = int(rng.choice(LENGTHS)) if cross else s_q
    window = int(rng.integers(0, max(1, s_kv // int(rng.integers(1, 9)))))
    sink = int(rng.choice([1, 2, 5, 64, 129, 400]))
    q, _, _, dout = workload.qkv(b, s_q, hkv * g, hkv, d, seed=seed, with_dout=True, dv=dv)
    _, k, v = workload.qkv(b, s_kv, hkv * g, hkv, d, seed=seed + 500, dv=dv)
    ids, pos = workload.random_segments(b, s_q, seed=seed, max_segments=3, pad_prob=0.25)
    kv_ids, kv_pos = ids, pos
    if cross:
        kv_ids = torch.ones(b, s_kv, dtype=torch.int32)
        kv_pos = torch.arange(s_kv, dtype=torch.int32)[None].repeat(b, 1)
        kv_ids[:, s_kv // 3: s_kv // 3 + s_kv // 7] = 0
        ids = torch.ones(b, s_q, dtype=torch.int32)
        pos = torch.arange(s_kv // 2, s_kv // 2 + s_q, dtype=torch.int32)[None].repeat(b, 1)
    desc = (ids, pos, kv_ids, kv_pos)
    scale = d ** -0.5
    dev = [t.to(DEV) for t in (q, k, v, dout, *desc)]
    kw = dict(window_left=window, sink_tokens=sink, scale=scale, check_status=True)
    out, lse = ga.attn_fwd(*dev[:3], *dev[4:], **kw)
    grads = ga.attn_bwd(*dev[:3], out, lse, dev[3], *dev[4:], deterministic=bool(seed & 4), **kw)
    ro, rl = A.attn_fwd(q, k, v, *desc, window, scale, sink_tokens=sink)
    check_out(out.cpu(), ro)
    check_lse(lse.cpu(), rl)
    for name, got, want in zip(("dq", "dk", "dv"), grads, A.attn_bwd(q, k, v, dout, *desc, window, scale,
                                                                     sink_tokens=sink)):
        check_grad(got.cpu(), want, name)
