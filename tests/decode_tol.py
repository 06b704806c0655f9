"""How far attn_decode may be from the plain fp64 form of tests/paged.py, key by key.

2^-10 of sum P |v| and 2e-4 for lse as derived in test_gpu_decode, and what f16 loses below its
normal numbers, which counts where a row's heaviest keys hold zeros in a column:
* P * v_scale is held as f16 2^7 times larger than relative to a reference that is no larger than
  the row's largest P * v_scale (P <= 1, so no larger than the largest scale that it sees).  Half
  of f16's smallest step, 2^-25, is then 2^-32 of that scale for each key, times its |code|.
* The kernel of many rows keeps the reference at 2^-119 of the largest weight or above, so half a
  step is no less than 2^(-25 - 7 - 119) = 2^-151 there.
* fp32 outputs and up to eight terms of their sums (pieces, warps) round to multiples of 2^-149."""
import numpy as np

from tests import paged


def floor(c, window, sink):
    """[n, sq, hq, d]: (2^-32 of the largest visible scale of V + 2^-151) sum |code| + 2^-146."""
    n, sq, hq, d = c["q"].shape
    pages, hkv, size, _ = c["v"].shape
    table, lens, vs = c["table"].numpy(), c["lens"].numpy(), c["vs"].numpy().astype(np.float64)
    code = np.abs(np.nan_to_num(paged.from_e4m3(paged.raw(c["v"])), nan=0.0))
    out = np.zeros((n, sq, hkv, hq // hkv, d))
    for i in range(n):
        for t in range(sq):
            p = int(lens[i]) - sq + t
            j = np.arange(max(0, min(p + 1, table.shape[1] * size)))
            if window >= 0:
                j = j[(p - j <= window) | (j < sink)]
            pid = table[i, j // size]
            ok = (pid >= 0) & (pid < pages)
            if not ok.any():
                continue
            pid, slot = pid[ok], (j % size)[ok]
            for h in range(hkv):
                out[i, t, h] = (2.0 ** -32 * vs[pid, h].max() + 2.0 ** -151) * code[pid, h, slot].sum(0)
    return out.reshape(n, sq, hq, d) + 2.0 ** -146


def check(got, want, least, bf16=False):
    (out, lse), (ro, rl, mag) = got, want
    out, lse = paged.np64(out), paged.np64(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(lse[fin] - rl[fin]) <= 2e-4)
    assert np.all(np.abs(out - ro) <= 2.0 ** -10 * mag + least + (2.0 ** -8 * np.abs(ro) if bf16 else 0))
    assert np.all(out[np.swapaxes(~fin, 1, 2)] == 0)
