"""Plain fp64 forms of the paged 8-bit cache's operators (numpy, one element or row at a time)."""
import numpy as np
import torch

# the 127 non-negative finite e4m3 values in code order (0x00 .. 0x7e)
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def to_e4m3(x):
    """Codes (uint8) nearest to fp64 x, ties to the even code, saturating; NaN is 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7f), code | (np.signbit(x).astype(np.uint8) << 7)).astype(np.uint8)


def from_e4m3(code):
    code = np.asarray(code)
    a = np.append(E4M3, np.nan)[code & 0x7f]
    return np.where(code & 0x80, -a, a)


def append(x, codes, scale, table, start, lens, tok_start):
    """In place on codes uint8 [pages, h, size, d] and scale [pages, h]; x fp64 [tokens, h, d]."""
    pages, heads, size, _ = codes.shape
    for i in range(table.shape[0]):
        if start[i] < 0:
            continue
        new = {}  # page -> [(slot, token row)]
        for t in range(lens[i]):
            pos, row = start[i] + t, tok_start[i] + t
            if pos // size < table.shape[1] and 0 <= row < x.shape[0]:
                new.setdefault(int(table[i, pos // size]), []).append((pos % size, row))
        for pid, put in new.items():
            if not 0 <= pid < pages:
                continue
            first = put[0][0]
            for h in range(heads):
                v = np.array([x[row, h] for _, row in put])
                fine = np.abs(v[np.isfinite(v)])
                top = fine.max() if fine.size else 0.0
                need = 2.0 ** -126
                while top > 448 * need:
                    need *= 2
                now = need if first == 0 else max(need, float(scale[pid, h]))
                if first and now > scale[pid, h]:
                    codes[pid, h, :first] = to_e4m3(from_e4m3(codes[pid, h, :first]) * (float(scale[pid, h]) / now))
                for (slot, _), row in zip(put, v):
                    codes[pid, h, slot] = to_e4m3(row / now)
                scale[pid, h] = now


def decode(q, k_codes, v_codes, k_scale, v_scale, table, lens, window, sink, scale):
    """(out, lse, sum of P |v|) in fp64; q [n, sq, hq, d]."""
    n, sq, hq, d = q.shape
    pages, hkv, size, _ = k_codes.shape
    g = hq // hkv
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((n, hq, sq), -np.inf)
    for i in range(n):
        for t in range(sq):
            p = int(lens[i]) - sq + t
            keys = [j for j in range(min(p + 1, table.shape[1] * size))
                    if (window < 0 or p - j <= window or j < sink) and 0 <= table[i, j // size] < pages]
            if not keys:
                continue
            pid, slot = table[i, np.array(keys) // size], np.array(keys) % size
            for h in range(hkv):
                k = from_e4m3(k_codes[pid, h, slot]) * k_scale[pid, h].astype(np.float64)[:, None]
                v = from_e4m3(v_codes[pid, h, slot]) * v_scale[pid, h].astype(np.float64)[:, None]
                s = scale * (q[i, t, h * g:h * g + g] @ k.T)
                m = s.max(axis=1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(axis=1, keepdims=True)
                out[i, t, h * g:h * g + g] = (e / z) @ v
                mag[i, t, h * g:h * g + g] = (e / z) @ np.abs(v)
                lse[i, h * g:h * g + g, t] = (m + np.log(z))[:, 0]
    return out, lse, mag


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def raw(t):
    """The bytes of a float8 (or uint8) tensor as a numpy array."""
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()
