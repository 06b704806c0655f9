"""Position rotation, appending to the paged 8-bit cache with it, and decoding for sequences that share a prefix.

The operators, each in a plain form (elementary torch operations in 32 bits,
angles and what decides a cache scale in 64) and, where ``own`` is true, as the
calls a user makes of the package:

* ``rope``: every pair (x1, x2) of the rotated part of each head of q and k turns
  by the angle pos * frequency, times an amplitude:
  y1 = amp * (x1 cos - x2 sin), y2 = amp * (x2 cos + x1 sin).  Pairs are (i,
  i + rot / 2) ("half") or (2i, 2i + 1) ("interleaved").  A training step
  turns q and k, and the gradients dq and dk back by the same angles.
* ``append``: new tokens' K, turned by their positions, and V into the pages of
  a cache held in 8 bits (e4m3) with one power-of-two scale for each page and
  head, and the same tokens' q turned beside them.
* ``shared``: attention of the last ``sq`` tokens of every sequence over that
  cache, where groups of sequences have the same first pages.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ================================================================== the cases
def listed():
    return [
        # q and k of one decoding step of 32 sequences, far into long contexts: launches count
        dict(name="rope_step", op="rope", train=False, b=32, s=1, at=900001, hq=32, hkv=8, d=128, rot=128, offset=0,
             interleaved=False, amp=1.0, fp32=False),
        # a packed training batch: forward and backward
        dict(name="rope_train", op="rope", train=True, b=2, s=8192, at=0, hq=16, hkv=4, d=128, rot=128, offset=0,
             interleaved=False, amp=1.0, fp32=False),
        # odd lengths, a quarter of a wide head in neighbouring pairs, frequencies and amplitude of a longer context
        dict(name="rope_part", op="rope", train=False, b=3, s=1777, at=3, hq=20, hkv=4, d=256, rot=64, offset=0,
             interleaved=True, amp=1.1386, fp32=False),
        # a prompt of 64k tokens, heads of 192 whose last 64 turn
        dict(name="rope_prompt", op="rope", train=False, b=1, s=65536, at=0, hq=32, hkv=8, d=192, rot=64, offset=128,
             interleaved=True, amp=1.0, fp32=False),
        # the append of one decoding step: one token of each of 32 sequences
        dict(name="append_tokens", op="append", packed=False, b=32, new=1, ragged=False, start=4000, hq=32, hkv=8,
             d=128, page=64, rot=128, offset=0, interleaved=False, amp=1.0),
        # ragged prompts packed in one row, behind a prefix that ends inside a (small) page; half of a small head
        dict(name="append_packed", op="append", packed=True, b=7, new=1500, ragged=True, start=100037, hq=8, hkv=4,
             d=64, page=16, rot=32, offset=0, interleaved=True, amp=1.0),
        # two long prompts at once
        dict(name="append_prompts", op="append", packed=False, b=2, new=32768, ragged=False, start=0, hq=32, hkv=8,
             d=128, page=64, rot=128, offset=0, interleaved=False, amp=1.2079),
        # four answers to one question behind a short instruction: latency counts
        dict(name="shared_few", op="shared", b=4, sq=1, groups=1, prefix=2048, omin=20, omax=300, hq=32, hkv=8, d=128,
             page=64, window=-1, sink=0, gaps=False),
        # 64 conversations behind one instruction of 8k tokens, four query heads to a kv head
        dict(name="shared_batch", op="shared", b=64, sq=1, groups=1, prefix=8192, omin=100, omax=2000, hq=32, hkv=8,
             d=128, page=64, window=-1, sink=0, gaps=False),
        # three instructions of unlike lengths, drafted tokens, small heads and pages, a window over part of the
        # prefix with its first tokens kept, empty slots
        dict(name="shared_groups", op="shared", b=45, sq=3, groups=3, prefix=6000, omin=1, omax=1500, hq=16, hkv=4,
             d=64, page=16, window=4095, sink=60, gaps=True),
        # wide heads, one query head to a kv head: a few rows for each key
        dict(name="shared_wide", op="shared", b=12, sq=1, groups=1, prefix=20000, omin=700, omax=3001, hq=4, hkv=4,
             d=256, page=32, window=-1, sink=0, gaps=False),
        # 128 questions about one long document, sixteen query heads to a kv head
        dict(name="shared_document", op="shared", b=128, sq=1, groups=1, prefix=32768, omin=30, omax=600, hq=128,
             hkv=8, d=128, page=64, window=-1, sink=0, gaps=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _turning(rng, d):
    """Which part of a head of d turns, and how."""
    rot = rng.choice([d, d, d // 2, rng.randrange(16, d + 1, 16)])
    return dict(rot=rot, offset=rng.choice([0, 0, d - rot, rng.randrange(0, d - rot + 1, 8)]),
                interleaved=rng.random() < 0.5, amp=rng.choice([1.0, 1.0, 1.1386, 0.9]))


def draw(rng):
    op = rng.choice(["rope", "append", "shared", "shared"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        d = rng.choice([64, 128, 128, 192, 256])
        train, fp32 = rng.random() < 0.5, rng.random() < 0.25
        b, hq = rng.choice([1, 1, 2, 3, 32]), hkv * rng.choice([1, 2, 3, 4, 8])
        s = _log(rng, 1, 65536 * 40 * 192 // ((hq + hkv) * d * b * (1 + train) * (1 + fp32)))
        return dict(op=op, train=train, b=b, s=min(s, 131072), at=rng.choice([0, _log(rng, 1, 1000000)]), hq=hq,
                    hkv=hkv, d=d, fp32=fp32, **_turning(rng, d))
    if op == "append":
        b = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _log(rng, 2, 60000 // b)
        return dict(op=op, packed=rng.random() < 0.4, b=b, new=new, ragged=rng.random() < 0.6,
                    start=rng.choice([0, rng.randrange(0, 3000), _log(rng, 1, 200000)]), hq=hkv * rng.choice([1, 2, 4]),
                    hkv=hkv, d=d, page=page, **_turning(rng, d))
    b, sq, g = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 4]), rng.choice([1, 2, 4, 5, 8, 16])
    rows = b * sq * g * hkv * d
    # (what a pass computes, and what the plain form copies for every sequence)
    most = min(128 * 128 * 128 * 33000 // rows, 128 * 8 * 128 * 33000 // (b * hkv * d), 130000)
    prefix = _log(rng, 1, max(1, most * 9 // 10))
    omax = _log(rng, 1, max(1, min(5000, most - prefix)))
    return dict(op=op, b=b, sq=sq, groups=rng.choice([1, 1, 2, 5]), prefix=prefix, omin=rng.randrange(0, omax + 1),
                omax=omax, hq=hkv * g, hkv=hkv, d=d, page=page, window=-1 if rng.random() < 0.6 else
                _log(rng, 1, max(2, prefix + omax)) - 1, sink=rng.choice([0, 1, 4, 77]), gaps=rng.random() < 0.3)


# -------------------------------------------------- what follows from a case alone
def _starts(c):
    return [c["start"] + 13 * i for i in range(c["b"])]


def _news(c):
    return [max(1, c["new"] * ((i * 5) % c["b"] + 1) // c["b"]) if c["ragged"] else c["new"]
            for i in range(c["b"])]


def _groups(c):
    """The first sequence of each group of sequences, and behind the last: groups of unlike sizes, perhaps empty."""
    n = c["groups"]
    return [c["b"] * (j * (j + 1)) // (n * (n + 1)) for j in range(n + 1)]


def _shared(c):
    """The pages that each group shares: the first the most."""
    return [c["prefix"] * (c["groups"] - j) // c["groups"] // c["page"] for j in range(c["groups"])]


def _group_of(c):
    at = _groups(c)
    return [max(j for j in range(c["groups"]) if at[j] <= i < at[j + 1]) for i in range(c["b"])]


def _lengths(c):
    """The cached tokens of each sequence, its new ones among them: what its group shares, and its own."""
    b, pages, of = c["b"], _shared(c), _group_of(c)
    return [0 if c["gaps"] and i % 7 == 3 else
            max(c["sq"], pages[of[i]] * c["page"] + c["omin"] + (c["omax"] - c["omin"]) * (i * 7919 % b) // max(1, b - 1))
            for i in range(b)]


def _seen(pos, window, sink):
    """(keys visible from a query at `pos`: how many of the window's, how many kept ones before it)"""
    near = pos + 1 if window < 0 else min(pos + 1, window + 1)
    return near, min(sink, pos + 1 - near)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["b"] * c["s"]
        values = n * (c["hq"] + c["hkv"])
        once = 2 * values * c["d"] * (4 if c["fp32"] else 2) + 4 * n + 4 * c["rot"]
        return dict(bytes=once * (1 + c["train"]), flops=3 * values * c["rot"] * (1 + c["train"]))
    if c["op"] == "append":
        n, per = sum(_news(c)), c["hkv"] * c["d"]
        pages = sum((st + m - 1) // c["page"] - st // c["page"] + 1 for st, m in zip(_starts(c), _news(c)))
        return dict(bytes=2 * n * per * 3 + 4 * n * c["hq"] * c["d"] + 2 * pages * c["hkv"] * 4 + 4 * pages + 8 * c["b"],
                    flops=3 * n * (c["hq"] + c["hkv"]) * c["rot"])
    at, pages, lengths = _groups(c), _shared(c), _lengths(c)
    keys = pairs = 0
    for j in range(c["groups"]):
        prefix, seen = pages[j] * c["page"], []
        for n in lengths[at[j]:at[j + 1]]:
            got = [_seen(p, c["window"], c["sink"]) for p in range(max(0, n - c["sq"]), n)]
            pairs += sum(a + k for a, k in got)
            if got:  # the new tokens see [lo, n) and the first tokens that are kept
                lo = n - (got[0][0] + len(got) - 1)
                kept = min(c["sink"], lo)
                seen.append((lo, kept))
                keys += n - max(lo, prefix) + max(0, kept - prefix)
        if seen:  # what the group shares, once: from the first window on, and the kept tokens before it
            lo = min(x for x, _ in seen)
            keys += max(0, prefix - lo) + min(prefix, lo, max(k for _, k in seen))
    rows = c["b"] * c["sq"] * c["hq"]
    return dict(bytes=2 * keys * c["hkv"] * c["d"] + 8 * (keys // c["page"]) * c["hkv"] + rows * (4 * c["d"] + 4),
                flops=4 * pairs * c["hq"] * c["d"])


# ================================================================= the inputs
def _pow2(e):
    """2^e in fp32 from whole exponents in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_of(amax):
    """The smallest power of two by which `amax` is at most 448 (no less than 2^-126)."""
    m, e = torch.frexp(amax)
    k = torch.where(m > 0.875, e - 8, e - 9)
    return _pow2(torch.where(amax > 0, k, torch.full_like(k, -126)).clamp(-126, 127))


def _pool(gen, pages, c):
    """Pages of normal values, each head of its own size, in e4m3 with a scale for each page and head."""
    size = torch.exp(0.5 * torch.randn(1, c["hkv"], 1, 1, generator=gen, device=DEV))
    x = torch.randn(pages, c["hkv"], c["page"], c["d"], generator=gen, device=DEV) * size
    scale = _scale_of(x.abs().amax((2, 3)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def _frequencies(c):
    """Radians per position of each pair, in 64 bits.  With an amplitude above 1 those of a context eight times longer:
    slow pairs turn eight times slower, fast ones as before, those between in proportion."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    f = 10000.0 ** (-2.0 * i / c["rot"])
    if c["amp"] > 1:
        turns = f * 4096 / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * (keep + (1 - keep) / 8)
    return f


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV).to(torch.float32 if c.get("fp32") else torch.bfloat16)

    if c["op"] == "rope":
        # positions of sequences that begin anywhere up to `at`
        first = torch.randint(0, c["at"] + 1, (c["b"], 1), generator=gen, device=DEV)
        pos = (first + torch.arange(c["s"], device=DEV)).to(torch.int32)
        st = dict(q=normal(c["b"], c["s"], c["hq"], c["d"]), k=normal(c["b"], c["s"], c["hkv"], c["d"]), pos=pos,
                  freqs=_frequencies(c))
        if c["train"]:
            st["dq"], st["dk"] = normal(c["b"], c["s"], c["hq"], c["d"]), normal(c["b"], c["s"], c["hkv"], c["d"])
    elif c["op"] == "append":
        news, starts, page = _news(c), _starts(c), c["page"]
        first = [a // page for a in starts]
        need = [(a + n - 1) // page + 1 - f for a, n, f in zip(starts, news, first)]
        pages = sum(need) + 3 + sum(need) // 32
        ids = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        # (pages before the first new token are not touched: given back, or another's)
        table = torch.full((c["b"], max(f + n for f, n in zip(first, need)) + 1), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, n in enumerate(need):
            table[i, first[i]:first[i] + n] = ids[at:at + n]
            at += n
        if c["packed"]:
            # sequence after sequence with three tokens of padding between, in one row
            begin = [sum(news[:i]) + 3 * i for i in range(c["b"])]
            rows, length = 1, begin[-1] + news[-1]
        else:
            begin, rows, length = None, c["b"], max(news)
        size = torch.exp(0.5 * torch.randn(1, 1, c["hkv"], 1, generator=gen, device=DEV))
        st = dict(table=table, start=_ints(starts), lens=_ints(news), begin=None if begin is None else _ints(begin),
                  freqs=_frequencies(c), q=normal(rows, length, c["hq"], c["d"]))
        st["q_out"] = torch.zeros_like(st["q"])
        for x in ("k", "v"):
            st[x] = (torch.randn(rows, length, c["hkv"], c["d"], generator=gen, device=DEV) * size).to(torch.bfloat16)
            # what the pages hold before: older tokens with scales of their own
            old = torch.randn(pages, c["hkv"], page, c["d"], generator=gen, device=DEV) * 90
            st[x + "_cache"] = old.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            st[x + "_scale"] = _pow2(torch.randint(-10, -4, (pages, c["hkv"]), generator=gen, device=DEV))
    else:
        lengths, at, shared, of = _lengths(c), _groups(c), _shared(c), _group_of(c)
        need = [max(0, -(-n // c["page"]) - shared[g]) for n, g in zip(lengths, of)]
        pages = sum(shared) + sum(need) + 3 + sum(need) // 32
        ids = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        width = max(shared + [shared[g] + n for n, g in zip(need, of)]) + 1
        table = torch.full((c["b"], width), -1, dtype=torch.int32, device=DEV)
        used = 0
        for j, n in enumerate(shared):
            table[at[j]:at[j + 1], :n] = ids[used:used + n]
            used += n
        for i, n in enumerate(need):
            table[i, shared[of[i]]:shared[of[i]] + n] = ids[used:used + n]
            used += n
        st = dict(q=normal(c["b"], c["sq"], c["hq"], c["d"]), table=table, lens=_ints(lengths),
                  shared=_ints([shared[g] for g in of]), groups=_ints(at),
                  largest=max(b - a for a, b in zip(at, at[1:])))
        st["k_cache"], st["k_scale"] = _pool(gen, pages, c)
        st["v_cache"], st["v_scale"] = _pool(gen, pages, c)
    st["case"] = c
    return st


# ============================================================ the plain forms
def _turn(x, pos, st, back=False, bits=torch.float32):
    """x [..., heads, d] turned by pos [...] in `bits` (angles always in 64), not rounded."""
    c = st["case"]
    angle = pos.double()[..., None] * st["freqs"]
    cos = (torch.cos(angle) * c["amp"]).to(bits)[..., None, :]
    sin = (torch.sin(angle) * (-c["amp"] if back else c["amp"])).to(bits)[..., None, :]
    y = x.to(bits)
    lo, n = c["offset"], c["rot"]
    part = y[..., lo:lo + n]
    if c["interleaved"]:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = part[..., :n // 2], part[..., n // 2:]
        turned = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    return torch.cat((y[..., :lo], turned, y[..., lo + n:]), -1)


def _plain_rope(st):
    got = {x: _turn(st[x], st["pos"], st).to(st[x].dtype) for x in ("q", "k")}
    if st["case"]["train"]:
        got.update({x: _turn(st[x], st["pos"], st, back=True).to(st[x].dtype) for x in ("dq", "dk")})
    return got


def _plain_append_one(x, cache, scale, table, start, pid, slot):
    """x [tokens, hkv, d]: every new token's values, for slot `slot` of page `pid`."""
    page = cache.shape[2]
    size = x.abs()
    size = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(-1)
    amax = torch.zeros(scale.shape, dtype=size.dtype, device=x.device).index_reduce_(0, pid, size, "amax")
    # the first page of a sequence keeps its older tokens, and its scale where that is larger
    held = start % page
    first = table.gather(1, (start // page)[:, None])[:, 0].long()
    old = scale[first]
    new = scale.clone()
    new[pid] = _scale_of(amax)[pid]
    new[first] = torch.where((held > 0)[:, None], torch.maximum(old, new[first]), new[first])
    raw = cache.view(torch.uint8)
    kept = raw[first].view(torch.float8_e4m3fn)
    again = (kept.float() * (old / new[first])[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    stays = torch.arange(page, device=x.device)[None, :] >= held[:, None]
    raw[first] = torch.where(stays[:, None, :, None], kept.view(torch.uint8), again.view(torch.uint8))
    code = (x / new[pid][:, :, None]).float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    raw[pid, :, slot] = code.view(torch.uint8)
    scale.copy_(new)


def _plain_append(st):
    c = st["case"]
    start, lens = st["start"].long(), st["lens"].long()
    row_of = torch.repeat_interleave(torch.arange(c["b"], device=DEV), lens)
    at = torch.arange(row_of.numel(), device=DEV) - (torch.cumsum(lens, 0) - lens)[row_of]
    begin = st["begin"].long() if c["packed"] else torch.arange(c["b"], device=DEV) * st["k"].shape[1]
    token, pos = begin[row_of] + at, start[row_of] + at
    pid, slot = st["table"][row_of, pos // c["page"]].long(), pos % c["page"]
    st["q_out"].flatten(0, 1)[token] = _turn(st["q"].flatten(0, 1)[token], pos, st).to(torch.bfloat16)
    for x in ("k", "v"):
        new = st[x].flatten(0, 1)[token]
        new = _turn(new, pos, st, bits=torch.float64) if x == "k" else new.float()
        _plain_append_one(new, st[x + "_cache"], st[x + "_scale"], st["table"], start, pid, slot)
    return {n: st[n] for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_shared(st):
    """Every sequence over all of its pages, as if none were shared."""
    c = st["case"]
    b, sq, hq, hkv, d, page = c["b"], c["sq"], c["hq"], c["hkv"], c["d"], c["page"]
    g = hq // hkv
    table = st["table"].clamp_min(0).long()

    def rows(x):  # [b, hkv, keys, d] in fp32
        code = st[x + "_cache"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        code *= st[x + "_scale"][table][:, :, :, None, None]
        return code.transpose(1, 2).reshape(b, hkv, -1, d)

    kp = torch.arange(table.shape[1] * page, device=DEV)[None, None, :]
    qp = (st["lens"].long()[:, None] - sq + torch.arange(sq, device=DEV))[:, :, None]
    see = kp <= qp
    if c["window"] >= 0:
        see = see & ((qp - kp <= c["window"]) | (kp < c["sink"]))
    q = st["q"].float().view(b, sq, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, sq * g, d)
    s = (q @ rows("k").transpose(-1, -2)).view(b, hkv, sq, g, -1) * d ** -0.5
    s = s.masked_fill(~see[:, None, :, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.masked_fill(m == float("-inf"), 0.0))
    z = p.sum(-1, keepdim=True)
    o = ((p / z.clamp_min(1e-30)).view(b, hkv, sq * g, -1) @ rows("v")).view(b, hkv, sq, g, d)
    return dict(out=o.transpose(1, 2).reshape(b, sq, hq, d).to(torch.bfloat16),
                lse=(m + torch.log(z)).squeeze(-1).permute(0, 1, 3, 2).reshape(b, hq, sq))


# ==================================================================== one pass
def run(st):
    c = st["case"]
    if not own:
        return dict(rope=_plain_rope, append=_plain_append, shared=_plain_shared)[c["op"]](st)
    import long_context_attention_attn_gb300 as ga
    if c["op"] == "shared":
        out, lse = ga.attn_decode_shared(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                         st["table"], st["lens"], st["shared"], st["groups"],
                                         max_group=st["largest"], window_left=c["window"], sink_tokens=c["sink"],
                                         scale=c["d"] ** -0.5)
        return dict(out=out, lse=lse)
    how = dict(offset=c["offset"], interleaved=c["interleaved"], amplitude=c["amp"])
    if c["op"] == "rope":
        q, k = ga.rope(st["q"], st["k"], st["pos"], st["freqs"], **how)
        got = dict(q=q, k=k)
        if c["train"]:
            got["dq"], got["dk"] = ga.rope_bwd(st["dq"], st["dk"], st["pos"], st["freqs"], **how)
        return got
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    lens = st["lens"] if c["ragged"] or c["packed"] else None
    q = ga.kv_cache_append_rope(st["q"], st["k"], st["v"], *cache, st["table"], st["start"], st["freqs"], lens=lens,
                                tok_start=st["begin"], max_new=c["new"], q_out=st["q_out"], **how)
    return dict(zip(("q_out", "k_cache", "v_cache", "k_scale", "v_scale"), (q, *cache)))


# ================================================================ in 64 bits
def exact(case, seed):
    """The definitions in 64 bits: turns as products of complex numbers, attention one sequence and head at a time."""
    st = prepare(case, seed)
    return dict(rope=_exact_rope, append=_exact_append, shared=_exact_shared)[case["op"]](case, st)


def _exact_turn(x, pos, freqs, c, sign=1):
    """x [tokens, heads, d] times amp * exp(i * sign * pos * freq), its pairs as complex numbers."""
    y = x.double().clone()
    lo, half = c["offset"], c["rot"] // 2
    if c["interleaved"]:
        one, two = slice(lo, lo + c["rot"], 2), slice(lo + 1, lo + c["rot"], 2)
    else:
        one, two = slice(lo, lo + half), slice(lo + half, lo + c["rot"])
    by = torch.polar(torch.full_like(freqs, c["amp"]).expand(pos.numel(), -1).contiguous(),
                     sign * pos.double()[:, None] * freqs[None, :])
    z = torch.complex(y[:, :, one].contiguous(), y[:, :, two].contiguous()) * by[:, None, :]
    y[:, :, one], y[:, :, two] = z.real, z.imag
    return y


def _exact_rope(c, st):
    pos = st["pos"].flatten()
    got = {}
    for x, sign in (("q", 1), ("k", 1), ("dq", -1), ("dk", -1)):
        if x in st:
            got[x] = _exact_turn(st[x].flatten(0, 1), pos, st["freqs"], c, sign).view(st[x].shape)
    return got


def _exact_append(c, st):
    """Codes before their rounding to 8 bits (the value over the page's scale), the scales, and q."""
    page, table = c["page"], st["table"].cpu()
    got = dict(q_out=st["q_out"].double())
    for x in ("k", "v"):
        got[x + "_cache"], got[x + "_scale"] = st[x + "_cache"].double(), st[x + "_scale"].double()
    for i, (a, n) in enumerate(zip(_starts(c), _news(c))):
        at = int(st["begin"][i]) if c["packed"] else i * st["k"].shape[1]
        pos = torch.arange(a, a + n, device=DEV)
        got["q_out"].flatten(0, 1)[at:at + n] = _exact_turn(st["q"].flatten(0, 1)[at:at + n], pos, st["freqs"], c)
        held, count = a % page, (a + n - 1) // page - a // page + 1
        pid = table[i, a // page:a // page + count].long().to(DEV)
        for x in ("k", "v"):
            code, scale = got[x + "_cache"], got[x + "_scale"]
            new = st[x].flatten(0, 1)[at:at + n].double()
            if x == "k":
                new = _exact_turn(new, pos, st["freqs"], c)
            full = torch.zeros(count * page, c["hkv"], c["d"], dtype=torch.float64, device=DEV)
            full[held:held + n] = new
            full = full.view(count, page, c["hkv"], c["d"]).transpose(1, 2)
            top = (full.abs().amax((2, 3)) / E4M3_MAX).clamp_min(2.0 ** -126)
            need = torch.ldexp(torch.ones_like(top), torch.round(torch.log2(top)).to(torch.int32))
            need = torch.where(need < top, 2 * need, torch.where(need >= 2 * top, need / 2, need))
            if held:
                need[0] = torch.maximum(need[0], scale[pid[0]])
            mine = torch.zeros(count * page, dtype=torch.bool, device=DEV)
            mine[held:held + n] = True
            kept = code[pid]
            if held:
                kept[0, :, :held] *= (scale[pid[0]] / need[0])[:, None, None]
            code[pid] = torch.where(mine.view(count, 1, page, 1), full / need[:, :, None, None], kept)
            scale[pid] = need
    return got


def _exact_shared(c, st):
    b, sq, hq, d, page = c["b"], c["sq"], c["hq"], c["d"], c["page"]
    g = hq // c["hkv"]
    out = torch.zeros(b, sq, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq, sq), float("-inf"), dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lengths(c)):
        if not n:
            continue
        ids = st["table"][i, :-(-n // page)].long()
        # [hkv, keys, d]
        k, v = ((st[x + "_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                 * st[x + "_scale"][ids].double()[:, :, None, None]).transpose(0, 1).reshape(c["hkv"], -1, d)[:, :n]
                for x in ("k", "v"))
        for t in range(max(0, sq - n), sq):
            gap = n - sq + t - torch.arange(n, device=DEV)
            see = gap >= 0
            if c["window"] >= 0:
                see &= (gap <= c["window"]) | (torch.arange(n, device=DEV) < c["sink"])
            score = torch.einsum("hgd,hkd->hgk", st["q"][i, t].double().view(-1, g, d), k) * d ** -0.5
            score = torch.where(see, score, torch.full_like(score, float("-inf")))
            norm = torch.logsumexp(score, -1)
            out[i, t] = torch.einsum("hgk,hkd->hgd", torch.exp(score - norm[..., None]), v).reshape(hq, d)
            lse[i, :, t] = norm.reshape(hq)
    return dict(out=out, lse=lse)
