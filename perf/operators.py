"""Attention under a window with first tokens kept, and a paged cache in 8 bits with what works on it.

The operators, each in a plain form (elementary torch operations in 32 bits)
and, where ``own`` is true, as the calls a user makes of the package:

* ``attend``: attention under a sliding window where the first ``sink`` tokens
  of every segment stay visible; forward (a prompt), or forward and backward
  (a training step).  Key j of query i's segment is visible iff
  pos_j <= pos_i and (pos_i - pos_j <= window or pos_j < sink).
* ``append``: new K / V tokens into the pages of a cache held in 8 bits (e4m3)
  with one power-of-two scale for each page and head.
* ``decode``: attention of the last ``sq`` tokens of every sequence over that
  cache, with the same window and first tokens.
* ``copy``: copies of whole pages of that cache with their scales.
"""
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ================================================================== the cases
def listed():
    return [
        # one short document of an odd length, a training step: launches count
        dict(name="attend_train_short", op="attend", train=True, b=1, s=777, hq=4, hkv=2, d=64, dv=64,
             slots=1, window=128, sink=4),
        # a packed training batch: two documents a row, padding between them, a window of 1024
        dict(name="attend_train_packed", op="attend", train=True, b=2, s=8192, hq=16, hkv=4, d=128, dv=128,
             slots=2, window=1024, sink=4),
        # a prompt of 8k tokens before its tokens go to the cache: forward only
        dict(name="attend_prompt", op="attend", train=False, b=1, s=8192, hq=32, hkv=8, d=128, dv=128,
             slots=1, window=1024, sink=64),
        # the append of one decoding step: one token of each of 32 sequences
        dict(name="append_tokens", op="append", packed=False, b=32, new=1, ragged=False, start=4000, hkv=8,
             d=128, page=64),
        # ragged prompts packed in one row, behind a shared prefix that ends inside a (small) page
        dict(name="append_packed", op="append", packed=True, b=7, new=1500, ragged=True, start=37, hkv=4,
             d=64, page=16),
        # two long prompts at once
        dict(name="append_prompts", op="append", packed=False, b=2, new=32768, ragged=False, start=0, hkv=8,
             d=128, page=64),
        # one conversation of 4k tokens: latency counts
        dict(name="decode_one", op="decode", b=1, sq=1, lmin=4096, lmax=4096, hq=32, hkv=8, d=128, page=64,
             window=-1, sink=0),
        # a batch of 64 conversations of very different lengths, sixteen query heads to a kv head
        dict(name="decode_batch", op="decode", b=64, sq=1, lmin=200, lmax=16384, hq=128, hkv=8, d=128,
             page=64, window=-1, sink=0),
        # a few sequences of up to 128k tokens
        dict(name="decode_128k", op="decode", b=12, sq=1, lmin=30000, lmax=131072, hq=64, hkv=8, d=128,
             page=128, window=-1, sink=0),
        # four drafted tokens under a window whose first tokens are kept; wide heads, small pages, and the
        # pages that fell out of the window given back
        dict(name="decode_draft", op="decode", b=24, sq=4, lmin=3, lmax=20001, hq=16, hkv=4, d=256, page=32,
             window=4095, sink=60),
        # forking 24 sequences: the last, partly filled page of each is copied
        dict(name="copy_fork", op="copy", pairs=24, hkv=8, d=128, page=64),
        # compacting a pool: 6000 pages move to its front
        dict(name="copy_compact", op="copy", pairs=6000, hkv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "append", "decode", "decode", "decode", "copy"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "attend":
        hq = hkv * rng.choice([1, 2, 3, 4, 8])
        b = rng.choice([1, 1, 2, 3])
        s = _log(rng, 33, 8192)
        while b * hq * s * s > 2 * 16 * 8192 * 8192:
            s = s * 3 // 4
        d, dv = rng.choice([(64, 64), (128, 128), (128, 128), (256, 256), (192, 128)])
        return dict(op=op, train=rng.random() < 0.6, b=b, s=s, hq=hq, hkv=hkv, d=d, dv=dv,
                    slots=rng.choice([1, 1, 2, 5]), window=_log(rng, 1, max(2, s)) - 1,
                    sink=_log(rng, 1, 300))
    if op == "append":
        b = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _log(rng, 2, 60000 // b)
        return dict(op=op, packed=rng.random() < 0.4, b=b, new=new, ragged=rng.random() < 0.6,
                    start=rng.randrange(0, 3000), hkv=hkv, d=d, page=page)
    if op == "decode":
        b = _log(rng, 1, 64)
        lmax = _log(rng, 1, min(131072, 900_000_000 // (b * hkv * d)))
        sq = rng.choice([1, 1, 1, 2, 3, 8])
        window = -1 if rng.random() < 0.5 else _log(rng, 1, max(2, lmax)) - 1
        return dict(op=op, b=b, sq=sq, lmin=rng.randrange(0, lmax + 1), lmax=lmax,
                    hq=hkv * rng.choice([1, 2, 4, 5, 8, 16]), hkv=hkv, d=d, page=page, window=window,
                    sink=0 if window < 0 else rng.choice([0, 1, 4, 77]))
    return dict(op=op, pairs=_log(rng, 1, 3000), hkv=hkv, d=d, page=page)


# -------------------------------------------------- what follows from a case alone
def _segments(c):
    """(start, length) of each segment of a row; the rest of a slot is padding."""
    slot = c["s"] // c["slots"]
    n = slot if c["slots"] == 1 else max(1, slot * 7 // 8)
    return [(i * slot, n) for i in range(c["slots"])]


def _lengths(c):
    """The cached tokens of each sequence of a decode case, its new ones among them."""
    b = c["b"]
    return [c["lmin"] + (c["lmax"] - c["lmin"]) * ((i * 7919 + b - 1) % b) // max(1, b - 1) if b > 1
            else c["lmax"] for i in range(b)]


def _starts(c):
    return [c["start"] + 13 * i for i in range(c["b"])]


def _news(c):
    return [max(1, c["new"] * ((i * 5) % c["b"] + 1) // c["b"]) if c["ragged"] else c["new"]
            for i in range(c["b"])]


def _seen(pos, window, sink):
    """(keys visible from a query at `pos`: how many of the window's, how many kept ones before it)"""
    near = pos + 1 if window < 0 else min(pos + 1, window + 1)
    return near, min(sink, pos + 1 - near)


def work(case):
    c = case
    if c["op"] == "attend":
        pairs = c["b"] * c["hq"] * sum(sum(_seen(p, c["window"], c["sink"])) for _, n in _segments(c) for p in range(n))
        rows_q, rows_k = c["b"] * c["s"] * c["hq"], c["b"] * c["s"] * c["hkv"]
        io = 2 * (rows_q * c["d"] + rows_k * (c["d"] + c["dv"]) + rows_q * c["dv"]) + 4 * rows_q + 8 * c["b"] * c["s"]
        flops = 2 * pairs * (c["d"] + c["dv"])
        if c["train"]:  # dO in, dQ, dK, dV out; S again, dP, dQ, dK, dV
            io += 2 * (rows_q * c["dv"] + rows_q * c["d"] + rows_k * (c["d"] + c["dv"]))
            flops += 2 * pairs * (3 * c["d"] + 2 * c["dv"])
        return dict(bytes=io, flops=flops)
    if c["op"] == "append":
        n, per = sum(_news(c)), c["hkv"] * c["d"]
        pages = sum((st + m - 1) // c["page"] - st // c["page"] + 1 for st, m in zip(_starts(c), _news(c)))
        return dict(bytes=2 * n * per * 3 + 2 * pages * c["hkv"] * 4 + 4 * pages + 8 * c["b"], flops=0)
    if c["op"] == "decode":
        keys = pairs = 0
        for n in _lengths(c):
            got = [_seen(p, c["window"], c["sink"]) for p in range(max(0, n - c["sq"]), n)]
            pairs += sum(a + k for a, k in got)
            if got:  # the union over the new tokens: the first one's window up to the last token, and the kept ones
                near = got[0][0] + len(got) - 1
                keys += near + min(c["sink"], n - near)
        rows = c["b"] * c["sq"] * c["hq"]
        return dict(bytes=2 * keys * c["hkv"] * c["d"] + 8 * (keys // c["page"]) * c["hkv"] + rows * (4 * c["d"] + 4),
                    flops=4 * pairs * c["hq"] * c["d"])
    return dict(bytes=4 * c["pairs"] * c["hkv"] * (c["page"] * c["d"] + 4) + 8 * c["pairs"], flops=0)


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


def _table(gen, lengths, c, behind=None):
    """A page table of pages in no order: -1 behind a sequence's end and where `behind` says a page is given back."""
    need = [-(-n // c["page"]) for n in lengths]
    pages = sum(need) + 3 + sum(need) // 32
    ids = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), max(need) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
        if behind is not None:
            lo, hi = behind[i]
            table[i, lo:hi] = -1
    return table, pages


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)

    if c["op"] == "attend":
        ids = torch.zeros(c["b"], c["s"], dtype=torch.int32, device=DEV)
        pos = torch.zeros_like(ids)
        for k, (at, n) in enumerate(_segments(c)):
            ids[:, at:at + n] = k + 1
            pos[:, at:at + n] = torch.arange(n, dtype=torch.int32, device=DEV)
        st = dict(q=normal(c["b"], c["s"], c["hq"], c["d"]), k=normal(c["b"], c["s"], c["hkv"], c["d"]),
                  v=normal(c["b"], c["s"], c["hkv"], c["dv"]), ids=ids, pos=pos)
        if c["train"]:
            st["dout"] = normal(c["b"], c["s"], c["hq"], c["dv"])
    elif c["op"] == "append":
        news, starts = _news(c), _starts(c)
        table, pages = _table(gen, [a + n for a, n in zip(starts, news)], c)
        if c["packed"]:
            # sequence after sequence with three tokens of padding between, in one row
            begin = [sum(news[:i]) + 3 * i for i in range(c["b"])]
            rows, length = 1, begin[-1] + news[-1]
        else:
            begin, rows, length = None, c["b"], max(news)
        size = torch.exp(0.5 * torch.randn(1, 1, c["hkv"], 1, generator=gen, device=DEV))
        st = dict(table=table, start=_ints(starts), lens=_ints(news), begin=None if begin is None else _ints(begin))
        for x in ("k", "v"):
            st[x] = (torch.randn(rows, length, c["hkv"], c["d"], generator=gen, device=DEV) * size).to(torch.bfloat16)
            # what the pages hold before: older tokens with scales of their own
            old = torch.randn(pages, c["hkv"], c["page"], c["d"], generator=gen, device=DEV) * 90
            st[x + "_cache"] = old.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            st[x + "_scale"] = _pow2(torch.randint(-10, -4, (pages, c["hkv"]), generator=gen, device=DEV))
    elif c["op"] == "decode":
        lengths = _lengths(c)
        behind = None
        if c["window"] >= 0:  # pages that no new token sees any more are given back
            behind = [(-(-c["sink"] // c["page"]), max(0, n - c["sq"] - c["window"]) // c["page"]) for n in lengths]
        table, pages = _table(gen, lengths, c, behind)
        st = dict(q=normal(c["b"], c["sq"], c["hq"], c["d"]), table=table, lens=_ints(lengths))
        st["k_cache"], st["k_scale"] = _pool(gen, pages, c)
        st["v_cache"], st["v_scale"] = _pool(gen, pages, c)
    else:
        pages = 2 * c["pairs"] + 5
        at = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        st = dict(src=at[:c["pairs"]].contiguous(), dst=at[c["pairs"]:2 * c["pairs"]].contiguous())
        st["k_cache"], st["k_scale"] = _pool(gen, pages, c)
        st["v_cache"], st["v_scale"] = _pool(gen, pages, c)
    st["case"] = c
    return st


# ============================================================ the plain forms
def _visible(qi, qp, ki, kp, window, sink):
    near = (qp - kp <= window) | (kp < sink) if window >= 0 else torch.ones_like(qp == kp)
    return (qi == ki) & (qi != 0) & (kp <= qp) & near


def _softmax(s, mask):
    """(weights, natural log of their sum) of masked scores; a row that sees nothing has weights 0 and -inf."""
    s = s.masked_fill(~mask, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.masked_fill(m == float("-inf"), 0.0))
    z = p.sum(-1, keepdim=True)
    return p / z.clamp_min(1e-30), (m + torch.log(z)).squeeze(-1)


def _plain_attend(st):
    c = st["case"]
    b, s, hq, hkv, scale = c["b"], c["s"], c["hq"], c["hkv"], c["d"] ** -0.5
    g = hq // hkv
    q = st["q"].float().view(b, s, hkv, g, -1).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * s, -1)
    k = st["k"].float().transpose(1, 2)
    v = st["v"].float().transpose(1, 2)
    ids, pos = st["ids"], st["pos"]
    mask = _visible(ids[:, :, None], pos[:, :, None], ids[:, None, :], pos[:, None, :], c["window"], c["sink"])
    p, lse = _softmax((q @ k.transpose(-1, -2)).view(b, hkv, g, s, s) * scale, mask[:, None, None])
    p = p.view(b, hkv, g * s, s)
    o = p @ v

    def rows(x):
        return x.view(b, hkv, g, s, -1).permute(0, 3, 1, 2, 4).reshape(b, s, hq, -1).to(torch.bfloat16)

    out = dict(out=rows(o), lse=lse.reshape(b, hq, s))
    if c["train"]:
        do = st["dout"].float().view(b, s, hkv, g, -1).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * s, -1)
        ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) * scale
        out["dq"] = rows(ds @ k)
        out["dk"] = (ds.transpose(-1, -2) @ q).transpose(1, 2).to(torch.bfloat16)
        out["dv"] = (p.transpose(-1, -2) @ do).transpose(1, 2).to(torch.bfloat16)
    return out


def _plain_append_one(x, cache, scale, table, start, lens, begin, row_of, at):
    """x fp32 [tokens, hkv, d]: the token of sequence row_of at `at` of its new ones lies at begin + at."""
    page = cache.shape[2]
    pos = start[row_of] + at
    pid = table[row_of, pos // page].long()
    slot = (pos % page).long()
    x = x[begin[row_of] + at]
    size = x.abs()
    size = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(-1)
    amax = torch.zeros_like(scale).index_reduce_(0, pid, size, "amax")
    # the first page of a sequence keeps its older tokens, and its scale where that is larger
    held = start % page
    first = table.gather(1, (start // page).long()[:, None])[:, 0].long()
    old = scale[first]
    new = scale.clone()
    new[pid] = _scale_of(amax)[pid]
    new[first] = torch.where((held > 0)[:, None], torch.maximum(old, new[first]), new[first])
    raw = cache.view(torch.uint8)
    kept = raw[first].view(torch.float8_e4m3fn)
    again = (kept.float() * (old / new[first])[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    stays = torch.arange(page, device=x.device)[None, :] >= held[:, None]
    raw[first] = torch.where(stays[:, None, :, None], kept.view(torch.uint8), again.view(torch.uint8))
    code = (x / new[pid][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    raw[pid, :, slot] = code.view(torch.uint8)
    scale.copy_(new)


def _plain_append(st):
    c = st["case"]
    start, lens = st["start"].long(), st["lens"].long()
    row_of = torch.repeat_interleave(torch.arange(c["b"], device=DEV), lens)
    at = torch.arange(row_of.numel(), device=DEV) - (torch.cumsum(lens, 0) - lens)[row_of]
    begin = st["begin"].long() if c["packed"] else torch.arange(c["b"], device=DEV) * st["k"].shape[1]
    for x in ("k", "v"):
        _plain_append_one(st[x].float().flatten(0, 1), st[x + "_cache"], st[x + "_scale"], st["table"], start, lens,
                          begin, row_of, at)
    return {n: st[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_decode(st):
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
    one = torch.ones_like(qp)
    mask = _visible(one, qp, one, kp, c["window"], c["sink"])
    q = st["q"].float().view(b, sq, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, sq * g, d)
    s = (q @ rows("k").transpose(-1, -2)).view(b, hkv, sq, g, -1) * d ** -0.5
    p, lse = _softmax(s, mask[:, None, :, None, :])
    o = p.view(b, hkv, sq * g, -1) @ rows("v")
    return dict(out=o.view(b, hkv, sq, g, d).transpose(1, 2).reshape(b, sq, hq, d).to(torch.bfloat16),
                lse=lse.permute(0, 1, 3, 2).reshape(b, hq, sq))


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for n in ("k_cache", "v_cache"):
        raw = st[n].view(torch.uint8)
        raw[dst] = raw[src]
    for n in ("k_scale", "v_scale"):
        st[n][dst] = st[n][src]
    return {n: st[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


# ==================================================================== one pass
def run(st):
    c = st["case"]
    if not own:
        return dict(attend=_plain_attend, append=_plain_append, decode=_plain_decode, copy=_plain_copy)[c["op"]](st)
    import long_context_attention_attn_gb300 as ga
    if c["op"] == "attend":
        kw = dict(window_left=c["window"], sink_tokens=c["sink"], scale=c["d"] ** -0.5)
        out, lse = ga.attn_fwd(st["q"], st["k"], st["v"], st["ids"], st["pos"], **kw)
        got = dict(out=out, lse=lse)
        if c["train"]:
            got["dq"], got["dk"], got["dv"] = ga.attn_bwd(st["q"], st["k"], st["v"], out, lse, st["dout"], st["ids"],
                                                          st["pos"], **kw)
        return got
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    if c["op"] == "decode":
        out, lse = ga.attn_decode(st["q"], *cache, st["table"], st["lens"], window_left=c["window"],
                                  sink_tokens=c["sink"], scale=c["d"] ** -0.5)
        return dict(out=out, lse=lse)
    if c["op"] == "append":
        lens = st["lens"] if c["ragged"] or c["packed"] else None
        ga.kv_cache_append(st["k"], st["v"], *cache, st["table"], st["start"], lens=lens, tok_start=st["begin"],
                           max_new=c["new"])
    else:
        ga.kv_cache_copy_pages(*cache, st["src"], st["dst"])
    return dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), cache))


# ================================================================ in 64 bits
def exact(case, seed):
    """The definitions in 64 bits, row by row: one head (or one sequence and head) at a time."""
    c = case
    if c["op"] == "copy":
        return None
    st = prepare(case, seed)
    return dict(attend=_exact_attend, append=_exact_append, decode=_exact_decode)[c["op"]](c, st)


def _weights(score, see):
    """exp(score - lse) where `see`, and lse (-inf for a row that sees nothing)."""
    lse = torch.logsumexp(torch.where(see, score, torch.full_like(score, float("-inf"))), 1)
    w = torch.where(see, torch.exp(score - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]),
                    torch.zeros_like(score))
    return w, lse


def _exact_attend(c, st):
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    g, scale = c["hq"] // c["hkv"], c["d"] ** -0.5
    out = torch.zeros(c["b"], c["s"], c["hq"], c["dv"], dtype=torch.float64, device=DEV)
    lse = torch.full((c["b"], c["hq"], c["s"]), float("-inf"), dtype=torch.float64, device=DEV)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i in range(c["b"]):
        for at, n in _segments(c):  # a segment sees only itself
            p = torch.arange(n, device=DEV)
            gap = p[:, None] - p[None, :]
            see = (gap >= 0) & ((gap <= c["window"]) | (p[None, :] < c["sink"]))
            r = slice(at, at + n)
            for h in range(c["hq"]):
                qh, kh, vh = q[i, r, h], k[i, r, h // g], v[i, r, h // g]
                w, lse[i, h, r] = _weights(qh @ kh.T * scale, see)
                out[i, r, h] = w @ vh
                if c["train"]:
                    do = st["dout"][i, r, h].double()
                    dw = do @ vh.T
                    ds = w * (dw - (w * dw).sum(1, keepdim=True)) * scale
                    dq[i, r, h] = ds @ kh
                    dk[i, r, h // g] += ds.T @ qh
                    dv[i, r, h // g] += w.T @ do
    got = dict(out=out, lse=lse)
    return dict(got, dq=dq, dk=dk, dv=dv) if c["train"] else got


def _exact_append(c, st):
    """Codes before their rounding to 8 bits (the value over the page's scale), and the scales."""
    got = {}
    page, table = c["page"], st["table"].cpu()
    for x in ("k", "v"):
        code, scale = st[x + "_cache"].double(), st[x + "_scale"].double()
        flat = st[x].double().flatten(0, 1)
        for i, (a, n) in enumerate(zip(_starts(c), _news(c))):
            at = int(st["begin"][i]) if c["packed"] else i * st[x].shape[1]
            held, count = a % page, (a + n - 1) // page - a // page + 1
            pid = table[i, a // page:a // page + count].long().to(DEV)
            full = torch.zeros(count * page, c["hkv"], c["d"], dtype=torch.float64, device=DEV)
            full[held:held + n] = flat[at:at + n]
            full = full.view(count, page, c["hkv"], c["d"]).transpose(1, 2)
            top = full.abs().amax((2, 3))
            top = (top / E4M3_MAX).clamp_min(2.0 ** -126)
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
        got[x + "_cache"], got[x + "_scale"] = code, scale
    return got


def _exact_decode(c, st):
    b, sq, hq, d, page = c["b"], c["sq"], c["hq"], c["d"], c["page"]
    g = hq // c["hkv"]
    out = torch.zeros(b, sq, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq, sq), float("-inf"), dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lengths(c)):
        ids = st["table"][i, :-(-n // page)].clamp_min(0).long()
        for h in range(c["hkv"] if n else 0):
            k, v = ((st[x + "_cache"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double()
                     * st[x + "_scale"][ids, h].double()[:, None, None]).reshape(-1, d)[:n] for x in ("k", "v"))
            for t in range(max(0, sq - n), sq):
                gap = n - sq + t - torch.arange(n, device=DEV)
                see = gap >= 0
                if c["window"] >= 0:
                    see &= (gap <= c["window"]) | (torch.arange(n, device=DEV) < c["sink"])
                w, lse[i, h * g:h * g + g, t] = _weights(st["q"][i, t, h * g:h * g + g].double() @ k.T * d ** -0.5,
                                                         see[None, :])
                out[i, t, h * g:h * g + g] = w @ v
    return dict(out=out, lse=lse)
