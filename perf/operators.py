"""Streaming attention, measured: the operators that train with, fill and read a
key/value cache in which a few first tokens (sinks) and a sliding window stay
visible.

  append   write new tokens' keys and values into a paged 8-bit cache (E4M3
           codes, one power-of-two scale per page, head and tensor)
  cache    attention of new query tokens over that cache (single tokens, a few
           drafted ones, chunks of a prompt), optionally with window and sinks
  sinks    sliding-window attention with sinks on whole sequences, forward or
           forward and backward

Each case runs in its plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the library's entry points; ``exact`` gives the same
outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
MIN_EXP = -100  # smallest exponent of an appended page's scale


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _cache(name, b, h, hk, d, page, t, length, left=-1, sinks=0, layout="bhnd"):
    return {"name": name, "op": "cache", "b": b, "h": h, "hk": hk, "d": d, "page": page, "t": t,
            "len": length, "left": left, "sinks": sinks, "layout": layout}


def _append(name, b, hk, d, page, t, length, layout="bhnd"):
    return {"name": name, "op": "append", "b": b, "hk": hk, "d": d, "page": page, "t": t,
            "len": length, "layout": layout}


def _sinks(name, b, h, hk, n, d, left, sinks, train, layout="bhnd"):
    return {"name": name, "op": "sinks", "b": b, "h": h, "hk": hk, "n": n, "d": d, "left": left,
            "sinks": sinks, "train": train, "layout": layout}


def listed():
    return [
        # one user's chat, next token over a short history: latency alone counts
        _cache("decode_one_short", 1, 32, 8, 128, 64, 1, 1000),
        # a full serving batch of mixed histories (one slot of it empty)
        _cache("decode_batch", 64, 32, 8, 128, 64, 1, 8192),
        # one long document: the keys have to be split over the whole device
        _cache("decode_long", 1, 32, 4, 128, 128, 1, 131000),
        # streaming decode: window and sinks over long histories, a head of keys per query head
        _cache("decode_stream", 32, 16, 16, 64, 32, 1, 32768, left=1023, sinks=4),
        # drafted tokens checked in one call; pages as small as they get
        _cache("draft_tokens", 16, 32, 4, 128, 16, 5, 4096),
        # a chunk of a prompt against what the cache already holds
        _cache("prompt_chunk", 2, 32, 8, 128, 64, 2048, 16384, layout="bnhd"),
        # every decode step of a serving batch writes one token per sequence
        _append("append_token", 32, 8, 128, 64, 1, 4096),
        # prompts of mixed lengths written at once, behind what is there
        _append("append_prompt", 4, 8, 128, 64, 8192, 9000, layout="bnhd"),
        # a small model's forward pass
        _sinks("sinks_fwd_small", 4, 16, 16, 1024, 64, 255, 16, False),
        # a long sequence's forward pass, grouped heads, heads inside the token
        _sinks("sinks_fwd_long", 1, 32, 8, 8192, 128, 1023, 4, False, layout="bnhd"),
        # training on odd lengths, more sinks than a tile holds
        _sinks("sinks_train_odd", 2, 16, 4, 1999, 64, 300, 130, True),
        # training on a long sequence
        _sinks("sinks_train_long", 1, 32, 8, 8192, 128, 1023, 4, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    layout = rng.choice(("bhnd", "bnhd"))
    d = rng.choice((64, 128, 128))
    op = rng.choice(("cache", "cache", "cache", "append", "sinks", "sinks"))
    if op == "cache":
        hk = rng.choice((1, 2, 4, 8, 16))
        h = hk * rng.choice((1, 2, 4, 5, 8, 16))
        page = rng.choice((16, 32, 64, 128))
        t = rng.choice((1, 1, 1, 2, rng.randint(3, 8), _log(rng, 9, 2048)))
        length = max(t, _log(rng, 1, 131072))
        b = _log(rng, 1, 64)
        while b > 1 and (b * hk * length * d > 64 * 8 * 8192 * 128 or
                         b * h * t * length > 2 * 32 * 2048 * 16384):
            b //= 2
        while h * t * length > 2 * 32 * 2048 * 16384:
            t, length = t // 2 + 1, max(t // 2 + 1, length // 2 + 1)
        left, sinks = rng.choice(((-1, 0), (-1, 0), (_log(rng, 16, 4096), rng.choice((0, 1, 4, 64)))))
        return {k: v for k, v in _cache("", b, h, hk, d, page, t, length, left, sinks, layout).items() if k != "name"}
    if op == "append":
        t = rng.choice((1, 1, rng.randint(2, 64), _log(rng, 65, 8192)))
        b = _log(rng, 1, 64) if t == 1 else _log(rng, 1, 4)
        return {k: v for k, v in _append("", b, rng.choice((1, 2, 4, 8)), d, rng.choice((16, 32, 64, 128)), t,
                                         t + _log(rng, 1, 4096), layout).items() if k != "name"}
    hk = rng.choice((1, 2, 4, 8))
    h = hk * rng.choice((1, 2, 4))
    n = _log(rng, 1, 8192)
    b = rng.choice((1, 2, 3))
    while b * h * n * n > 32 * 8192 * 8192:
        n = n // 2 + 1
    return {k: v for k, v in _sinks("", b, h, hk, n, d, _log(rng, 1, 2048), rng.choice((1, 4, 16, 64, 200)),
                                    rng.choice((False, True)), layout).items() if k != "name"}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lens(case):
    """Tokens in the cache of each sequence (new ones included) and new ones of each: mixed
    lengths between a half and the whole; in a batch of 8 or more one slot is empty."""
    b, t, length = case["b"], case["t"], case["len"]
    new = [t - (i * 7919) % (t // 2 + 1) for i in range(b)]
    lens = [max(new[i], length - (i * 104729) % (length // 2 + 1)) for i in range(b)]
    if case["op"] == "cache" and b >= 8:
        lens[3] = new[3] = 0
    return lens, new


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _pool(g, case, pages_per_seq):
    """A pool of filled pages (the last one belongs to nobody), and a table that deals them out."""
    b, hk, d, page = case["b"], case["hk"], case["d"], case["page"]
    n = b * pages_per_seq + 1
    out = []
    for _ in range(2):
        codes = torch.empty((n, hk, page, d), dtype=torch.uint8, device="cuda")
        scale = torch.empty((n, hk), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 28) // (hk * page * d))
        for i in range(0, n, step):
            m = min(step, n - i)
            x = torch.randn((m, hk, page, d), generator=g, device="cuda")
            x *= torch.exp(0.3 * torch.randn((m, hk, 1, 1), generator=g, device="cuda"))
            s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
            codes[i:i + m] = (x / s[:, :, None, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
            scale[i:i + m] = s
        out += [codes, scale]
    table = torch.randperm(n - 1, generator=g, device="cuda").int().view(b, pages_per_seq)
    return out[0], out[2], out[1], out[3], table


def _order(x, layout):
    """[b, heads, tokens, d] data laid out as `layout` says."""
    return x if layout == "bhnd" else x.transpose(1, 2).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    layout = case["layout"]
    if case["op"] == "sinks":
        b, h, hk, n, d = (case[k] for k in ("b", "h", "hk", "n", "d"))
        st["q"], st["k"], st["v"], st["do"] = (_order(_bf16(g, b, heads, n, d), layout)
                                               for heads in (h, hk, hk, h))
        return st
    lens, new = _lens(case)
    st["seq_lens"], st["new_lens"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, new))
    st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["table"] = _pool(
        g, case, -(-max(max(lens), 1) // case["page"]))
    b, t, d = case["b"], case["t"], case["d"]
    if case["op"] == "append":
        size = torch.exp(0.5 * torch.randn((b, case["hk"], t, 1), generator=g, device="cuda"))
        st["k"], st["v"] = (_order((size * torch.randn((b, case["hk"], t, d), generator=g, device="cuda"))
                                   .bfloat16(), layout) for _ in range(2))
    else:
        st["q"] = _order(_bf16(g, b, case["h"], t, d), layout)
        # rows behind a sequence's last query token are left as they are
        st["o"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((b, case["h"], t), device="cuda")
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _heads_first(x, layout):
    return x if layout == "bhnd" else x.transpose(1, 2)


def _visible(pos, j, left, sinks):
    seen = j <= pos
    if left >= 0:
        seen &= (j >= pos - left) | (j < sinks)
    return seen


def _plain_attend(q, k, v, scale, seen):
    """q [b, hk, g, t, d], k and v [b, hk, l, d] in 32 bits; seen broadcasts to [b, hk, g, t, l]."""
    b, hk, grp, t, d = q.shape
    s = torch.matmul(q.reshape(b, hk, grp * t, d), k.transpose(2, 3)).view(b, hk, grp, t, -1) * scale
    s = s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp_(s.sub_(m))
    l = p.sum(-1, keepdim=True)
    empty = l == 0
    p /= torch.where(empty, torch.ones_like(l), l)
    o = torch.matmul(p.view(b, hk, grp * t, -1), v).view(b, hk, grp, t, d)
    lse = torch.where(empty, torch.full_like(l, math.inf), m + torch.log(l)).squeeze(-1)
    return o, lse, p


def _plain_sinks(st):
    b, h, hk, n, d, layout = (st[k] for k in ("b", "h", "hk", "n", "d", "layout"))
    scale = 1.0 / math.sqrt(d)
    q, k, v = (_heads_first(st[x], layout).float() for x in ("q", "k", "v"))
    i = torch.arange(n, device="cuda")
    seen = _visible(i[:, None], i[None, :], st["left"], st["sinks"])
    q = q.reshape(b, hk, h // hk, n, d)
    o, lse, p = _plain_attend(q, k, v, scale, seen)
    out = [_order(o.view(b, h, n, d).bfloat16(), layout), lse.view(b, h, n)]
    if not st["train"]:
        return out
    do = _heads_first(st["do"], layout).float().reshape(b, hk, h // hk, n, d)
    rows = (b, hk, h // hk * n)
    dv = torch.matmul(p.view(*rows, n).transpose(2, 3), do.reshape(*rows, d))
    ds = torch.matmul(do.reshape(*rows, d), v.transpose(2, 3)).view(p.shape)
    ds -= (do * o).sum(-1, keepdim=True)
    ds *= p
    ds *= scale
    dq = torch.matmul(ds.view(*rows, n), k)
    dk = torch.matmul(ds.view(*rows, n).transpose(2, 3), q.reshape(*rows, d))
    return out + [_order(x.view(b, -1, n, d).bfloat16(), layout) for x in (dq, dk, dv)]


def _gathered(pages, scale, table):
    """Every sequence's pages in order, as 32-bit values [b, hk, tokens, d]."""
    b, m = table.shape
    _, hk, page, d = pages.shape
    at = table.long()
    x = pages.view(E4M3)[at].float() * scale[at][..., None, None]
    return x.transpose(1, 2).reshape(b, hk, m * page, d)


def _plain_cache(st):
    b, h, hk, t, d, layout = (st[k] for k in ("b", "h", "hk", "t", "d", "layout"))
    k, v = (_gathered(st[x + "_pages"], st[x + "_scale"], st["table"]) for x in ("k", "v"))
    i = torch.arange(t, device="cuda")
    j = torch.arange(k.shape[2], device="cuda")
    pos = (st["seq_lens"] - st["new_lens"])[:, None] + i
    seen = _visible(pos[:, :, None], j, st["left"], st["sinks"])[:, None, None]
    q = _heads_first(st["q"], layout).float().reshape(b, hk, h // hk, t, d)
    o, lse, _ = _plain_attend(q, k, v, 1.0 / math.sqrt(d), seen)
    there = (i < st["new_lens"][:, None])[:, None]
    o = _order(o.view(b, h, t, d).bfloat16(), layout)
    o = torch.where(there[..., None] if layout == "bhnd" else there.transpose(1, 2)[..., None], o, st["o"])
    return [o, torch.where(there, lse.view(b, h, t), st["lse"])]


def _plain_append_one(st, name, pid, tok, live, has_old, is_old, is_new):
    b, hk, page, t = (st[k] for k in ("b", "hk", "page", "t"))
    n = tok.shape[1]
    pages, scale = st[name + "_pages"].view(E4M3), st[name + "_scale"]
    x = _heads_first(st[name], st["layout"]).float()
    idx = tok.clamp(0, t - 1).view(b, 1, n * page, 1).expand(b, hk, n * page, x.shape[3])
    x = x.gather(2, idx).view(b, hk, n, page, -1).transpose(1, 2)  # [b, n, hk, page, d]
    amax = torch.where(is_new & torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax((3, 4))
    frac, exp = torch.frexp(amax)
    exp = torch.where(frac <= 0.875, exp - 9, exp - 8).clamp(min=MIN_EXP)
    fresh = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, exp, MIN_EXP))
    was, codes = scale[pid], pages[pid].float()
    new = torch.where(has_old & (amax <= 448 * was), was, fresh)
    old_codes = (codes * (was / new)[..., None, None]).clamp(-448, 448)
    new_codes = (x / new[..., None, None]).clamp(-448, 448)
    out = torch.where(is_new, new_codes, torch.where(is_old, old_codes, codes))
    st[name + "_pages"][pid] = out.to(E4M3).view(torch.uint8)
    scale[pid] = torch.where(live[:, :, None], new, was)


def _plain_append(st):
    page, t = st["page"], st["t"]
    first = st["seq_lens"] - st["new_lens"]
    n = (t + page - 2) // page + 1  # pages that t tokens can touch
    at = (first // page)[:, None] + torch.arange(n, device="cuda")
    live = (at * page < st["seq_lens"][:, None]) & (st["new_lens"] > 0)[:, None]
    nobody = st["k_scale"].shape[0] - 1  # written back as it is
    pid = torch.where(live, st["table"].gather(1, at.clamp(max=st["table"].shape[1] - 1).long()), nobody).long()
    tok = at[:, :, None] * page + torch.arange(page, device="cuda") - first[:, None, None]  # [b, n, page]
    is_new = (live[:, :, None] & (tok >= 0) & (tok < st["new_lens"][:, None, None]))[:, :, None, :, None]
    is_old = (live[:, :, None] & (tok < 0))[:, :, None, :, None]
    has_old = (live & (tok[:, :, 0] < 0))[:, :, None]
    slots = (pid, tok, live, has_old, is_old, is_new)
    _plain_append_one(st, "k", *slots)
    _plain_append_one(st, "v", *slots)
    return _append_outputs(st)


def _append_outputs(st):
    return [st["k_pages"].view(E4M3), st["v_pages"].view(E4M3), st["k_scale"], st["v_scale"]]


# ---------------------------------------------------------------------------
# The library's operators
# ---------------------------------------------------------------------------
def _own(st):
    from exact_attention_52_gb300 import api
    if st["op"] == "append":
        api.cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"],
                         st["table"], st["seq_lens"], new_lens=st["new_lens"], layout=st["layout"])
        return _append_outputs(st)
    if st["op"] == "cache":
        return api.fwd_cache(st["q"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["table"],
                             st["seq_lens"], q_lens=st["new_lens"], layout=st["layout"],
                             window_left=st["left"], sinks=st["sinks"], o=st["o"], lse=st["lse"])
    o, lse = api.fwd_sinks(st["q"], st["k"], st["v"], st["left"], st["sinks"], layout=st["layout"])
    if not st["train"]:
        return [o, lse]
    return [o, lse, *api.bwd_sinks(st["q"], st["k"], st["v"], o, st["do"], lse, st["left"], st["sinks"],
                                   layout=st["layout"])]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "cache": _plain_cache, "sinks": _plain_sinks}[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def _pairs(first, last, left, sinks):
    """Visible (query, key) pairs of queries at positions first .. last."""
    def upto(n):  # of the first n queries
        if left < 0 or n <= left + 1:
            return n * (n + 1) // 2
        out, few = n - left - 1, min(n - left - 1, sinks)  # queries past the window; few see only some sinks
        return (left + 1) * (left + 2) // 2 + out * (left + 1) + few * (few + 1) // 2 + (out - few) * sinks
    return upto(last + 1) - upto(first)


def work(case):
    d = case["d"]
    if case["op"] == "sinks":
        b, h, hk, n = (case[k] for k in ("b", "h", "hk", "n"))
        pairs = b * h * _pairs(0, n - 1, case["left"], case["sinks"])
        row = 2 * b * n * d
        fwd = {"bytes": row * (2 * h + 2 * hk) + 4 * b * h * n, "flops": 4 * d * pairs}
        if not case["train"]:
            return fwd
        # backward: q, k, v, o, do and the statistics read, dq, dk and dv written
        return {"bytes": fwd["bytes"] + row * (4 * h + 4 * hk) + 4 * b * h * n, "flops": 14 * d * pairs}
    lens, new = _lens(case)
    hk = case["hk"]
    if case["op"] == "append":
        tokens = sum(new)
        return {"bytes": tokens * hk * d * 2 * 3 + 8 * case["b"] * hk, "flops": 2 * tokens * hk * d * 2}
    keys = pairs = 0
    for length, m in zip(lens, new):
        if m == 0:
            continue
        pairs += _pairs(length - m, length - 1, case["left"], case["sinks"])
        oldest = 0 if case["left"] < 0 else max(0, length - m - case["left"])
        keys += length - oldest + min(case["sinks"], oldest)
    q = sum(new) * case["h"]
    return {"bytes": keys * hk * 2 * (d + 4 / case["page"]) + q * (4 * d + 4), "flops": 4 * d * case["h"] * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _to_e4m3(y):
    """The nearest E4M3 number (ties to even, saturating) to each 64-bit y, by its spacing."""
    a = y.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.copysign(torch.round(a / step) * step, y)


def _exact_append(st):
    lens, new = st["seq_lens"].tolist(), st["new_lens"].tolist()
    table, page = st["table"].tolist(), st["page"]
    out = []
    scales = []
    for name in ("k", "v"):
        vals = st[name + "_pages"].view(E4M3).double()
        scale = st[name + "_scale"].double().clone()
        x = _heads_first(st[name], st["layout"]).double()
        for b, (end, m) in enumerate(zip(lens, new)):
            lo = end - m
            while lo < end:
                slot = lo % page
                cnt = min(page - slot, end - lo)
                pid = table[b][lo // page]
                tok = x[b, :, lo - (end - m):lo - (end - m) + cnt]
                top = tok.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / 448.0))
                e += (top > 448.0 * torch.exp2(e)).double()
                e -= (top <= 448.0 * torch.exp2(e - 1)).double()
                s = torch.exp2(e.clamp(min=MIN_EXP))
                if slot:
                    s = torch.where(top <= 448.0 * scale[pid], scale[pid], s)
                    vals[pid, :, :slot] = _to_e4m3(vals[pid, :, :slot] * (scale[pid] / s)[:, None, None])
                scale[pid] = s
                vals[pid, :, slot:slot + cnt] = _to_e4m3(tok / s[:, None, None])
                lo += cnt
        out.append(vals)
        scales.append(scale)
    return out + scales


def _exact_rows(q, k, v, pos, scale, left, sinks):
    """O, LSE and P of queries q [t, d] at positions pos over keys 0 .. len(k) - 1, in 64 bits."""
    far = torch.arange(k.shape[0], device=k.device)[None, :] - pos[:, None]  # key minus query
    hidden = far > 0
    if left >= 0:
        old = far < -left
        old[:, :sinks] = False
        hidden |= old
    s = (q @ k.T) * scale
    s[hidden] = -math.inf
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    return p @ v, lse, p


def _exact_cache(st):
    lens, new = st["seq_lens"].tolist(), st["new_lens"].tolist()
    q = _heads_first(st["q"], st["layout"]).double()
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    grp, page, d = st["h"] // st["hk"], st["page"], st["d"]
    for b, (length, m) in enumerate(zip(lens, new)):
        if m == 0:
            continue
        ids = st["table"][b, :-(-length // page)].long()
        pos = torch.arange(length - m, length, device="cuda")
        for hk in range(st["hk"]):
            k, v = ((st[x + "_pages"][ids, hk].view(E4M3).double() * st[x + "_scale"][ids, hk].double()[:, None, None])
                    .reshape(-1, d)[:length] for x in ("k", "v"))
            for h in range(hk * grp, hk * grp + grp):
                o[b, h, :m], lse[b, h, :m], _ = _exact_rows(q[b, h, :m], k, v, pos, d ** -0.5, st["left"], st["sinks"])
    return [_order(o, st["layout"]), lse]


def _exact_sinks(st):
    q, k, v, do = (_heads_first(st[x], st["layout"]).double() for x in ("q", "k", "v", "do"))
    b, h, n, d = q.shape
    grp = h // st["hk"]
    scale = d ** -0.5
    o, dq = torch.empty_like(q), torch.empty_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.empty((b, h, n), dtype=torch.float64, device="cuda")
    pos = torch.arange(n, device="cuda")
    for i in range(b):
        for a in range(h):
            c = a // grp
            o[i, a], lse[i, a], p = _exact_rows(q[i, a], k[i, c], v[i, c], pos, scale, st["left"], st["sinks"])
            if st["train"]:
                dv[i, c] += p.T @ do[i, a]
                dp = do[i, a] @ v[i, c].T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                dq[i, a] = ds @ k[i, c]
                dk[i, c] += ds.T @ q[i, a]
    out = [_order(o, st["layout"]), lse]
    return out + [_order(x, st["layout"]) for x in (dq, dk, dv)] if st["train"] else out


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "cache": _exact_cache, "sinks": _exact_sinks}[case["op"]](st)
