"""What lies between the projections and the attention, and a cache whose sequences share their first
tokens, measured:

  rope     rotary positions on the heads of queries and keys (interleaved or half layout, part of
           the head, frequencies scaled for long contexts), optionally with a norm of each head in
           the same pass; forward, or forward and backward
  append   a serving step's write: new tokens' queries and keys normed and rotated, keys and values
           written into the paged 8-bit cache (E4M3 codes, one power-of-two scale per page, head and
           tensor), queries given back for the attention
  prefix   attention of new query tokens over that cache in a batch whose groups of sequences share
           the pages of a long prefix

Each case runs in its plain form (elementary torch operations in 32 bits, angles in 64) or, with
``own`` set, through the library's entry points; ``exact`` gives the same outputs from the
definitions in 64 bits.
"""

import functools
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
MIN_EXP = -100  # smallest exponent of an appended page's scale
BASE = 10000.0
TRAINED = 4096  # context length that scaled frequencies start from
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _rope(name, b, h, hk, n, d, rot, pairs, scaling, norm, train, given=False, layout="bhnd"):
    return {"name": name, "op": "rope", "b": b, "h": h, "hk": hk, "n": n, "d": d, "rot": rot, "pairs": pairs,
            "scaling": scaling, "norm": norm, "train": train, "given": given, "layout": layout}


def _append(name, b, h, hk, d, rot, pairs, scaling, norm, page, t, length, layout="bnhd"):
    return {"name": name, "op": "append", "b": b, "h": h, "hk": hk, "d": d, "rot": rot, "pairs": pairs,
            "scaling": scaling, "norm": norm, "page": page, "t": t, "len": length, "layout": layout}


def _prefix(name, b, groups, h, hk, d, page, t, prefix, length, layout="bhnd"):
    return {"name": name, "op": "prefix", "b": b, "groups": groups, "h": h, "hk": hk, "d": d, "page": page,
            "t": t, "prefix": prefix, "len": length, "layout": layout}


def listed():
    return [
        # one token of each of a few chats, positions handed over: latency alone counts
        _rope("rope_tokens", 4, 32, 8, 1, 128, 128, "half", "none", False, False, given=True, layout="bnhd"),
        # a small model's forward pass that rotates half of each head
        _rope("rope_fwd_small", 4, 16, 16, 1024, 64, 32, "interleaved", "none", False, False),
        # a long sequence's forward pass, stretched context, heads inside the token
        _rope("rope_fwd_long", 1, 32, 8, 8192, 128, 128, "half", "yarn", False, False, layout="bnhd"),
        # training on odd lengths and packed documents, with norms
        _rope("norm_rope_train_odd", 2, 16, 4, 1999, 64, 64, "half", "ntk", True, True, given=True),
        # training on a long sequence, with norms
        _rope("norm_rope_train_long", 1, 32, 8, 8192, 128, 128, "half", "none", True, True, layout="bnhd"),
        # every decode step of a serving batch
        _append("append_token", 32, 32, 8, 128, 128, "half", "yarn", True, 64, 1, 4096),
        # drafted tokens, pages as small as they get, part of the head rotated
        _append("append_draft", 16, 32, 4, 128, 64, "interleaved", "linear", False, 16, 5, 4096),
        # prompts of mixed lengths written at once, behind what is there
        _append("append_prompt", 4, 32, 8, 128, 128, "half", "none", True, 64, 8192, 9000),
        # a few chats behind one system prompt: latency
        _prefix("prefix_few", 4, 1, 32, 8, 128, 64, 1, 2048, 300),
        # a full serving batch behind one long prompt (one slot of it empty)
        _prefix("prefix_batch", 64, 1, 32, 8, 128, 64, 1, 8192, 1024),
        # several prompts in a batch, drafted tokens, small heads
        _prefix("prefix_groups", 48, 3, 16, 4, 64, 32, 4, 4096, 500, layout="bnhd"),
        # many questions about one long document
        _prefix("prefix_document", 32, 1, 32, 4, 128, 128, 1, 131072, 400),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    layout = rng.choice(("bhnd", "bnhd"))
    d = rng.choice((64, 128, 128))
    op = rng.choice(("rope", "rope", "append", "append", "prefix", "prefix"))
    rot = rng.choice((d, d, d // 2, rng.choice(range(16, d + 1, 16))))
    pairs = rng.choice(("half", "interleaved"))
    scaling = rng.choice(("none", "linear", "ntk", "yarn"))
    norm = rng.choice((False, True))
    hk = rng.choice((1, 2, 4, 8))
    h = hk * rng.choice((1, 2, 4, 5))
    if op == "rope":
        b, n = rng.choice((1, 2, 3, 8)), _log(rng, 1, 8192)
        while b * (h + hk) * n * d > 40 * 8192 * 128:
            n = n // 2 + 1
        c = _rope("", b, h, hk, n, d, rot, pairs, scaling, norm, rng.choice((False, True)), rng.choice((False, True)), layout)
    elif op == "append":
        t = rng.choice((1, 1, rng.randint(2, 64), _log(rng, 65, 8192)))
        b = _log(rng, 1, 64) if t <= 64 else _log(rng, 1, 4)
        while b > 1 and b * t * (2 * h + 3 * hk) * d > 27000 * 88 * 128:
            b -= 1
        c = _append("", b, h, hk, d, rot, pairs, scaling, norm, rng.choice((16, 32, 64, 128)), t,
                    t + _log(rng, 1, 4096), layout)
    else:
        groups = rng.choice((1, 1, 2, 3))
        b, t = groups * _log(rng, 1, 32), rng.choice((1, 1, 2, rng.randint(3, 8), _log(rng, 9, 300)))
        page = rng.choice((16, 32, 64, 128))
        prefix, length = page * _log(rng, 1, 131072 // page), t + _log(rng, 1, 2000)
        while b > groups and b * hk * (length + t * h // hk) * d > 64 * 8 * 1024 * 128:
            b -= groups
        while b * h * t * (prefix + length) > 32 * 32 * 131072 or groups * hk * prefix > 8 * 131072:
            prefix = max(page, prefix // 2 // page * page)
            if prefix == page:
                t, length = t // 2 + 1, length // 2 + t // 2 + 1
        c = _prefix("", b, groups, h, hk, d, page, t, prefix, length, layout)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lens(case):
    """Tokens in the cache of each sequence (new ones and a prefix included) and new ones of each: mixed
    lengths between a half and the whole; in a batch of 8 or more one slot is empty."""
    b, t, length = case["b"], case["t"], case["len"]
    new = [t - (i * 7919) % (t // 2 + 1) for i in range(b)]
    lens = [max(new[i], length - (i * 104729) % (length // 2 + 1)) + case.get("prefix", 0) for i in range(b)]
    if case["op"] == "prefix" and b >= 8:
        lens[3] = new[3] = 0
    return lens, new


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _order(x, layout):
    """[b, heads, tokens, d] data laid out as `layout` says."""
    return x if layout == "bhnd" else x.transpose(1, 2).contiguous()


def _heads(g, case, heads, n):
    """Projections' outputs: every head of every token at a size of its own."""
    shape = (case["b"], heads, n)
    size = torch.exp(0.3 * torch.randn((*shape, 1), generator=g, device="cuda"))
    return _order((size * torch.randn((*shape, case["d"]), generator=g, device="cuda")).bfloat16(), case["layout"])


def _codes(g, n, hk, page, d):
    """Filled pages: codes and scales."""
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
    return codes, scale


def _pool(g, case, shared, own_pages):
    """A pool of filled pages (the last one belongs to nobody) and the sequences' table: `shared`
    pages of its group before `own_pages` of its own."""
    b, groups = case["b"], case.get("groups", 1)
    n = groups * shared + b * own_pages + 1
    ids = torch.randperm(n - 1, generator=g, device="cuda").int()
    mine = ids[groups * shared:].view(b, own_pages)
    common = ids[:groups * shared].view(groups, 1, shared).expand(groups, b // groups, shared).reshape(b, shared)
    table = torch.cat([common, mine], 1).contiguous()
    out = [_codes(g, n, case["hk"], case["page"], case["d"]) for _ in range(2)]
    return {"k_pages": out[0][0], "v_pages": out[1][0], "k_scale": out[0][1], "v_scale": out[1][1], "table": table}


def _frequencies(case):
    """Angle per position of each pair, and what cosine and sine are multiplied by (64 bits)."""
    rot, scaling, s = case["rot"], case["scaling"], 4.0
    base = BASE * s ** (rot / (rot - 2)) if scaling == "ntk" else BASE
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / s for x in theta], 1.0
    if scaling == "yarn":  # pairs that turn often within the trained length stay, those that never turn are stretched
        keep = [min(1.0, max(0.0, (TRAINED * x / (2.0 * math.pi) - 1.0) / 31.0)) for x in theta]
        return [x * (k + (1.0 - k) / s) for x, k in zip(theta, keep)], 0.1 * math.log(s) + 1.0
    return theta, 1.0


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    b, h, hk, d = (case[k] for k in ("b", "h", "hk", "d"))
    if case["op"] != "prefix":
        theta, st["factor"] = _frequencies(case)
        st["theta"] = torch.tensor(theta, dtype=torch.float64, device="cuda")
        st["weights"] = [1.3 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in "qk"] if case["norm"] else [None, None]
    if case["op"] == "rope":
        n = case["n"]
        st["q"], st["k"] = (_heads(g, case, x, n) for x in (h, hk))
        if case["train"]:
            st["dq_out"], st["dk_out"] = (_order(_bf16(g, b, x, n, d), case["layout"]) for x in (h, hk))
        # packed documents, far into a long text
        start = torch.randint(0, 1 << 17, (b, 1), generator=g, device="cuda")
        st["positions"] = (start + torch.arange(n, device="cuda") % max(1, n * 3 // 5)).int() if case["given"] else None
        return st
    lens, new = _lens(case)
    t, page = case["t"], case["page"]
    st["seq_lens"], st["new_lens"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, new))
    if case["op"] == "append":
        st.update(_pool(g, case, 0, -(-max(max(lens), 1) // page)))
        st["q"], st["k"], st["v"] = (_heads(g, case, x, t) for x in (h, hk, hk))
        st["q_out"] = torch.zeros_like(st["q"])  # rows behind a sequence's new tokens are left as they are
        return st
    shared = case["prefix"] // page
    st.update(_pool(g, case, shared, max(1, -(-max(lens) // page) - shared)))
    st["group_first"] = torch.arange(0, b + 1, b // case["groups"], dtype=torch.int32, device="cuda")
    st["prefix_lens"] = torch.full((case["groups"],), case["prefix"], dtype=torch.int32, device="cuda")
    st["q"] = _order(_bf16(g, b, h, t, d), case["layout"])
    st["o"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros((b, h, t), device="cuda")
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _heads_first(x, layout):
    return x if layout == "bhnd" else x.transpose(1, 2)


def _turn(st, positions):
    """Cosines and sines [b or 1, 1, n, rot/2] of the positions [b or 1, n], angles in 64 bits."""
    a = positions.double()[:, None, :, None] * st["theta"]
    return (torch.cos(a) * st["factor"]).float(), (torch.sin(a) * st["factor"]).float()


def _rotate(x, c, s, rot, pairs):
    """x [b, heads, n, d]: its first rot elements rotated."""
    if pairs == "half":
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
    else:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _unit(x):
    """A head over its root mean square, and that one's inverse."""
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_rope(st):
    rot, pairs, layout = st["rot"], st["pairs"], st["layout"]
    pos = st["positions"] if st["given"] else torch.arange(st["n"], device="cuda")[None]
    c, s = _turn(st, pos)
    out, grads, dws = [], [], []
    for name, w in zip("qk", st["weights"]):
        x = _heads_first(st[name], layout).float()
        u, r = _unit(x) if st["norm"] else (x, None)
        out.append(_order(_rotate(u * w if st["norm"] else u, c, s, rot, pairs).bfloat16(), layout))
        if st["train"]:
            dn = _rotate(_heads_first(st["d" + name + "_out"], layout).float(), c, -s, rot, pairs)
            if st["norm"]:
                dws.append((dn * u).sum((0, 1, 2)))
                dn = dn * w
                dn = (dn - u * (dn * u).mean(-1, keepdim=True)) * r
            grads.append(_order(dn.bfloat16(), layout))
    return out + grads + dws


def _plain_append_one(st, name, x, pid, tok, live, has_old, is_old, is_new):
    """x: the new tokens' values in 32 bits [b, hk, t, d]."""
    b, hk, page, t = (st[k] for k in ("b", "hk", "page", "t"))
    n = tok.shape[1]
    pages, scale = st[name + "_pages"].view(E4M3), st[name + "_scale"]
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
    page, t, layout = st["page"], st["t"], st["layout"]
    first = st["seq_lens"] - st["new_lens"]
    i = torch.arange(t, device="cuda")
    c, s = _turn(st, first[:, None] + i)
    q, k = (_heads_first(st[x], layout).float() for x in "qk")
    if st["norm"]:
        q, k = (_unit(x)[0] * w for x, w in zip((q, k), st["weights"]))
    q, k = (_rotate(x, c, s, st["rot"], st["pairs"]) for x in (q, k))
    there = (i < st["new_lens"][:, None])[:, None, :, None]
    q_out = torch.where(there, q.bfloat16(), _heads_first(st["q_out"], layout))
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
    _plain_append_one(st, "k", k, *slots)
    _plain_append_one(st, "v", _heads_first(st["v"], layout).float(), *slots)
    return [_order(q_out, layout), *_cache_of(st)]


def _cache_of(st):
    return [st["k_pages"].view(E4M3), st["v_pages"].view(E4M3), st["k_scale"], st["v_scale"]]


def _gathered(pages, scale, table):
    """Pages of each row of the table in order, as 32-bit values [rows, hk, tokens, d]."""
    rows, m = table.shape
    _, hk, page, d = pages.shape
    at = table.long()
    x = pages.view(E4M3)[at].float() * scale[at][..., None, None]
    return x.transpose(1, 2).reshape(rows, hk, m * page, d)


def _plain_prefix(st):
    b, h, hk, t, d, groups, layout = (st[k] for k in ("b", "h", "hk", "t", "d", "groups", "layout"))
    each, grp, shared = b // groups, h // hk, st["prefix"] // st["page"]
    # the prefix once for each group, the rest for each sequence
    kp, vp = (_gathered(st[x + "_pages"], st[x + "_scale"], st["table"][::each, :shared]) for x in "kv")
    ko, vo = (_gathered(st[x + "_pages"], st[x + "_scale"], st["table"][:, shared:]) for x in "kv")
    q = _heads_first(st["q"], layout).float() / math.sqrt(d)
    q = q.reshape(groups, each, hk, grp * t, d).transpose(1, 2)  # [groups, hk, each, rows, d]
    sp = torch.matmul(q.reshape(groups, hk, each * grp * t, d), kp.transpose(2, 3))
    q = q.transpose(1, 2).reshape(b, hk, grp * t, d)
    so = torch.matmul(q, ko.transpose(2, 3)).view(b, hk, grp, t, -1)
    i = torch.arange(t, device="cuda")
    pos = (st["seq_lens"] - st["new_lens"])[:, None] + i - st["prefix"]
    seen = torch.arange(ko.shape[2], device="cuda") <= pos[:, :, None]
    so = so.masked_fill_(~seen[:, None, None], -math.inf).view(b, hk, grp * t, -1)
    sp = sp.view(groups, hk, each, grp * t, -1)
    so = so.view(groups, each, hk, grp * t, -1).transpose(1, 2)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    pp, po = torch.exp_(sp.sub_(m)), torch.exp(so - m)
    l = pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
    o = torch.matmul(pp.view(groups, hk, each * grp * t, -1), vp).view(groups, hk, each, grp * t, d)
    o = o + torch.matmul(po.transpose(1, 2).reshape(b, hk, grp * t, -1), vo).view(groups, each, hk, grp * t, d).transpose(1, 2)
    o = (o / l).transpose(1, 2).reshape(b, h, t, d)
    lse = (m + torch.log(l)).transpose(1, 2).reshape(b, h, t)
    there = (i < st["new_lens"][:, None])[:, None]
    o = torch.where(there[..., None], o.bfloat16(), _heads_first(st["o"], layout))
    return [_order(o, layout), torch.where(there, lse, st["lse"])]


# ---------------------------------------------------------------------------
# The library's operators
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _table(rot, pairs, scaling):
    """The table of frequencies that a program lays out once, when it loads its model."""
    from exact_attention_52_gb300 import api
    return api.rope_table(rot, base=BASE, scaling=None if scaling == "none" else scaling, factor=4.0,
                          original_len=TRAINED, interleaved=pairs == "interleaved")


def _own(st):
    from exact_attention_52_gb300 import api
    if st["op"] == "prefix":
        return api.fwd_cache_prefix(st["q"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["table"],
                                    st["seq_lens"], st["prefix_lens"], group_first=st["group_first"],
                                    q_lens=st["new_lens"], layout=st["layout"], o=st["o"], lse=st["lse"])
    table, (wq, wk), layout = _table(st["rot"], st["pairs"], st["scaling"]), st["weights"], st["layout"]
    if st["op"] == "append":
        q = api.cache_append_rope(st["q"], st["k"], st["v"], table, st["k_pages"], st["v_pages"], st["k_scale"],
                                  st["v_scale"], st["table"], st["seq_lens"], new_lens=st["new_lens"], q_weight=wq,
                                  k_weight=wk, eps=EPS, layout=layout, q_out=st["q_out"])
        return [q, *_cache_of(st)]
    out = api.rope(st["q"], st["k"], table, positions=st["positions"], q_weight=wq, k_weight=wk, eps=EPS, layout=layout)
    if not st["train"]:
        return out
    grads = api.rope_bwd(st["dq_out"], st["dk_out"], table, positions=st["positions"], q=st["q"], k=st["k"], q_weight=wq,
                         k_weight=wk, eps=EPS, layout=layout)
    return [*out, *grads[:2], *(grads[2:] if st["norm"] else ())]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "prefix": _plain_prefix}[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    b, h, hk, d = (case[k] for k in ("b", "h", "hk", "d"))
    if case["op"] == "rope":
        rows = b * (h + hk) * case["n"]
        passes = 2 + (0 if not case["train"] else 3 if case["norm"] else 2)
        return {"bytes": 2 * d * rows * passes + 4 * b * case["n"] * case["given"],
                "flops": rows * (3 * case["rot"] + 4 * d * case["norm"]) * (3 if case["train"] else 1)}
    lens, new = _lens(case)
    if case["op"] == "append":
        tokens = sum(new)
        return {"bytes": tokens * d * (4 * h + 2 * hk * 3) + 8 * b * hk,
                "flops": tokens * ((h + hk) * (3 * case["rot"] + 4 * d * case["norm"]) + 4 * hk * d)}
    rows = sum(new)
    keys = case["groups"] * case["prefix"] + sum(max(0, x - case["prefix"]) for x in lens)
    pairs = sum(m * x - m * (m - 1) // 2 for x, m in zip(lens, new))
    return {"bytes": keys * hk * 2 * (d + 4 / case["page"]) + rows * h * (4 * d + 4), "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_matrix(st, positions):
    """The rotation of each position as complex factors [b or 1, 1, n, rot/2]."""
    a = positions.double()[:, None, :, None] * torch.tensor(_frequencies(st)[0], dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(a, _frequencies(st)[1]), a)


def _exact_turn(x, z, st):
    """x's pairs as complex numbers, times z."""
    rot, n = st["rot"], st["rot"] // 2
    first = torch.arange(n, device="cuda") * (1 if st["pairs"] == "half" else 2)
    second = first + (n if st["pairs"] == "half" else 1)
    y = torch.complex(x[..., first], x[..., second]) * z
    out = x.clone()
    out[..., first], out[..., second] = y.real, y.imag
    return out


def _exact_norm(x, w):
    rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) ** 0.5
    return x / rms * w.double()


def _exact_rope(st):
    pos = st["positions"].long() if st["given"] else torch.arange(st["n"], device="cuda")[None]
    z = _exact_matrix(st, pos)
    out, grads, dws = [], [], []
    for name, w in zip("qk", st["weights"]):
        x = _heads_first(st[name], st["layout"]).double()
        y = _exact_turn(_exact_norm(x, w) if st["norm"] else x, z, st)
        out.append(_order(y, st["layout"]))
        if not st["train"]:
            continue
        dn = _exact_turn(_heads_first(st["d" + name + "_out"], st["layout"]).double(), z.conj(), st)
        if st["norm"]:
            d = x.shape[-1]
            rms = ((x * x).sum(-1, keepdim=True) / d + EPS) ** 0.5
            dws.append(torch.einsum("bhnd,bhnd->d", dn, x / rms))
            up = dn * w.double()
            dn = up / rms - x * (up * x).sum(-1, keepdim=True) / (d * rms ** 3)
        grads.append(_order(dn, st["layout"]))
    return out + grads + dws


def _to_e4m3(y):
    """The nearest E4M3 number (ties to even, saturating) to each 64-bit y, by its spacing."""
    a = y.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.copysign(torch.round(a / step) * step, y)


def _exact_append(st):
    lens, new = st["seq_lens"].tolist(), st["new_lens"].tolist()
    table, page = st["table"].tolist(), st["page"]
    pos = (st["seq_lens"] - st["new_lens"]).long()[:, None] + torch.arange(st["t"], device="cuda")
    z = _exact_matrix(st, pos)
    turned = {}
    for name, w in zip("qk", st["weights"]):
        x = _heads_first(st[name], st["layout"]).double()
        turned[name] = _exact_turn(_exact_norm(x, w) if st["norm"] else x, z, st)
    turned["v"] = _heads_first(st["v"], st["layout"]).double()
    q = torch.zeros_like(turned["q"])
    for b, m in enumerate(new):
        q[b, :, :m] = turned["q"][b, :, :m]
    out, scales = [], []
    for name in "kv":
        vals = st[name + "_pages"].view(E4M3).double()
        scale = st[name + "_scale"].double().clone()
        for b, (end, m) in enumerate(zip(lens, new)):
            lo = end - m
            while lo < end:
                slot = lo % page
                cnt = min(page - slot, end - lo)
                pid = table[b][lo // page]
                tok = turned[name][b, :, lo - (end - m):lo - (end - m) + cnt]
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
    return [_order(q, st["layout"]), *out, *scales]


def _exact_prefix(st):
    """Sequence by sequence over its whole table, as if nothing were shared."""
    lens, new = st["seq_lens"].tolist(), st["new_lens"].tolist()
    q = _heads_first(st["q"], st["layout"]).double()
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    grp, page, d = st["h"] // st["hk"], st["page"], st["d"]
    for b, (length, m) in enumerate(zip(lens, new)):
        if m == 0:
            continue
        ids = st["table"][b, :-(-length // page)].long()
        hidden = torch.arange(length, device="cuda") > torch.arange(length - m, length, device="cuda")[:, None]
        for hk in range(st["hk"]):
            k, v = ((st[x + "_pages"][ids, hk].view(E4M3).double() * st[x + "_scale"][ids, hk].double()[:, None, None])
                    .reshape(-1, d)[:length] for x in "kv")
            s = (q[b, hk * grp:hk * grp + grp, :m] @ k.T) * d ** -0.5
            s = s.masked_fill(hidden, -math.inf)
            lse[b, hk * grp:hk * grp + grp, :m] = torch.logsumexp(s, -1)
            o[b, hk * grp:hk * grp + grp, :m] = torch.softmax(s, -1) @ v
    return [_order(o, st["layout"]), lse]


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "prefix": _exact_prefix}[case["op"]](st)
