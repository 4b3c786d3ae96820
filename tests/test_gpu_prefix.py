"""attn_fwd_cache_prefix against the fp64 oracle of the cache attention, which knows nothing of
shared pages.  Tolerances are those of the cache attention (test_gpu_cache): joining the two parts
adds a few fp32 roundings, 2^-22 of the sums, to the 2^-15 that scores and exponentials have.

A call works in two parts where groups have six sequences on average and the table can hold 256 MB;
here tables are as wide as that needs, the entries behind the sequences' own holding no page, or as
narrow as the sequences are."""

import numpy as np
import pytest

from exact_attention_52_gb300 import api
from oracle import rope as rope_oracle
from oracle import streaming

from .test_gpu_cache import Pool, bf16, check_clean, check_out, i32
from .test_gpu_debug_checks import debug_library
from .test_gpu_rope import THETA, table_of

pytestmark = pytest.mark.gpu


def shared_pool(seed, B, Hk, d, page, firsts, prefixes, lens, token_major=False):
    """A pool whose groups' tables begin with the same pages."""
    pool = Pool(seed, B, Hk, d, page, max(1, -(-max(*lens, *prefixes, 1) // page)), token_major)
    for g, n in enumerate(prefixes):
        for b in range(firsts[g] + 1, firsts[g + 1]):
            pool.table[b, :-(-n // page)] = pool.table[firsts[g], :-(-n // page)]
    return pool


def wide(table, pool):
    """`table` with entries behind, so many that it can hold 256 MB."""
    cols = -(-(1 << 28) // (2 * pool.d * pool.Hk * pool.B * pool.page))
    out = np.full((pool.B, max(cols, table.shape[1])), 10 ** 6, dtype=np.int32)
    out[:, :table.shape[1]] = table
    return out


def run(*args, **kw):
    run_with(*args, **kw)
    run_with(*args, widen=True, **kw)


def run_with(pool, H, T, firsts, prefixes, lens, q_lens, layout="bhnd", amp=1.0, table=None, widen=False, **kw):
    import torch
    q, qv = bf16(pool.rng, (pool.B, H, T, pool.d), layout, amp)
    o = torch.full_like(q, 7.0)
    lse = torch.full((pool.B, H, T), 7.0, device="cuda")
    dev = pool.dev()
    if widen or table is not None:
        table = pool.table if table is None else table
        dev[4] = i32(wide(table, pool) if widen else table)
    args = (q, *dev, i32(lens), i32(prefixes))
    kw.update(group_first=None if firsts is None else i32(firsts), q_lens=None if q_lens is None else i32(q_lens), layout=layout)
    api.fwd_cache_prefix(*args, o=o, lse=lse, **kw)
    check_clean()
    ql = [T] * pool.B if q_lens is None else q_lens
    ref = streaming.cache_forward(qv, pool.k, pool.v, pool.ks, pool.vs, pool.table, lens, ql,
                                  kw.get("scale") or pool.d ** -0.5)
    check_out(o, lse, ref, layout)
    ob = o if layout == "bhnd" else o.transpose(1, 2)
    for b, t in np.argwhere(~ref[3]):
        assert torch.all(ob[b, :, t] == 7.0) and torch.all(lse[b, :, t] == 7.0)
    o2, lse2 = api.fwd_cache_prefix(*args, **kw)  # the same bits again, with tensors of its own
    at = torch.from_numpy(ref[3]).cuda()[:, None]
    oa, ob = ((x if layout == "bhnd" else x.transpose(1, 2)) for x in (o, o2))
    assert torch.equal(torch.where(at[..., None], oa, 0).view(torch.int16), torch.where(at[..., None], ob, 0).view(torch.int16))
    assert torch.equal(torch.where(at, lse, 0).view(torch.int32), torch.where(at, lse2, 0).view(torch.int32))
    return o, lse


# (B, H, Hk, T, page, group_first, prefix_lens, seq_lens, q_lens)
SHAPES = [
    (1, 1, 1, 1, 16, [0, 1], [128], [129], None),
    (6, 1, 1, 1, 16, [0, 6], [128], [129, 129, 130, 128 + 16, 300, 129], None),
    (6, 4, 4, 1, 64, [0, 6], [0], [1, 2, 64, 65, 300, 7], None),
    (7, 8, 2, 1, 16, [0, 7], [127], [128, 300, 129, 128, 200, 512, 140], None),   # shorter than a tile: read for each sequence
    (6, 8, 2, 1, 64, [0, 6], [300], [301, 500, 333, 301, 320, 1000], None),       # not a whole tile, nor a whole page
    (6, 6, 2, 3, 32, [0, 6], [512], [515, 700, 0, 900, 514, 512 + 33], [3, 2, 0, 1, 2, 3]),
    (19, 4, 1, 1, 128, [0, 4, 4, 19], [256, 128, 1280], [257 + 9 * i for i in range(4)] + [1281 + 50 * i for i in range(15)], None),  # an empty group
    (14, 4, 2, 2, 16, [1, 3, 12], [128, 384], [50, 130, 140] + [386 + 7 * i for i in range(9)] + [2, 3], [2] * 14),  # sequences of no group
    (9, 40, 2, 1, 1024, [0, 9], [2048], [2048 + 3 * i + 1 for i in range(9)], None),
    (40, 32, 4, 1, 64, [0, 40], [640], [641 + 7 * i for i in range(40)], None),   # more than one pair of query tiles
    (6, 8, 2, 16, 32, [0, 6], [256], [256 + 16, 700, 300, 272, 280, 256], [16, 13, 1, 16, 9, 0]),  # as many rows as the part kernels take
    (8, 5, 1, 12, 16, [0, 8], [1024], [1036 + 120 * i for i in range(8)], None),
    (5, 4, 1, 1, 128, [0, 2, 2, 5], [256, 128, 1280], [300, 257, 1281, 1400, 2000], None),    # few in a group: one part
    (3, 8, 2, 40, 32, [0, 3], [256], [256 + 40, 700, 300], [40, 33, 1]),                      # prompts: one part
    (4, 5, 1, 100, 64, [0, 2, 4], [900, 256], [1000, 1300, 356, 999], [100, 0, 100, 71]),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("shape", SHAPES)
def test_prefix_matches_oracle(shape, layout, d):
    B, H, Hk, T, page, firsts, prefixes, lens, ql = shape
    pool = shared_pool(7 * B + T, B, Hk, d, page, firsts, prefixes, lens, layout == "bnhd")
    run(pool, H, T, firsts, prefixes, lens, ql, layout)


@pytest.mark.parametrize("d", [64, 128])
def test_range_checked_build(d):
    """The library whose tensor-memory accesses and product operands are checked finds nothing."""
    with debug_library():
        for shape in (SHAPES[4], SHAPES[9], SHAPES[10]):
            B, H, Hk, T, page, firsts, prefixes, lens, ql = shape
            run(shared_pool(B + d, B, Hk, d, page, firsts, prefixes, lens), H, T, firsts, prefixes, lens, ql)


@pytest.mark.parametrize("T", [1, 14, 30])
def test_one_group_by_default_and_a_scale(T):
    lens = [500, 600, 414, 900, 450, 417]
    pool = shared_pool(3, 6, 2, 128, 32, [0, 6], [384], lens)
    run(pool, 8, T, None, [384], lens, None, scale=0.3, amp=2.0)


def test_long_prefix():
    lens = [20000 + 40 * i for i in range(6)]
    pool = shared_pool(4, 6, 1, 64, 64, [0, 6], [19999], lens)
    run(pool, 8, 1, [0, 6], [19999], lens, None)


def test_many_groups():
    """Groups of a few sequences each among many rows, some of them empty or with nothing shared."""
    rng = np.random.default_rng(21)
    B, T = 60, 4
    cuts = sorted(int(x) for x in rng.integers(0, B + 1, 9))
    firsts = [0] + cuts + [B]
    prefixes = [int(x) for x in rng.choice([0, 128, 256, 300, 700], len(firsts) - 1)]
    lens = [0] * B
    for g, n in enumerate(prefixes):
        for b in range(firsts[g], firsts[g + 1]):
            lens[b] = n + T + int(rng.integers(0, 90))
    pool = shared_pool(22, B, 2, 64, 32, firsts, prefixes, lens)
    run(pool, 32, T, firsts, prefixes, lens, [int(x) for x in rng.integers(0, T + 1, B)])


@pytest.mark.parametrize("T", [1, 15, 40])
def test_a_slot_without_queries_may_hold_any_table(T):
    """The first sequence of a group that has queries stands for it; tables of the others are not read."""
    lens, ql = [0, 500, 700, 0, 450, 431], [0, T, T, 0, T, 1]
    pool = shared_pool(5, 6, 2, 64, 16, [0, 6], [384], lens)
    junk = pool.table.copy()
    junk[0], junk[3] = 10 ** 6, -5
    run(pool, 4, T, [0, 6], [384], lens, ql, table=junk)


def test_a_group_without_queries():
    lens, ql = [0, 0] + [257 + 20 * i for i in range(10)], [0, 0] + [1] * 10
    pool = shared_pool(6, 12, 2, 128, 16, [0, 2, 12], [128, 256], lens)
    junk = pool.table.copy()
    junk[:2] = 10 ** 6
    run(pool, 4, 1, [0, 2, 12], [128, 256], lens, ql, table=junk)


@pytest.mark.parametrize("T", [1, 15, 40])
@pytest.mark.parametrize("where", ["prefix", "rest", "both"])
def test_value_scales_far_apart(where, T):
    """Parts whose sums are taken apart join with parts whose sums are not."""
    lens = [400, 512, 700, 333, 296, 450]
    pool = shared_pool(8, 6, 2, 128, 64, [0, 6], [256], lens)
    for b in range(6):
        for pg in range(pool.table.shape[1]):
            if where == "both" or (pg < 4) == (where == "prefix"):
                pool.vs[pool.table[b, pg]] = 2.0 ** (-100 if (b + pg) % 2 or pg < 4 else 60)
    run(pool, 4, T, [0, 6], [256], lens, None)


@pytest.mark.parametrize("T", [1, 15, 40])
def test_nan_values_reach_the_rows_that_see_them(T):
    lens = [300, 400, 310, 297, 500, 450]
    for pg, col in ((1, 3), (None, 5)):  # in the prefix; behind the second sequence's last token
        pool = shared_pool(9, 6, 1, 64, 64, [0, 6], [256], lens)
        if pg is not None:
            pool.v[pool.table[0, pg], 0, 10, col] = 0x7F
        else:
            pool.v[pool.table[1, 400 // 64], 0, 400 % 64, col] = 0x7F
            pool.k[pool.table[1, 400 // 64], 0, 400 % 64, col] = 0xFF
        run(pool, 4, T, [0, 6], [256], lens, None)


def test_lengths_that_do_not_fit_are_reported():
    import torch
    pool = shared_pool(10, 6, 2, 64, 16, [0, 6], [256], [300] * 6)
    q = torch.randn(6, 4, 2, 64, device="cuda").bfloat16()
    dev, narrow = pool.dev(), pool.dev()
    dev[4] = i32(wide(pool.table, pool))
    good = [300, 290, 280, 258, 300, 270]
    call = lambda dev, lens=good, prefix=256: api.fwd_cache_prefix(q, *dev, i32(lens), i32([prefix]))
    call(dev)
    check_clean()
    for short in (257, 2, 0):
        lens = good[:1] + [short] + good[2:]
        call(dev, lens)
        assert api.check_device_error()[0] == -5
        # in one part the prefix says nothing
        got, ref = call(narrow, lens), api.fwd_cache(q, *narrow, i32(lens))
        check_clean()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for kw in (dict(lens=[300, -7, 280, 270, 300, 290]), dict(lens=[300, 2 ** 30, 280, 270, 300, 290]), dict(prefix=2 ** 30),
               dict(prefix=-1)):
        call(dev, **kw)
        assert api.check_device_error()[0] == -5, kw
    bad = pool.table.copy()
    bad[0, 3] = 10 ** 6
    dev[4] = i32(wide(bad, pool))
    call(dev)
    assert api.check_device_error()[0] == -5


def test_captured_calls_follow_their_lengths():
    """Lengths, prefixes and groups stay on the device; two captured calls have workspaces of their own."""
    import torch
    pool = shared_pool(11, 12, 2, 128, 64, [0, 12], [512], [600] * 12)
    dev = pool.dev()
    dev[4] = i32(wide(pool.table, pool))
    q = torch.randn(12, 8, 1, 128, device="cuda").bfloat16()
    seq, pre, first = i32([520 + 4 * i for i in range(12)]), i32([512, 512]), i32([0, 5, 12])
    call = lambda: api.fwd_cache_prefix(q, *dev, seq, pre, group_first=first)
    call()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    s = torch.cuda.Stream()
    for step in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            graphs[1][0].replay()
        s.synchronize()
        torch.cuda.synchronize()
        ref = call()
        for _, out in graphs:
            assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
        seq += 9
        pre.copy_(i32([256, 384]))
        first.copy_(i32([0, 7, 12]))
    check_clean()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = api.fwd_cache_prefix(q, *dev, seq, pre, group_first=first, stream=s)
    s.synchronize()
    ref = call()
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_two_calls_at_once():
    """Calls on two streams, each with the workspace kept for its stream."""
    import torch
    pool = shared_pool(31, 8, 2, 128, 64, [0, 8], [1024], [1100 + 9 * i for i in range(8)])
    dev = pool.dev()
    dev[4] = i32(wide(pool.table, pool))
    lens, pre = i32([1100 + 9 * i for i in range(8)]), i32([1024])
    qs = [torch.randn(8, 16, 2, 128, device="cuda").bfloat16() for _ in range(2)]
    call = lambda q: api.fwd_cache_prefix(q, *dev, lens, pre)
    ref = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = call(qs[i])
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_clean()


def test_decoding_behind_a_shared_prompt():
    """The operators as they are used: a prompt written and rotated once, then steps of a few tokens
    of six sequences behind it, each written, rotated and attended in two calls."""
    import torch
    B, H, Hk, d, page, prompt = 6, 8, 2, 128, 32, 320
    rng = np.random.default_rng(12)
    pool = shared_pool(12, B, Hk, d, page, [0, B], [prompt], [prompt + 40] * B)
    dev, table = pool.dev(), table_of(64)
    dev[4] = i32(wide(pool.table, pool))
    w = torch.from_numpy(rng.uniform(0.5, 1.5, d).astype(np.float32)).cuda()
    kw = dict(q_weight=w, k_weight=w, layout="bnhd")
    new = lambda b, t, h: torch.from_numpy(rng.standard_normal((b, t, h, d)).astype(np.float32)).bfloat16().cuda()
    # the prompt, as the first sequence's
    one = [*dev[:4], dev[4][:1]]
    api.cache_append_rope(new(1, prompt, H), new(1, prompt, Hk), new(1, prompt, Hk), table, *one, i32([prompt]), **kw)
    lens = np.full(B, prompt)
    for step in range(12):
        T = 1 + step % 3
        m = [T, (step + 1) % (T + 1), T, T, step % (T + 1), T]
        lens = lens + m
        q, k, v = new(B, T, H), new(B, T, Hk), new(B, T, Hk)
        seq, nl = i32(lens), i32(m)
        qr = api.cache_append_rope(q, k, v, table, *dev, seq, new_lens=nl, q_out=torch.zeros_like(q), **kw)
        o, lse = api.fwd_cache_prefix(qr, *dev, seq, i32([prompt]), q_lens=nl, layout="bnhd")
        check_clean()
        # the oracle on what the cache holds now, queries rotated by the oracle
        kc, vc = (x.cpu().numpy() for x in dev[:2])
        ks, vs = (x.double().cpu().numpy() for x in dev[2:4])
        qv = qr.transpose(1, 2).double().cpu().numpy()
        ref = streaming.cache_forward(qv, kc, vc, ks, vs, pool.table, lens, m, d ** -0.5)
        check_out(o, lse, ref, "bnhd")
        x = q.transpose(1, 2).double().cpu().numpy()
        pos = lens[:, None] - np.asarray(m)[:, None] + np.arange(T)
        y, size = rope_oracle.forward(x, rope_oracle.angles(pos, THETA[64])[:, None], 1.0, 64, False, w.double().cpu().numpy())
        there = ref[3][:, None, :, None]
        assert np.all(np.where(there, np.abs(qv - y) <= 2.0 ** -20 * size + 2.0 ** -8 * (np.abs(y) + size), qv == 0))


def test_arguments_that_are_refused():
    import torch
    pool = shared_pool(13, 2, 2, 64, 16, [0, 2], [128], [140, 150])
    dev = pool.dev()
    q, lens, pre = torch.randn(2, 4, 1, 64, device="cuda").bfloat16(), i32([140, 150]), i32([128])
    api.fwd_cache_prefix(q, *dev, lens, pre)
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]), dict(q=torch.randn(2, 3, 1, 64, device="cuda").bfloat16()),
           dict(prefix_lens=pre.long()), dict(prefix_lens=pre.cpu()), dict(prefix_lens=i32([[128]])), dict(prefix_lens=i32([])),
           dict(prefix_lens=i32([128, 128])), dict(prefix_lens=i32([1, 1, 1]), group_first=i32([0, 1, 1, 2])),
           dict(group_first=i32([0, 1, 2])), dict(group_first=i32([0])), dict(q_lens=i32([1])), dict(layout="nbhd"),
           dict(o=q.float()), dict(lse=torch.zeros(2, 4, device="cuda")), dict(k_pages=dev[0][0]),
           dict(workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))]
    for b in bad:
        a = dict(q=q, k_pages=dev[0], v_pages=dev[1], k_scale=dev[2], v_scale=dev[3], page_table=dev[4], seq_lens=lens,
                 prefix_lens=pre)
        a.update(b)
        with pytest.raises(ValueError):
            api.fwd_cache_prefix(**a)
    with pytest.raises(api.AttnError):
        api.fwd_cache_prefix(q, *dev, lens, pre, scale=0.0)
    with pytest.raises(api.AttnError):
        api.fwd_cache_prefix(q, *dev, lens, pre, o=q[:, :1].expand(2, 4, 1, 64))
