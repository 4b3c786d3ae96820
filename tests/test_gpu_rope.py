"""attn_rope, attn_rope_bwd and attn_cache_append_rope against the fp64 oracle.

Tolerances.  A cosine or sine is off by at most 2^-22.3: the angle off the nearest quarter turn goes
to fp32 (2^-25 of at most pi / 4), the function and the factor add a step each (2^-24 of at most 1,
twice).  A normed element is off by 2^-21 of itself: the sum of up to 128 squares in a
tree (2^-24 times 12 additions, halved by the square root), the inverse root (two steps) and two
products.  So a rotated element is off by e = 2^-20 (|n1| + |n2|) f before it is rounded to bf16,
  |y - ref| <= e + 2^-8 (|ref| + e);
a gradient, in the same way with the mean over the head, by 2^-19 of the sum of its terms'
magnitudes, and a weight's gradient by 2^-15 of them: 2^-20 a term and 2^-24 for each of the at
most 400 additions that a term goes through here."""

import numpy as np
import pytest

from exact_attention_52_gb300 import api
from oracle import rope, streaming
from oracle.attention import _E4M3

from .helpers import device_bf16_to_f64
from .test_gpu_cache import Pool, bf16, check_clean, i32

pytestmark = pytest.mark.gpu


def heads(t, layout):
    return device_bf16_to_f64(t if layout == "bhnd" else t.transpose(1, 2))


def weight(rng, d, dtype="fp32"):
    """A weight on the device, and its values."""
    import torch
    w = torch.from_numpy((1.0 + 0.3 * rng.standard_normal(d)).astype(np.float32))
    w = w.bfloat16() if dtype == "bf16" else w
    return w.cuda(), w.double().numpy()


def close(got, ref, e):
    bad = ~(np.abs(got - ref) <= e + 2.0 ** -8 * (np.abs(ref) + e))
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - ref)[bad][:4], ref[bad][:4], int(bad.sum()))


THETA = {r: api.rope_frequencies(r, 10000.0)[0] for r in range(16, 129, 16)}


def table_of(rot, interleaved=False, magnitude=None):
    return api.rope_table(rot, 10000.0, interleaved=interleaved, magnitude=magnitude)


# (B, H, Hk, N, layout, positions)
SHAPES = [
    (1, 1, 1, 1, "bhnd", None),
    (3, 5, 2, 1, "bnhd", "rows"),
    (2, 3, 3, 7, "bnhd", None),
    (1, 7, 1, 33, "bhnd", "one"),
    (2, 40, 8, 65, "bnhd", "rows"),
    (5, 4, 2, 300, "bhnd", "rows"),
    (1, 2, 2, 4001, "bnhd", "one"),
]


def positions_of(rng, kind, B, N):
    """(argument, [B or 1, N] numbers): also negative ones and ones close to 2^31."""
    if kind is None:
        return None, np.arange(N)[None]
    p = rng.integers(-1000, 2 ** 31 - 1, (B, N) if kind == "rows" else (N,))
    p.flat[0] = 2 ** 31 - 1
    return i32(p), p.reshape(-1, N)


@pytest.mark.parametrize("rot,interleaved", [(16, True), (32, False), (48, True), (64, False), (64, True), (96, False),
                                             (128, False), (128, True)])
@pytest.mark.parametrize("norms", ["", "q", "k", "qk"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward_match_the_oracle(shape, norms, rot, interleaved):
    B, H, Hk, N, layout, kind = shape
    d = 64 if rot <= 48 else 128 if rot > 64 else (64, 128)[N % 2]
    rng = np.random.default_rng(B * 1000 + N + rot)
    f = 1.0 if rot % 32 else 1.25
    table = table_of(rot, interleaved, f)
    arg, pos = positions_of(rng, kind, B, N)
    a = rope.angles(pos, THETA[rot])[:, None]
    (q, qv), (k, kv) = bf16(rng, (B, H, N, d), layout), bf16(rng, (B, Hk, N, d), layout, 3.0)
    (gq, gqv), (gk, gkv) = bf16(rng, (B, H, N, d), layout), bf16(rng, (B, Hk, N, d), layout)
    dtype = ("fp32", "bf16")[H % 2]
    (wq, wqv), (wk, wkv) = (weight(rng, d, dtype) if x in norms else (None, None) for x in "qk")
    kw = dict(positions=arg, q_weight=wq, k_weight=wk, eps=1e-5, layout=layout)
    out = api.rope(q, k, table, **kw)
    grads = api.rope_bwd(gq, gk, table, q=q if wq is not None else None, k=k if wk is not None else None, **kw)
    for y, x, dx, dw, xv, gv, wv in zip(out, (q, k), grads[:2], grads[2:], (qv, kv), (gqv, gkv), (wqv, wkv)):
        ref, size = rope.forward(xv, a, f, rot, interleaved, wv, 1e-5)
        close(heads(y, layout), ref, 2.0 ** -20 * size)
        ref, wref, size, wsize = rope.backward(gv, a, f, rot, interleaved, xv, wv, 1e-5)
        close(heads(dx, layout), ref, 2.0 ** -19 * size)
        assert (dw is None) == (wv is None)
        if wv is not None:
            assert np.all(np.abs(dw.double().cpu().numpy() - wref) <= 2.0 ** -15 * wsize)


def test_elements_that_pass_stay_bit_for_bit():
    """Without a norm the elements behind the first rot are copied, whatever they hold, and what
    one head holds reaches no other."""
    import torch
    g = np.random.default_rng(3)
    q, _ = bf16(g, (2, 6, 9, 128))
    q[0, 1, 2, 40:] = float("inf")
    q[1, 3, 4, 100] = float("nan")
    k = q[:, :2].clone()
    k[0, 1, 5, 3] = float("nan")
    clean = torch.nan_to_num(q, 0.0, 0.0, 0.0)
    for inter in (False, True):
        for w in (None, torch.ones(128, device="cuda")):
            y, z = api.rope(q, k, table_of(32, inter), q_weight=w, k_weight=w)
            ref = api.rope(clean, clean, table_of(32, inter), q_weight=w, k_weight=w)[0]
            same = torch.ones(2, 6, 9, dtype=torch.bool, device="cuda")
            same[0, 1, 2] = same[1, 3, 4] = False
            assert torch.equal(y[same].view(torch.int16), ref[same].view(torch.int16))
            if w is None:
                assert torch.equal(y[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16))
                assert torch.equal(y[0, 1, 2, :32], ref[0, 1, 2, :32])
            rows = torch.isnan(z).any(-1)
            assert rows[0, 1, 5] and rows.sum() <= 2


def test_outputs_may_be_inputs_and_views():
    """In place, on slices of a packed projection, with positions shared by the batch."""
    import torch
    B, N, H, Hk, d = 3, 50, 6, 2, 64
    packed = torch.randn(B, N, (H + 2 * Hk), d, device="cuda").bfloat16()
    q, k = packed[:, :, :H], packed[:, :, H:H + Hk]
    w = torch.rand(d, device="cuda") + 0.5
    pos = torch.arange(N, device="cuda", dtype=torch.int32) * 7
    table = table_of(48)
    kw = dict(positions=pos, q_weight=w, k_weight=w, layout="bnhd")
    ref = api.rope(q.contiguous(), k.contiguous(), table, **kw)
    assert torch.equal(ref[0], api.rope(q, k, table, positions=pos.expand(B, N), q_weight=w, k_weight=w, layout="bnhd")[0])
    v = packed[:, :, H + Hk:].clone()
    dy = torch.randn(B, N, H, d, device="cuda").bfloat16()
    dk = torch.randn(B, N, Hk, d, device="cuda").bfloat16()
    g = api.rope_bwd(dy, dk, table, q=q, k=k, **kw)
    g2 = api.rope_bwd(dy, dk, table, q=q, k=k, dq=dy, dk=dk, **kw)
    assert g2[0] is dy and all(torch.equal(x, y) for x, y in zip(g, g2))
    out = api.rope(q, k, table, q_out=q, k_out=k, **kw)
    assert out[0] is q and torch.equal(q, ref[0]) and torch.equal(k, ref[1]) and torch.equal(packed[:, :, H + Hk:], v)
    # one tensor alone
    alone = api.rope(ref[0], None, table, positions=pos, layout="bnhd")
    assert alone[1] is None and torch.equal(alone[0], api.rope(ref[0], ref[1], table, positions=pos, layout="bnhd")[0])
    g = api.rope_bwd(dy, None, table, positions=pos, q=q, q_weight=w, layout="bnhd")
    assert g[1] is None and g[3] is None and g[2].shape == (d,)


def test_many_rows_sum_the_same_every_time():
    """Long sums of a weight's gradient: the same bits in every run, and close to 64 bits."""
    import torch
    rng = np.random.default_rng(8)
    B, H, Hk, N, d = 2, 8, 4, 4099, 64
    q, k, gq, gk = (torch.randn(B, x, N, d, device="cuda").bfloat16() for x in (H, Hk, H, Hk))
    w, wv = weight(rng, d)
    run = lambda: api.rope_bwd(gq, gk, table_of(64), q=q, k=k, q_weight=w, k_weight=w)
    first = run()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, run()))
    a = rope.angles(np.arange(N), THETA[64])[None, None]
    for dw, x, g in ((first[2], q, gq), (first[3], k, gk)):
        _, ref, _, size = rope.backward(g.double().cpu().numpy(), a, 1.0, 64, False, x.double().cpu().numpy(), wv)
        assert np.all(np.abs(dw.double().cpu().numpy() - ref) <= 2.0 ** -15 * size)


def test_streams_and_graphs():
    import torch
    B, H, Hk, N, d = 2, 4, 2, 100, 128
    q, k, gq, gk = (torch.randn(B, x, N, d, device="cuda").bfloat16() for x in (H, Hk, H, Hk))
    w, table = torch.rand(d, device="cuda") + 0.5, table_of(128)
    pos = i32(np.arange(N))
    def step():
        return (*api.rope(q, k, table, positions=pos, q_weight=w, k_weight=w),
                *api.rope_bwd(gq, gk, table, positions=pos, q=q, k=k, q_weight=w, k_weight=w))
    ref = [x.clone() for x in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = api.rope(q, k, table, positions=pos, q_weight=w, k_weight=w, stream=s)
    g = api.rope_bwd(gq, gk, table, positions=pos, q=q, k=k, q_weight=w, k_weight=w, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (*y, *g)))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.cuda.graph(other):  # two captured calls have workspaces of their own
        out2 = step()
    pos += 5
    q *= 2
    graph.replay()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.current_stream())
        other.replay()
    s.synchronize()
    torch.cuda.synchronize()
    new = step()
    assert not torch.equal(ref[0], new[0])
    for o in (out, out2):
        assert all(torch.equal(a, b) for a, b in zip(o, new))


def test_two_calls_at_once():
    """Calls on two streams have workspaces of their own."""
    import torch
    B, H, Hk, N, d = 1, 8, 2, 3001, 128
    w, table, streams = torch.rand(d, device="cuda") + 0.5, table_of(128), [torch.cuda.Stream() for _ in range(2)]
    data = [[torch.randn(B, x, N, d, device="cuda").bfloat16() for x in (H, Hk, H, Hk)] for _ in streams]
    call = lambda q, k, gq, gk: api.rope_bwd(gq, gk, table, q=q, k=k, q_weight=w, k_weight=w)
    ref = [call(*x) for x in data]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = call(*data[i])
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_past_32_bits():
    """Heads 2^32 elements apart, and an output whose tokens are far apart."""
    import torch
    far = (1 << 32) + 64
    room = torch.zeros(far + 40 * 64, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, 2, 33, 64, device="cuda").bfloat16()
    view = room.as_strided((1, 2, 33, 64), (8, far, 64, 1))
    view.copy_(x)
    w, table = torch.rand(64, device="cuda") + 0.5, table_of(32)
    ref = api.rope(x, x, table, q_weight=w)
    got = api.rope(view, x, table, q_weight=w, k_out=room.as_strided((1, 2, 33, 64), (8, 64 * 40, 64, 1), (1 << 31) + 8))
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    g = torch.randn_like(x)
    ref = api.rope_bwd(g, None, table, q=x, q_weight=w)
    got = api.rope_bwd(g, None, table, q=view, q_weight=w, dq=view)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])


# ---------------------------------------------------------------------------
# The cache's write
# ---------------------------------------------------------------------------
def run_append(pool, H, T, lens, new, rot, interleaved, norms="qk", layout="bnhd", amp=1.0):
    """One call against the oracle; returns the device's tensors."""
    import torch
    B, Hk, d, page = pool.B, pool.Hk, pool.d, pool.page
    f = 1.125
    table = table_of(rot, interleaved, f)
    (q, qv), (k, kv), (v, vv) = (bf16(pool.rng, (B, x, T, d), layout, amp) for x in (H, Hk, Hk))
    (wq, wqv), (wk, wkv) = (weight(pool.rng, d) if x in norms else (None, None) for x in "qk")
    dev = pool.dev()
    before = [x.clone() for x in dev]
    q_out = torch.full_like(q, 7.0)
    ql = [T] * B if new is None else new
    seq, nl = i32(lens), None if new is None else i32(new)
    got = api.cache_append_rope(q, k, v, table, *dev, seq, new_lens=nl, q_weight=wq, k_weight=wk, eps=1e-5, layout=layout,
                                q_out=q_out)
    check_clean()
    assert got is q_out
    first = np.asarray(lens) - np.asarray(ql)
    pos = first[:, None] + np.arange(T)
    # queries: bit for bit what rope gives at these positions, other rows as they were
    ref = api.rope(q, k, table, positions=i32(pos), q_weight=wq, k_weight=wk, eps=1e-5, layout=layout)
    there = torch.from_numpy((np.arange(T) < np.asarray(ql)[:, None]) & (pos >= 0)).cuda()
    at = there[:, None, :, None] if layout == "bhnd" else there[:, :, None, None]
    assert torch.equal(q_out, torch.where(at, ref[0], torch.full_like(q, 7.0)))
    # values: bit for bit what cache_append writes
    plain = [x.clone() for x in before]
    api.cache_append(k, v, *plain, seq, new_lens=nl, layout=layout)
    for i in (1, 3, 4):
        assert torch.equal(dev[i], plain[i])
    # keys: the oracle's rotated ones, rounded once
    a = rope.angles(pos, THETA[rot])[:, None]
    y, size = rope.forward(kv, a, f, rot, interleaved, wkv, 1e-5)
    e = 2.0 ** -20 * size
    codes, scale = pool.k.copy(), pool.ks.copy()
    streaming.cache_append(y, y, codes, codes.copy(), scale, scale.copy(), pool.table, lens, ql)
    gc, gs = dev[0].cpu().numpy(), dev[2].double().cpu().numpy()
    touched = np.zeros(gc.shape[:3], dtype=bool)
    for b in range(B):
        for t in range(ql[b]):
            if pos[b, t] < 0:
                continue
            pid, slot = pool.table[b][pos[b, t] // page], pos[b, t] % page
            touched[pid, :, slot] = True
            for h in range(Hk):
                s = gs[pid, h]
                val = _E4M3[gc[pid, h, slot] & 0x7F] * np.where(gc[pid, h, slot] & 0x80, -1.0, 1.0) * s
                r = y[b, h, t]
                fin = np.isfinite(r)
                off = np.abs(val - np.clip(r, -448 * s, 448 * s))[fin]
                bound = np.maximum(2.0 ** -4 * (np.abs(r) + e[b, h, t]), s * 2.0 ** -10) + e[b, h, t]
                assert np.all(off <= bound[fin]), (b, h, t, off.max())
    # scales: the oracle's, but where an error of a key moves the largest over a border
    near = np.zeros(scale.shape, dtype=bool)
    for b in range(B):
        for t in range(ql[b]):
            if pos[b, t] >= 0:
                m = np.abs(y[b, :, t])
                x = np.log2(np.maximum(m, 1e-300) / 448.0)
                near[pool.table[b][pos[b, t] // page]] |= (np.abs(x - np.rint(x)) < 2.0 ** -17).any(-1)
    assert np.array_equal(gs[~near], scale[~near])
    # slots that no new token takes: as they were, or rounded again where the page's scale grew
    same = ~touched & ~near[:, :, None]
    assert np.array_equal(gc[same], codes[same])
    return dev


APPENDS = [
    (1, 1, 1, 1, 16, [1], None),
    (1, 1, 1, 1, 16, [17], None),
    (3, 8, 2, 1, 64, [200, 0, 65], [1, 0, 1]),
    (4, 6, 2, 3, 16, [5, 3, 300, 64], [3, 3, 2, 0]),
    (2, 8, 4, 7, 64, [130, 2], [7, 7]),          # more tokens than positions: some are not written
    (2, 40, 2, 100, 32, [100, 457], [100, 71]),
    (1, 5, 1, 131, 128, [333], None),            # tokens of a page beyond those held in registers
    (2, 3, 3, 600, 1024, [700, 2000], [600, 599]),
    (1, 4, 2, 300, 256, [300], None),
    (2, 5, 3, 20, 32, [50, 20], [20, 17]),       # query heads need not be shared evenly
    (1, 9, 5, 700, 64, [1000], [700]),           # several heads of K a block, not a multiple of them
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot,interleaved,norms,layout", [(64, False, "qk", "bnhd"), (64, True, "", "bhnd"),
                                                          (32, False, "k", "bhnd"), (16, True, "q", "bnhd"),
                                                          (128, False, "", "bnhd"), (112, True, "qk", "bhnd")])
@pytest.mark.parametrize("shape", APPENDS)
def test_append_matches_the_oracle(shape, rot, interleaved, norms, layout, d):
    B, H, Hk, T, page, lens, new = shape
    rot = min(rot, d)
    pool = Pool(50 + T + rot, B, Hk, d, page, max(1, -(-max(lens) // page)), token_major=layout == "bnhd")
    run_append(pool, H, T, lens, new, rot, interleaved, norms, layout)


def test_append_where_scales_grow_and_vanish():
    """Large keys make older codes round again; tiny ones keep the page's scale."""
    for amp in (1e4, 1e-4, 1e-38):
        pool = Pool(7, 2, 2, 128, 16, 4)
        run_append(pool, 4, 5, [21, 40], [5, 4], 128, False, "", amp=amp)


def test_append_through_a_wider_table():
    """A table that is a part of a wider one, and new tokens that are slices of a packed projection."""
    import torch
    pool = Pool(17, 3, 2, 64, 32, 4)
    dev, ref = pool.dev(), pool.dev()
    outer = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    outer[:, 2:6] = dev[4]
    dev[4] = outer[:, 2:6]
    packed = torch.randn(3, 5, 4 + 2 + 2, 64, device="cuda").bfloat16()
    q, k, v = packed[:, :, :4], packed[:, :, 4:6], packed[:, :, 6:]
    w, lens = torch.rand(64, device="cuda") + 0.5, i32([40, 128, 5])
    want = api.cache_append_rope(q.contiguous(), k.contiguous(), v.contiguous(), table_of(48, True), *ref, lens, q_weight=w,
                                 k_weight=w, layout="bnhd")
    got = api.cache_append_rope(q, k, v, table_of(48, True), *dev, lens, q_weight=w, k_weight=w, layout="bnhd", q_out=q)
    check_clean()
    assert torch.equal(got, want) and got.data_ptr() == q.data_ptr()
    assert all(torch.equal(x, y) for x, y in zip(dev[:4], ref[:4]))


def test_append_of_values_that_are_not_finite():
    import torch
    pool = Pool(9, 1, 1, 64, 16, 4)
    dev = pool.dev()
    k = torch.randn(1, 1, 3, 64, device="cuda").bfloat16()
    k[0, 0, 1, 40] = float("inf")
    k[0, 0, 2, 50] = float("nan")
    q = torch.randn(1, 2, 3, 64, device="cuda").bfloat16()
    api.cache_append_rope(q, k, k, table_of(32), *dev, i32([10]))
    check_clean()
    pid = int(pool.table[0][0])
    c = dev[0][pid, 0, 7:10].cpu().numpy()
    assert c[1, 40] == 0x7E and (c[2, 50] & 0x7F) == 0x7F
    assert ((c & 0x7F) == 0x7F).sum() == 1  # elements that pass reach no other
    assert float(dev[2][pid, 0]) < 1.0      # of finite magnitudes


def test_append_reports_bad_pages_and_lengths():
    import torch
    pool = Pool(11, 2, 1, 64, 16, 2)
    k = torch.randn(2, 1, 1, 64, device="cuda").bfloat16()
    for lens, entry in (([40, 5], None), ([-3, 5], None), ([20, 5], 10 ** 6)):
        dev = pool.dev()
        if entry is not None:
            dev[4][0, 1] = entry
        before = [x.clone() for x in dev]
        api.cache_append_rope(k.clone(), k, k, table_of(64), *dev, i32(lens))
        assert api.check_device_error()[0] == -5
        mine = set(int(x) for x in pool.table[0])
        for pid in mine:
            assert torch.equal(dev[0][pid], before[0][pid]) and torch.equal(dev[1][pid], before[1][pid])
        other = int(pool.table[1][0])
        assert not torch.equal(dev[0][other], before[0][other])


def test_a_captured_append_follows_its_lengths():
    """The lengths stay on the device: a replayed call writes and rotates at the new positions."""
    import torch
    pool = Pool(13, 2, 2, 128, 16, 8)
    q, k, v = (torch.randn(2, h, 1, 128, device="cuda").bfloat16() for h in (8, 2, 2))
    table, seq = table_of(128), i32([10, 33])
    dev, ref = pool.dev(), pool.dev()
    api.cache_append_rope(q, k, v, table, *pool.dev(), seq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.cache_append_rope(q, k, v, table, *dev, seq)
    for _ in range(20):
        graph.replay()
        want = api.cache_append_rope(q, k, v, table, *ref, seq)
        assert torch.equal(out, want) and all(torch.equal(x, y) for x, y in zip(dev, ref))
        seq += 1
    check_clean()


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------
def test_arguments_that_are_refused():
    import torch
    q, k = torch.randn(2, 4, 8, 64, device="cuda").bfloat16(), torch.randn(2, 2, 8, 64, device="cuda").bfloat16()
    t, w = table_of(64), torch.ones(64, device="cuda")
    pos = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]), dict(q=q.transpose(2, 3)), dict(k=k[:1]), dict(k=k[:, :, :5]),
           dict(k=torch.randn(2, 2, 8, 128, device="cuda").bfloat16()), dict(table=table_of(128)), dict(table=None),
           dict(table=api.rope_table(64, device="cpu")), dict(positions=pos.long()), dict(positions=pos.cpu()),
           dict(positions=pos[:, :7]), dict(positions=pos[:1]), dict(positions=pos.t().contiguous().t()),
           dict(q_weight=w[:32]), dict(q_weight=w.half()), dict(q_weight=w.cpu()), dict(q_weight=w, k_weight=w.bfloat16()),
           dict(k_weight=torch.ones(128, device="cuda")[::2]), dict(layout="nbhd"), dict(q_out=k), dict(k_out=k.float()),
           dict(q_out=q.cpu())]
    for b in bad:
        a = dict(q=q, k=k, table=t)
        a.update(b)
        with pytest.raises(ValueError):
            api.rope(**a)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(api.AttnError, match="ATTN_ERR_INVALID"):
            api.rope(q, k, t, q_weight=w, eps=eps)
    api.rope(q, k, t, eps=0.0)  # no norm, no epsilon
    with pytest.raises(api.AttnError, match="ATTN_ERR_INVALID"):  # one place for several rows
        api.rope(q, k, t, q_out=q[:, :1].expand(2, 4, 8, 64))
    for b in (dict(q=None), dict(q=q[:, :2]), dict(dq_weight=w.bfloat16()), dict(dk_weight=w[:32]), dict(dq=k),
              dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        a = dict(dq_out=q, dk_out=k, table=t, q=q, k=k, q_weight=w, k_weight=w)
        a.update(b)
        with pytest.raises(ValueError):
            api.rope_bwd(**a)
    pool = Pool(1, 2, 2, 64, 16, 2)
    dev = pool.dev()
    api.cache_append_rope(q, k, k, t, *dev, i32([8, 9]))
    for i, b in ((2, k[:, :1]), (2, k.float()), (3, None), (4, dev[0][:, :1]), (6, dev[2][:1]), (8, dev[4].long()), (9, i32([8]))):
        a = [q, k, k, t, *dev, i32([8, 9])]
        a[i] = b
        with pytest.raises(ValueError):
            api.cache_append_rope(*a)
