"""Paged 8-bit cache: attn_cache_append and attn_fwd_cache against the fp64 oracle.

Codes and scales have to be the oracle's bit for bit (a scale is a power of two, so a
code carries one rounding).  Outputs of attn_fwd_cache: with M = sum_j P_ij |V_j|,
  e = (2^-11 + 2^-15) M   weights rounded to f16 (half a step, 2^-11 relative), and 2^-15
                          for scores and exponentials in fp32 (scores below 32 in log2
                          units: 128 fp32 additions and one rounding of the exponent stay
                          under 2^-16, the exponential under 2^-21),
  |O - ref| <= e + 2^-8 (|ref| + e)   (bf16 store), and |LSE - ref| <= 2^-14."""

import numpy as np
import pytest

import oracle
from exact_attention_52_gb300 import api
from oracle import streaming

from .helpers import device_bf16_to_f64

pytestmark = pytest.mark.gpu


class Pool:
    """A cache of B sequences, its pages dealt out at random, filled with data of its own."""

    def __init__(self, seed, B, Hk, d, page, max_pages, token_major=False, spare=3):
        import torch
        self.rng = np.random.default_rng(seed)
        self.B, self.Hk, self.d, self.page = B, Hk, d, page
        P = B * max_pages + spare
        self.table = self.rng.permutation(P)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        self.k, self.v = (self.rng.integers(0, 0x7F, (P, Hk, page, d)).astype(np.uint8) |
                          (self.rng.integers(0, 2, (P, Hk, page, d)).astype(np.uint8) << 7) for _ in range(2))
        for x in (self.k, self.v):  # magnitudes around 1
            x[...] = streaming.e4m3_encode(self.rng.standard_normal(x.shape) * 64)
        self.ks, self.vs = (2.0 ** self.rng.integers(-7, -4, (P, Hk)).astype(np.float64) for _ in range(2))
        self.token_major = token_major
        self.torch = torch

    def dev(self):
        """k_pages, v_pages, k_scale, v_scale, table on the device."""
        torch = self.torch
        if self.token_major:  # [P, page, Hk, d] storage seen as [P, Hk, page, d]
            pages = [torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3))).cuda().transpose(1, 2)
                     for x in (self.k, self.v)]
        else:
            pages = [torch.from_numpy(x.copy()).cuda() for x in (self.k, self.v)]
        scales = [torch.from_numpy(x.astype(np.float32)).cuda() for x in (self.ks, self.vs)]
        return [*pages, *scales, torch.from_numpy(self.table).cuda()]


def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(rng, shape, layout="bhnd", amp=1.0):
    """bf16 data [b, h, t, d] on the device in `layout`, and its values."""
    import torch
    x = torch.from_numpy((amp * rng.standard_normal(shape)).astype(np.float32)).bfloat16()
    vals = x.double().numpy()
    x = x.cuda()
    return (x if layout == "bhnd" else x.transpose(1, 2).contiguous()), vals


def check_clean():
    rc, site = api.check_device_error()
    assert rc == 0, f"device error {rc} at site {site:#x}"


def check_out(o, lse, ref, layout="bhnd"):
    o_ref, lse_ref, mag, there = ref
    og = device_bf16_to_f64(o if layout == "bhnd" else o.transpose(1, 2))
    lg = lse.double().cpu().numpy()
    at = np.broadcast_to(there[:, None, :], lg.shape)
    assert np.array_equal(np.isnan(og[at]), np.isnan(o_ref[at]))
    e = (2.0 ** -11 + 2.0 ** -15) * mag
    bad = np.abs(og - o_ref) > e + 2.0 ** -8 * (np.abs(o_ref) + e)
    assert not bad[at].any(), (np.argwhere(bad & at[..., None])[:4], np.nanmax(np.abs(og - o_ref)[at]))
    assert np.array_equal(np.isposinf(lg[at]), np.isposinf(lse_ref[at]))
    fin = at & np.isfinite(lse_ref)
    assert np.all(np.abs(lg[fin] - lse_ref[fin]) <= 2.0 ** -14)


def run_cache(pool, H, T, seq_lens, q_lens, left=-1, sinks=0, layout="bhnd", scale=None, amp=1.0):
    import torch
    q, qv = bf16(pool.rng, (pool.B, H, T, pool.d), layout, amp)
    o = torch.full_like(q, 7.0)
    lse = torch.full((pool.B, H, T), 7.0, device="cuda")
    api.fwd_cache(q, *pool.dev(), i32(seq_lens), q_lens=None if q_lens is None else i32(q_lens), layout=layout,
                  scale=scale, window_left=left, sinks=sinks, o=o, lse=lse)
    check_clean()
    ql = [T] * pool.B if q_lens is None else q_lens
    ref = streaming.cache_forward(qv, pool.k, pool.v, pool.ks, pool.vs, pool.table, seq_lens, ql,
                                  pool.d ** -0.5 if scale is None else scale, left, sinks)
    check_out(o, lse, ref, layout)
    # rows behind a sequence's queries are left as they were
    gone = ~ref[3]
    ob = o if layout == "bhnd" else o.transpose(1, 2)
    for b, t in np.argwhere(gone):
        assert torch.all(ob[b, :, t] == 7.0) and torch.all(lse[b, :, t] == 7.0)


# (B, H, Hk, T, page, seq_lens, q_lens)
SHAPES = [
    (1, 1, 1, 1, 16, [1], None),
    (1, 1, 1, 1, 16, [17], None),
    (2, 4, 4, 1, 32, [1, 63], None),
    (3, 8, 2, 1, 64, [200, 0, 65], None),
    (2, 8, 1, 1, 16, [300, 129], None),
    (2, 40, 2, 1, 128, [1000, 777], None),    # 20 query heads a group: two row tiles
    (4, 6, 2, 3, 16, [5, 3, 300, 64], [3, 3, 2, 0]),
    (2, 8, 4, 7, 64, [130, 2], [7, 7]),       # more queries than tokens: some see nothing
    (1, 4, 1, 40, 32, [555], None),
    (1, 2, 1, 1, 64, [20000], None),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left,sinks", [(-1, 0), (20, 0), (33, 4), (0, 1), (100, 40), (100000, 3)])
@pytest.mark.parametrize("shape", SHAPES)
def test_cache_forward_matches_oracle(shape, left, sinks, d):
    B, H, Hk, T, page, lens, ql = shape
    pool = Pool(1000 + T + H, B, Hk, d, page, max(1, -(-max(lens) // page)))
    run_cache(pool, H, T, lens, ql, left, sinks)


# Queries enough for the kernel of prompts (more than 64 rows a key/value head): tiles
# that end inside the 128 rows, one and two tiles a pair, several pairs, more queries than
# tokens, sequences without any, every page size, key tiles that end inside a page.
PROMPTS = [
    (1, 1, 1, 65, 16, [65], None),
    (1, 1, 1, 65, 64, [3], None),              # most rows see nothing
    (1, 2, 1, 128, 128, [128], None),
    (2, 6, 2, 100, 32, [1000, 357], [100, 71]),
    (3, 5, 1, 131, 16, [131, 0, 700], [131, 0, 1]),
    (1, 16, 1, 300, 1024, [2100], None),
    (2, 3, 3, 700, 64, [700, 1333], None),
    (1, 40, 2, 9, 256, [5000], None),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left,sinks", [(-1, 0), (20, 0), (140, 4), (0, 1), (300, 200), (100000, 3)])
@pytest.mark.parametrize("shape", PROMPTS)
def test_cache_forward_of_prompts_matches_oracle(shape, left, sinks, d):
    B, H, Hk, T, page, lens, ql = shape
    pool = Pool(2000 + T + H, B, Hk, d, page, max(1, -(-max(lens) // page)))
    run_cache(pool, H, T, lens, ql, left, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout,token_major", [("bnhd", True), ("bhnd", False)])
def test_cache_forward_of_prompts_layouts(layout, token_major, d):
    pool = Pool(17, 2, 2, d, 32, 20, token_major=token_major)
    run_cache(pool, 8, 90, [611, 305], [90, 43], 333, 2, layout=layout)


def test_cache_forward_of_prompts_large_scores_and_values():
    """Scores that rise far beyond the first tile's maximum (tiles redone, outputs rescaled),
    page scales far apart."""
    pool = Pool(19, 1, 2, 128, 16, 80)
    pool.vs *= 2.0 ** pool.rng.integers(-40, 41, pool.vs.shape)
    pool.ks[:] = 2.0 ** -5 * (1 + np.arange(len(pool.ks))[:, None] % 2)
    run_cache(pool, 8, 70, [1250], None, amp=2.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [2, 70, 300])
@pytest.mark.parametrize("step", [1.0, 4.0, 8.0, 14.0])
def test_scores_that_grow_along_the_keys(step, T, d):
    """The running maximum is passed inside a tile, at each of its parts, by little and by
    far, by some rows of a warp and not by others.  A query has one element that is not
    zero, so a score is one product: below 2^9 it and its maximum's difference carry two
    roundings of 2^-16, inside the bound's share for scores."""
    import torch
    H, N, page = 2, 700, 64
    pool = Pool(61 + T, 1, 1, d, page, 11)
    at = np.minimum(step * (np.arange(704) // 16), 224.0) + np.arange(704) % 16 / 16.0
    for j in range(11):
        pool.k[pool.table[0, j], 0, :, 0] = streaming.e4m3_encode(at[page * j:page * j + page])
    pool.ks[:] = 1.0
    q = np.zeros((1, H, T, d), np.float32)
    q[..., 0] = np.array([1.0, -1.0, 0.5, 0.0, 0.25, 1.0, -0.125])[np.arange(H * T).reshape(1, H, T) % 7]
    q = torch.from_numpy(q).bfloat16()
    o, lse = api.fwd_cache(q.cuda(), *pool.dev(), i32([N]), scale=1.0)
    check_clean()
    check_out(o, lse, streaming.cache_forward(q.double().numpy(), pool.k, pool.v, pool.ks, pool.vs, pool.table,
                                              [N], [T], 1.0, -1, 0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout,token_major", [("bnhd", False), ("bhnd", True), ("bnhd", True)])
def test_cache_forward_layouts(layout, token_major, d):
    pool = Pool(7, 2, 2, d, 32, 5, token_major=token_major)
    run_cache(pool, 8, 3, [150, 31], [3, 1], 50, 2, layout=layout)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [2, 70])
def test_cache_forward_of_zero_and_tiny_rows(T, d):
    """Query rows of zeros, of subnormals and of one large among tiny numbers; a page whose
    codes are zeros and whose scale is the least an append writes; hidden scores in all."""
    import torch
    pool = Pool(18, 1, 1, d, 16, 12)
    pool.k[pool.table[0, 3]] = 0
    pool.ks[pool.table[0, 3]] = 2.0 ** -100
    q, _ = bf16(pool.rng, (1, 8, T, d))
    q[:, 0] = 0
    q[:, 1] *= 2.0 ** -128
    q[:, 2] *= 2.0 ** -20
    q[:, 2, :, 5] = 3.0
    q[:, 3, 1:] = 0
    qv = q.double().cpu().numpy()
    for left, sinks in ((-1, 0), (60, 3)):
        o, lse = api.fwd_cache(q, *pool.dev(), i32([185]), window_left=left, sinks=sinks)
        check_clean()
        check_out(o, lse, streaming.cache_forward(qv, pool.k, pool.v, pool.ks, pool.vs, pool.table, [185], [T],
                                                  d ** -0.5, left, sinks))


def test_cache_forward_many_sequences_share_the_device():
    """More items than CTAs, lengths from 0 to long: shares begin and end inside items."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 400, 150)]
    lens[7], lens[100] = 3000, 2500
    pool = Pool(8, 150, 4, 64, 16, 190)
    run_cache(pool, 8, 1, lens, [0 if n == 0 else 1 for n in lens])


@pytest.mark.parametrize("B", [31, 32, 33, 64, 65])
@pytest.mark.parametrize("T,longest", [(1, 60), (1, 900), (3, 300)])
def test_cache_forward_ragged_batches(T, longest, B):
    """Shares of ragged batches, whole items and parts, with empty sequences among them."""
    rng = np.random.default_rng(B + longest)
    lens = [int(x) for x in rng.integers(0, longest, B)]
    lens[B // 2], lens[0], lens[-1] = longest, 0, 1
    pool = Pool(9 + B, B, 2, 64, 16, -(-longest // 16))
    run_cache(pool, 6, T, lens, [min(n, T) for n in lens])


def test_cache_forward_large_scores_and_values():
    """Scores that reach far beyond the first block's maximum, page scales far apart."""
    pool = Pool(9, 2, 2, 128, 16, 20)
    pool.vs *= 2.0 ** pool.rng.integers(-40, 41, pool.vs.shape)
    pool.ks[:] = 2.0 ** -5
    run_cache(pool, 8, 1, [310, 200], None, amp=2.0)


def run_far(pool, H, T, n, left=-1, sinks=0, amp=1.0):
    """run_cache for value scales from 2^-126 to 2^126.  Against a score below 32 a sum of score
    and log2 sv, a maximum and log2 of a sum may all reach 2^8: two roundings of 2^-18 and
    three of 2^-17 in exponents, 2^-15 log2 units together, beside what the module's bound
    has: |O - ref| <= e + 2^-8 (|ref| + e) + 2^-134 with e = (2^-11 + 2^-14) M, the last being half
    a step of bf16 numbers below 2^-126 (their last bit is 2^-126 2^-7); LSE as there."""
    import torch
    q, qv = bf16(pool.rng, (pool.B, H, T, pool.d), amp=amp)
    lens = [n] * pool.B
    o, lse = api.fwd_cache(q, *pool.dev(), i32(lens), window_left=left, sinks=sinks)
    check_clean()
    o_ref, lse_ref, mag, _ = streaming.cache_forward(qv, pool.k, pool.v, pool.ks, pool.vs, pool.table, lens,
                                                     [T] * pool.B, pool.d ** -0.5, left, sinks)
    og, lg = device_bf16_to_f64(o), lse.double().cpu().numpy()
    e = (2.0 ** -11 + 2.0 ** -14) * mag
    bad = ~(np.abs(og - o_ref) <= e + 2.0 ** -8 * (np.abs(o_ref) + e) + 2.0 ** -134)
    assert not bad.any(), (np.argwhere(bad)[:4], og[bad][:4], o_ref[bad][:4])
    assert np.all(np.abs(lg - lse_ref) <= 2.0 ** -14)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 5, 70, 300])
@pytest.mark.parametrize("exponent", [-126, -122, -110, -100, 100])
def test_value_scales_that_are_all_small_or_large(exponent, T, d):
    """Every visible page of one extreme value scale, from one token to thousands of equal scores."""
    for n, amp in ((max(1, T), 1.0), (T + 8200, 0.0), (T + 500, 2.0)):
        pool = Pool(80, 1, 2, d, 64, -(-n // 64))
        pool.vs[:] = 2.0 ** exponent
        run_far(pool, 4, T, n, amp=amp)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 5, 70, 300])
@pytest.mark.parametrize("amp", [0.0, 2.0])
@pytest.mark.parametrize("low,high", [(-100, 40), (-100, -8), (-60, 30), (-126, 100)])
def test_value_scales_far_apart(low, high, amp, T, d):
    """Pages of two value scales far apart, at equal scores and at others: one page of the one
    among the others, first, last or amid; every other page; the whole at random."""
    n = 1100 + T
    for which in ("first", "last", "amid", "turns", "random"):
        for lo, hi in ((low, high), (high, low)):
            pool = Pool(81, 1, 2, d, 16, -(-n // 16))
            exps, pages = np.full(pool.table.shape[1], hi), pool.table[0]
            if which == "turns":
                exps[::2] = lo
            elif which == "random":
                exps = pool.rng.integers(low, high + 1, len(exps))
            else:
                exps[{"first": 0, "last": n // 16 - 1, "amid": len(exps) // 2}[which]] = lo
            pool.vs[pages] = 2.0 ** exps.astype(np.float64)[:, None]
            run_far(pool, 4, T, n, amp=amp)
            run_far(pool, 4, T, n, 500, 20, amp=amp)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T,n", [(40, 1, 900), (24, 5, 900), (6, 300, 1400), (20, 70, 1400)])
@pytest.mark.parametrize("exponent", [-100, 45, 110])
def test_a_far_value_scale_within_a_walk(exponent, B, T, n, d):
    """Enough sequences that a walk has several key tiles: ordinary pages, then one far from
    them somewhere in each sequence and head, then ordinary ones again."""
    pool = Pool(83, B, 8, d, 16, -(-n // 16))
    pool.vs[...] = 2.0 ** pool.rng.integers(-9, -5, pool.vs.shape)
    for b in range(B):
        for h in range(8):
            pool.vs[pool.table[b, pool.rng.integers(0, pool.table.shape[1])], h] = 2.0 ** exponent
    run_far(pool, 8, T, n, amp=1.5)
    run_far(pool, 8, T, n, 700, 30, amp=1.5)


@pytest.mark.parametrize("T", [1, 70])
def test_a_page_of_zeros_among_others(T):
    """What an append makes of values that are all zeros (a scale of 2^-100) beside pages of
    ordinary and of large values."""
    import torch
    pool = Pool(82, 1, 2, 64, 16, 20)
    dev = pool.dev()
    k, kv = bf16(pool.rng, (1, 2, 300, 64))
    v, vv = bf16(pool.rng, (1, 2, 300, 64), amp=2.0 ** 20)
    v[:, :, 32:80], vv[:, :, 32:80] = 0, 0
    v[:, :, 100:], vv[:, :, 100:] = v[:, :, 100:] * 2.0 ** -20, vv[:, :, 100:] * 2.0 ** -20
    api.cache_append(k, v, *dev, i32([300]))
    streaming.cache_append(kv, vv, pool.k, pool.v, pool.ks, pool.vs, pool.table, [300], [300])
    assert float(dev[3].min()) == 2.0 ** -100 and np.array_equal(dev[1].cpu().numpy(), pool.v)
    for amp in (0.0, 1.0):
        run_far(pool, 4, T, 300, amp=amp)


def test_pages_that_no_query_sees_are_not_read():
    """Table entries outside window and sinks hold nonsense and no error is recorded."""
    pool = Pool(10, 2, 2, 128, 16, 40)
    lens, left, sinks = [600, 333], 70, 5
    for b, n in enumerate(lens):
        for pg in range(40):
            lo, hi = pg * 16, pg * 16 + 15
            if lo >= n or (hi < n - 1 - left and lo >= sinks):
                pool.table[b, pg] = -1 if pg % 2 else 1 << 30
    run_cache(pool, 4, 1, lens, None, left, sinks)


def test_pages_that_no_query_of_a_prompt_sees_are_not_read():
    pool = Pool(15, 2, 2, 64, 16, 40)
    lens, ql, left, sinks = [600, 333], [90, 70], 70, 5
    for b, n in enumerate(lens):
        for pg in range(40):
            lo, hi = pg * 16, pg * 16 + 15
            if lo >= n or (hi < n - ql[b] - left and lo >= sinks):
                pool.table[b, pg] = -1 if pg % 2 else 1 << 30
                continue
            for x in (pool.k, pool.v):  # slots behind the sequence or between sinks and window: NaN
                for j in range(lo, hi + 1):
                    if j >= n or (j < n - ql[b] - left and j >= sinks):
                        x[pool.table[b, pg], :, j % 16] = 0x7F
    run_cache(pool, 4, 90, lens, ql, left, sinks)


@pytest.mark.parametrize("T", [1, 70])
def test_windows_and_sinks_as_large_as_they_get(T):
    pool = Pool(16, 1, 1, 64, 16, 12)
    for left, sinks in ((2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0), (3, 2 ** 31 - 1), (191, 1), (0, 192)):
        run_cache(pool, 2, T, [150], None, left, sinks)
        run_cache(pool, 2, T, [1], None, left, sinks)


@pytest.mark.parametrize("T,seq", [(1, 300), (3, 77), (70, 300)])
def test_cache_in_the_debug_build(T, seq):
    """The range-checked library gives the oracle's answer with the error word clear."""
    saved = api._lib
    api._lib = api.load_library(api.DEBUG_LIB_PATH)
    try:
        for d in (64, 128):
            run_cache(Pool(14, 2, 2, d, 32, 10), 8, T, [seq, 5], None, 60, 3)
    finally:
        api._lib = saved


@pytest.mark.parametrize("T,n", [(1, 300), (3, 77), (70, 300), (300, 700)])
def test_far_value_scales_and_nan_in_the_debug_build(T, n):
    """The copies of the code for value scales far apart, and the look for NaN values, stay
    within their tensor-memory columns."""
    saved = api._lib
    api._lib = api.load_library(api.DEBUG_LIB_PATH)
    try:
        for d in (64, 128):
            pool = Pool(84, 2, 2, d, 32, -(-n // 32))
            pool.vs[pool.table[:, 0]] = 2.0 ** -100
            pool.vs[pool.table[1, -1]] = 2.0 ** 60
            run_far(pool, 8, T, n)
            pool = Pool(85, 2, 2, d, 32, -(-n // 32))
            pool.v[pool.table[0, (n - 2) // 32], 1, (n - 2) % 32, 5] = 0x7F
            run_cache(pool, 8, T, [n, n], None, 60, 3)
    finally:
        api._lib = saved


@pytest.mark.parametrize("T", [1, 70])
def test_first_call_of_a_process_may_be_captured(T):
    """A fresh process whose first call of the library is made under stream capture."""
    import subprocess
    import sys
    code = f"""
import torch
from exact_attention_52_gb300 import api
q = torch.randn(1, 4, {T}, 64, device="cuda").bfloat16()
kp, vp = (torch.randint(0, 100, (8, 2, 32, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
ks, vs = (torch.ones(8, 2, device="cuda") for _ in range(2))
table, lens = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8), torch.tensor([200], dtype=torch.int32, device="cuda")
k = torch.randn(1, 2, {T}, 64, device="cuda").bfloat16()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    api.cache_append(k, k, kp, vp, ks, vs, table, lens)
    o, lse = api.fwd_cache(q, kp, vp, ks, vs, table, lens)
g.replay()
torch.cuda.synchronize()
o2, lse2 = api.fwd_cache(q, kp, vp, ks, vs, table, lens)
assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
assert api.check_device_error() == (0, 0)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("T", [1, 4])
def test_nan_codes_in_hidden_places_do_not_matter(T):
    """NaN codes behind the sequence, between sinks and window, and (T > 1) in tokens that
    only later queries see: rows that do not see them are finite, the others NaN as the
    oracle's."""
    pool = Pool(11, 1, 1, 128, 16, 10)
    n, left, sinks = 130, 40, 3
    first = n - T
    hidden = [j for j in range(160) if j >= n or (j < first - left and j >= sinks)]
    for j in hidden + ([n - 1] if T > 1 else []):
        for x in (pool.k, pool.v):
            x[pool.table[0, j // 16], 0, j % 16, ::3] = 0x7F if j % 2 else 0xFF
    if T > 1:  # the last token's key is a number: only its value is NaN
        pool.k[pool.table[0, (n - 1) // 16], 0, (n - 1) % 16] = 0x30
    run_cache(pool, 8, T, [n], None, left, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,n,left,sinks", [(70, 130, -1, 0), (300, 1000, 40, 3), (300, 300, -1, 0), (600, 5000, 700, 20)])
def test_nan_values_of_a_prompt_reach_the_rows_that_see_them(T, n, left, sinks, d):
    """NaN codes in a few values of tokens that some queries of a tile see and others do
    not: NaN in just those rows and columns, as the oracle's, and numbers everywhere else;
    keys behind the sequence and between sinks and window all NaN."""
    pool = Pool(13 + T, 1, 2, d, 32, -(-n // 32) + 1)
    first = n - T
    at = lambda j: (pool.table[0, j // 32], slice(None), j % 32)
    for j in range(pool.table.shape[1] * 32):
        if j >= n or (left >= 0 and sinks <= j < first - left):
            pool.k[at(j)] = pool.v[at(j)] = 0xFF
    for j, col in ((first + T // 2, 5), (first + T // 2, d - 1), (n - 1, 33), (first + 40, 0), (0, 17)):
        pool.v[pool.table[0, j // 32], j % 2, j % 32, col] = 0x7F if col % 2 else 0xFF
    run_cache(pool, 4, T, [n], None, left, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [70, 128])
def test_nan_values_of_a_lone_query_tile(T, d):
    """One NaN value per sequence and head, in every key tile in turn, where two groups of
    warps share a query tile's keys: the one that ends later may be the one that met it."""
    B, Hk, n, page = 10, 4, 1100, 64
    pool = Pool(17, B, Hk, d, page, 18)
    for b in range(B):
        for h in range(Hk):
            j = min(n - 1, 128 * ((b * Hk + h) % 9) + 97)
            pool.v[pool.table[b, j // page], h, j % page, (7 * b + h) % d] = 0x7F
    run_cache(pool, Hk, T, [n] * B, None)


@pytest.mark.parametrize("d", [64, 128])
def test_nan_values_far_apart_in_a_long_prompt(d):
    """Segments of some 800 key tiles, several a CTA, with NaN values in the first and the last
    key tile and one amid: NaN where a row sees one, and elsewhere the bits of the call on
    zeros in their place; the look for them is bounded, so the call takes about as long."""
    import torch
    torch.manual_seed(d)
    Hk, T, n, page = 40, 600, 131072 - 5, 1024
    table = torch.randperm(128, device="cuda", dtype=torch.int32).view(1, 128)
    kp, vp = (torch.randint(0, 0x78, (128, Hk, page, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((128, Hk), 2.0 ** -8, device="cuda") for _ in range(2))
    q, lens = torch.randn(1, Hk, T, d, device="cuda").bfloat16(), i32([n])
    at = [(0, 0, 5), (1, 0, 5), (1, n - 1, 7), (2, n - 1, 0), (3, n - 300, d - 1), (4, 70000, 33), (39, n - 2, 1), (39, 17, 2)]

    def put(code):
        for h, j, c in at:
            vp[table[0, j // page], h, j % page, c] = code

    def timed():
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ends[0].record()
        out = api.fwd_cache(q, kp, vp, ks, vs, table, lens)
        ends[1].record()
        torch.cuda.synchronize()
        return out, ends[0].elapsed_time(ends[1])

    put(0)
    timed()
    (want, lse), clean = timed()
    put(0x7F)
    (o, lse2), found = timed()
    check_clean()
    nan = torch.zeros_like(want, dtype=torch.bool)
    for h, j, c in at:
        nan[0, h, max(0, j - (n - T)):, c] = True
    assert torch.equal(torch.isnan(o), nan) and not torch.isnan(want).any()
    assert torch.equal(o[~nan], want[~nan]) and torch.equal(lse, lse2)
    assert found <= 5 * clean + 20, (clean, found)  # ms: some seven tiles to look through a segment


def test_bad_pages_and_lengths_are_reported():
    import torch
    pool = Pool(12, 2, 1, 64, 16, 4)
    good = pool.dev()
    q, _ = bf16(pool.rng, (2, 2, 1, 64))
    k, _ = bf16(pool.rng, (2, 1, 1, 64))
    for entry in (-1, good[0].shape[0], 2 ** 31 - 1):
        table = good[4].clone()
        table[1, 2] = entry
        api.fwd_cache(q, *good[:4], table, i32([64, 40]))
        assert api.check_device_error()[0] == -5
        before = [t.clone() for t in good[:4]]
        api.cache_append(k, k, *good[:4], table, i32([64, 40]), new_lens=i32([0, 1]))
        assert api.check_device_error()[0] == -5
        assert all(torch.equal(a, b) for a, b in zip(before, good[:4]))
    api.cache_append(k, k, *good, i32([64, 65]), new_lens=i32([0, 1]))  # one token behind the table
    assert api.check_device_error()[0] == -5
    many, _ = bf16(pool.rng, (2, 2, 70, 64))
    for x in (q, many):
        for lens in ([64, 65], [-1, 3], [2 ** 31 - 1, 64]):
            api.fwd_cache(x, *good, i32(lens))
            assert api.check_device_error()[0] == -5
        table = good[4].clone()
        table[0, 1] = -7
        api.fwd_cache(x, *good[:4], table, i32([64, 40]))
        assert api.check_device_error()[0] == -5
        api.fwd_cache(x, *good, i32([64, 0]))
        assert api.check_device_error() == (0, 0)
    assert api.check_device_error() == (0, 0)


@pytest.mark.parametrize("new", [0, 1, 3])
@pytest.mark.parametrize("length", [-1, -2 ** 31, 65, 67, 68, 2 ** 31 - 1, 2 ** 31 - 16])
def test_append_reports_lengths_outside_the_table(length, new):
    """A length that is negative or behind the table is reported, tokens of it or not; what it
    has inside the table is written, and nothing else; the other sequence as ever."""
    pool = Pool(41, 2, 1, 64, 16, 4)
    dev = pool.dev()
    k, kv = bf16(pool.rng, (2, 1, 3, 64))
    api.cache_append(k, k, *dev, i32([length, 40]), new_lens=i32([new, 2]))
    assert api.check_device_error()[0] == -5
    inside = max(0, 64 - (length - new)) if 64 < length <= 64 + new else 0  # first of the new tokens
    if inside:
        streaming.cache_append(kv[:1, :, :inside], kv[:1, :, :inside], pool.k, pool.v, pool.ks, pool.vs, pool.table[:1],
                               [64], [inside])
    streaming.cache_append(kv[1:], kv[1:], pool.k, pool.v, pool.ks, pool.vs, pool.table[1:], [40], [2])
    for got, want in zip(dev[:4], (pool.k, pool.v, pool.ks, pool.vs)):
        assert np.array_equal(got.cpu().numpy(), want.astype(got.cpu().numpy().dtype))
    check_clean()


def odd_single(t, dims):
    """t with a stride of 1 or 3 over its dimensions of one element, as PyTorch may hold it."""
    strides = list(t.stride())
    for n, i in enumerate(dims):
        assert t.shape[i] == 1
        strides[i] = 1 + 2 * (n % 2)
    return t.as_strided(t.shape, strides)


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_strides_over_one_element_are_not_looked_at(layout):
    """One token of one sequence and head, or a single page: the strides of such dimensions are
    not multiples of anything, and the call is the one of dense tensors."""
    import torch
    pool = Pool(42, 1, 1, 64, 16, 1, spare=0)
    dev, odd = pool.dev(), [odd_single(t, range(t.dim() - 2)) if t.dim() == 4 else t for t in pool.dev()]
    assert odd[4].shape == (1, 1)
    odd[4] = odd_single(odd[4], (0, 1))
    q, k = (bf16(pool.rng, (1, 1, 1, 64), layout)[0] for _ in range(2))
    lens = i32([5])
    want = api.fwd_cache(q, *dev, lens, layout=layout)
    got = api.fwd_cache(odd_single(q, range(3)), *odd, lens, layout=layout, o=odd_single(torch.empty_like(q), range(3)))
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    api.cache_append(k, k, *dev, lens, layout=layout)
    api.cache_append(odd_single(k, range(3)), odd_single(k, (2, 1, 0)), *odd, lens, layout=layout)
    assert all(torch.equal(x, y) for x, y in zip(dev, odd))
    # new tokens as a column, [B, Hk, d, 1] seen as [B, Hk, 1, d]; two sequences of one page each
    pool = Pool(43, 2, 2, 128, 32, 1)
    dev, odd = pool.dev(), pool.dev()
    odd[4] = odd[4].as_strided((2, 1), (1, 2))
    q, k = (bf16(pool.rng, (2, h, 1, 128))[0] for h in (4, 2))
    column = lambda t: t.reshape(*t.shape[:2], 128, 1).transpose(2, 3)
    assert column(k).stride()[2] == 1 and odd[4].stride()[1] == 2
    lens = i32([7, 30])
    for args, x, y in ((dev, k, q), (odd, column(k), column(q))):
        api.cache_append(x, x, *args, lens)
        want, got = got, api.fwd_cache(y, *args, lens)
    assert all(torch.equal(x, y) for x, y in zip((*want, *dev), (*got, *odd)))
    check_clean()


def test_reads_and_writes_past_32_bits():
    """A pool of 2.1 GB per tensor whose last pages are in use."""
    import torch
    P, Hk, page, d = 2080, 8, 1024, 128
    kp, vp = (torch.zeros((P, Hk, page, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    assert kp.numel() > 1 << 31
    ks, vs = (torch.ones((P, Hk), device="cuda") for _ in range(2))
    rng = np.random.default_rng(13)
    table = np.array([[P - 1, P - 2]], dtype=np.int32)
    k, kv = bf16(rng, (1, Hk, 1100, d))
    v, vv = bf16(rng, (1, Hk, 1100, d))
    q, qv = bf16(rng, (1, 16, 1, d))
    args = (kp, vp, ks, vs, torch.from_numpy(table).cuda(), i32([1100]))
    api.cache_append(k, v, *args)
    o, lse = api.fwd_cache(q, *args)
    check_clean()
    small = [np.zeros((2, Hk, page, d), dtype=np.uint8) for _ in range(2)]
    sc = [np.ones((2, Hk)) for _ in range(2)]
    streaming.cache_append(kv, vv, *small, *sc, [[1, 0]], [1100], [1100])
    for dev, ref in ((kp, small[0]), (vp, small[1])):
        assert np.array_equal(dev[P - 2:].cpu().numpy(), ref)
        assert int(dev[:P - 2].count_nonzero()) == 0
    check_out(o, lse, streaming.cache_forward(qv, *small, *sc, [[1, 0]], [1100], [1], d ** -0.5))


# (B, Hk, page, T, [(seq_lens, new_lens), ...])
APPENDS = [
    (1, 1, 16, 1, [([1], None), ([2], None), ([17], None)]),
    (2, 2, 16, 40, [([40, 3], [40, 3]), ([41, 30], [1, 27]), ([48, 70], [7, 40])]),
    (3, 1, 64, 100, [([100, 64, 0], [100, 64, 0]), ([101, 65, 1], [1, 1, 1]), ([190, 128, 2], [89, 63, 1])]),
    (1, 3, 128, 300, [([300], None), ([450], [150])]),
    (1, 1, 32, 10, [([4], None)]),  # more new tokens than the sequence has: the last 4 are written
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout,token_major", [("bhnd", False), ("bnhd", True)])
@pytest.mark.parametrize("case", APPENDS)
def test_append_matches_oracle(case, layout, token_major, d):
    B, Hk, page, T, calls = case
    pool = Pool(20 + T, B, Hk, d, page, -(-max(max(c[0]) for c in calls) // page), token_major=token_major)
    dev = pool.dev()
    for n, (lens, new) in enumerate(calls):
        # later calls bring larger values: scales grow and older codes are rounded again
        k, kv = bf16(pool.rng, (B, Hk, T, d), layout, amp=2.0 ** (2 * n))
        v, vv = bf16(pool.rng, (B, Hk, T, d), layout, amp=2.0 ** (-3 * n))
        api.cache_append(k, v, *dev, i32(lens), new_lens=None if new is None else i32(new), layout=layout)
        streaming.cache_append(kv, vv, pool.k, pool.v, pool.ks, pool.vs, pool.table, lens,
                               [T] * B if new is None else new)
        check_clean()
        for got, want in zip(dev[:4], (pool.k, pool.v, pool.ks, pool.vs)):
            assert np.array_equal(got.cpu().numpy(), want.astype(got.cpu().numpy().dtype)), n


def test_append_special_values():
    """Zeros, subnormals, infinities, NaN, the largest numbers, values on a rounding border."""
    import torch
    rows = np.zeros((1, 1, 6, 64), dtype=np.float32)
    rows[0, 0, 1] = 1e-39
    rows[0, 0, 2, :4] = [np.inf, -np.inf, np.nan, 2.0]
    rows[0, 0, 3, :6] = [448, 449, -450, 17, 19, 21]
    rows[0, 0, 4] = 3.3e38
    rows[0, 0, 5, :3] = [2.0 ** -133, 2.0 ** -126, 1.0]
    x = torch.from_numpy(rows).bfloat16()
    for t in range(6):
        pool = Pool(30, 1, 1, 64, 16, 1)
        dev = pool.dev()
        one = x[:, :, t:t + 1].contiguous()
        api.cache_append(one.cuda(), one.cuda(), *dev, i32([1]))
        streaming.cache_append(one.double().numpy(), one.double().numpy(), pool.k, pool.v, pool.ks, pool.vs,
                               pool.table, [1], [1])
        assert np.array_equal(dev[2].cpu().numpy(), pool.ks.astype(np.float32)), t
        assert np.array_equal(dev[0].cpu().numpy(), pool.k), t
    check_clean()


@pytest.mark.parametrize("scale", [0.3, 0.007, 1.0 / 3.0, 2.0 ** -110, 1e30])
def test_append_keeps_a_scale_that_is_no_power_of_two(scale):
    """A page of a user's own scale: codes are the fp32 quotients x / scale, rounded."""
    pool = Pool(31, 1, 2, 128, 32, 1)
    pool.ks[:], pool.vs[:] = np.float32(scale), np.float32(scale)
    dev = pool.dev()
    k, kv = bf16(pool.rng, (1, 2, 20, 128))
    api.cache_append(k, k, *dev, i32([29]), new_lens=i32([20]))
    streaming.cache_append(kv, kv, pool.k, pool.v, pool.ks, pool.vs, pool.table, [29], [20])
    check_clean()
    for got, want in zip(dev[:4], (pool.k, pool.v, pool.ks, pool.vs)):
        assert np.array_equal(got.cpu().numpy(), want.astype(got.cpu().numpy().dtype))


def test_refusals():
    import torch
    pool = Pool(40, 2, 2, 64, 16, 3)
    kp, vp, ks, vs, table = pool.dev()
    lens = i32([20, 30])
    q, _ = bf16(pool.rng, (2, 4, 1, 64))
    k, _ = bf16(pool.rng, (2, 2, 1, 64))
    ok = dict(q=q, k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs, page_table=table, seq_lens=lens)
    api.fwd_cache(**ok)
    bad = [dict(q=q.float()), dict(q=q[:1]), dict(q=q.cpu()), dict(k_pages=kp.to(torch.int32)), dict(v_pages=vp[:-1]),
           dict(k_scale=ks.half()), dict(v_scale=vs.t()), dict(page_table=table.long()), dict(page_table=table[:1]),
           dict(page_table=table.t()), dict(seq_lens=lens.long()), dict(seq_lens=lens.cpu()), dict(q_lens=lens[:1]),
           dict(layout="nbhd"), dict(o=torch.empty_like(q).float()), dict(lse=torch.empty(2, 4, 2, device="cuda")),
           dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(k_pages=kp[..., ::2], v_pages=vp[..., ::2])]
    for change in bad:
        with pytest.raises(ValueError):
            api.fwd_cache(**{**ok, **change})
    # three query heads over two, a page of 12 or 8 tokens, bounds below -1, scales that are not positive
    for change in (dict(q=q[:, :3]), dict(o=torch.empty_like(q)[:, :1].expand(-1, 4, -1, -1)), dict(k_pages=kp[:, :, :12], v_pages=vp[:, :, :12]), dict(window_left=-2),
                   dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")),
                   dict(k_pages=kp[:, :, :8], v_pages=vp[:, :, :8])):
        with pytest.raises((ValueError, api.AttnError)):
            api.fwd_cache(**{**ok, **change})
    with pytest.raises(api.AttnError):  # heads that share their pages' memory
        api.cache_append(k, k, kp[:, :1].expand(-1, 2, -1, -1), vp[:, :1].expand(-1, 2, -1, -1), ks, vs, table, lens)
    for args in ((k.float(), k), (k, k[:1]), (k[..., ::2], k[..., ::2]), (k.cpu(), k.cpu()), (q, q)):
        with pytest.raises((ValueError, api.AttnError)):
            api.cache_append(*args, kp, vp, ks, vs, table, lens)
    check_clean()


def test_a_workspace_without_its_bytes_is_refused(monkeypatch):
    """An expanded or strided tensor as workspace is refused by both halves of the binding."""
    import torch
    pool = Pool(44, 2, 2, 64, 16, 3)
    dev, lens = pool.dev(), i32([20, 30])
    q, k = (bf16(pool.rng, (2, h, 20, 64))[0] for h in (4, 2))
    o, lse = api.fwd_sinks(q, k, k, 5, 1)
    room = max(api.fwd_cache_workspace_bytes(2, 4, 2, 20, 64), api.bwd_sinks_workspace_bytes(2, 4, 2, 20, 64, 1))
    byte = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for half in range(2):
        for ws in (byte.expand(room), torch.empty(2 * room, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError, match="contiguous bytes"):
                api.fwd_cache(q, *dev, lens, workspace=ws)
            with pytest.raises(ValueError, match="contiguous bytes"):
                api.bwd_sinks(q, k, k, o, q, lse, 5, 1, workspace=ws)
        monkeypatch.setattr(api, "_compiled_calls", lambda: None)
    check_clean()


def test_on_another_stream_and_in_a_replayed_graph():
    """A captured decode step (write, then attend) is replayed with new tokens and lengths in
    the captured buffers; an eager call on a stream of its own gives the same bits."""
    import torch
    pool = Pool(50, 3, 2, 128, 16, 6)
    dev = pool.dev()
    q, k, v = (bf16(pool.rng, (3, h, 1, 128))[0] for h in (8, 2, 2))
    lens = i32([40, 15, 80])
    o, lse = torch.empty_like(q), torch.empty((3, 8, 1), device="cuda")
    ws = torch.empty(api.fwd_cache_workspace_bytes(3, 8, 2, 1, 128), dtype=torch.uint8, device="cuda")
    eager = [t.clone() for t in dev]

    def step():
        api.cache_append(k, v, *dev, lens)
        api.fwd_cache(q, *dev, lens, o=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(3):
        for t, h in ((q, 8), (k, 2), (v, 2)):
            t.copy_(bf16(pool.rng, (3, h, 1, 128))[0])
        lens.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        api.cache_append(k, v, *eager, lens, stream=side)
        o2, lse2 = api.fwd_cache(q, *eager, lens, stream=side)
        side.synchronize()
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2), n
        assert all(torch.equal(a, b) for a, b in zip(dev, eager))
    check_clean()


def test_two_calls_at_once_with_a_workspace_each():
    import torch
    pool = Pool(60, 4, 2, 128, 64, 40)
    dev = pool.dev()
    lens = i32([2500, 2000, 1500, 2222])
    qs = [bf16(pool.rng, (4, 16, 1, 128))[0] for _ in range(2)]
    alone = [api.fwd_cache(q, *dev, lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [api.fwd_cache(q, *dev, lens, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for (o, lse), (o2, lse2) in zip(alone, got):
            assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    check_clean()


def test_calls_of_two_threads_on_one_stream():
    """Each thread's calls without a workspace keep one of their own."""
    import threading

    import torch
    pool = Pool(61, 4, 2, 128, 64, 40)
    dev = pool.dev()
    lens = i32([2500, 2000, 1500, 2222])
    qs = [bf16(pool.rng, (4, 16, 1, 128))[0] for _ in range(2)]
    want = [api.fwd_cache(q, *dev, lens)[0] for q in qs]
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        start.wait()
        for _ in range(40):
            got[i].append(api.fwd_cache(qs[i], *dev, lens)[0])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o.view(torch.int16), want[i].view(torch.int16)) for o in got[i])
    check_clean()


def test_kept_workspaces_are_given_back():
    """What calls of this thread keep, on two streams, is back in the allocator after
    release_workspaces, and the calls' results are not touched."""
    import torch
    pool = Pool(63, 2, 2, 128, 64, 10)
    dev, lens = pool.dev(), i32([600, 500])
    q = bf16(pool.rng, (2, 16, 70, 128))[0]
    api.release_workspaces()
    room = api.fwd_cache_workspace_bytes(2, 16, 2, 70, 128)
    before, outs = torch.cuda.memory_allocated(), []
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(api.fwd_cache(q, *dev, lens))
    taken = torch.cuda.memory_allocated() - before
    assert taken >= 2 * room
    api.release_workspaces()
    assert torch.cuda.memory_allocated() - before <= taken - 2 * room
    outs.append(api.fwd_cache(q, *dev, lens))
    torch.cuda.synchronize()
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    check_clean()


def test_a_graph_keeps_no_workspace_of_eager_calls():
    """Two graphs captured without a workspace, replayed at once on two streams."""
    import torch
    pool = Pool(62, 4, 2, 128, 64, 40)
    dev = pool.dev()
    lens = i32([2500, 2000, 1500, 2222])
    qs = [bf16(pool.rng, (4, 16, 1, 128))[0] for _ in range(2)]
    want = [api.fwd_cache(q, *dev, lens) for q in qs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for q, s in zip(qs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(api.fwd_cache(q, *dev, lens))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        api.fwd_cache(qs[0], *dev, lens)
    torch.cuda.synchronize()
    for (o, lse), (o2, lse2) in zip(want, outs):
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    check_clean()


@pytest.mark.parametrize("d", [64, 128])
def test_a_prompt_through_the_cache_is_the_whole_sequence_call(d):
    """A prompt's own attention over what the cache holds of it against attn_fwd_sinks on the
    values the codes stand for (four significant bits: exact in bf16), and the next tokens one
    by one against its later rows.  Both sides are within 1e-2 (beyond their bf16 rounding) of
    the same numbers; LSE within 1e-3."""
    import torch
    B, H, Hk, N, more, left, sinks, page = 2, 8, 2, 333, 3, 90, 5, 32
    pool = Pool(71, B, Hk, d, page, -(-(N + more) // page))
    dev = pool.dev()
    k, v = (bf16(pool.rng, (B, Hk, N + more, d))[0] for _ in range(2))
    q, _ = bf16(pool.rng, (B, H, N + more, d))
    outs = []
    for lo, hi in [(0, N)] + [(n, n + 1) for n in range(N, N + more)]:
        lens = i32([hi] * B)
        api.cache_append(k[:, :, lo:hi], v[:, :, lo:hi], *dev, lens)
        outs.append(api.fwd_cache(q[:, :, lo:hi].contiguous(), *dev, lens, window_left=left, sinks=sinks))
    table = dev[4].long()
    kd, vd = ((pages[table].view(torch.float8_e4m3fn).float() * sc[table][..., None, None]).transpose(1, 2)
              .reshape(B, Hk, -1, d)[:, :, :N + more].bfloat16().contiguous() for pages, sc in zip(dev[:2], dev[2:4]))
    o, lse = api.fwd_sinks(q, kd, vd, left, sinks)
    check_clean()
    got = torch.cat([x for x, _ in outs], 2).double()
    assert torch.all((got - o.double()).abs() <= 2e-2 + 2.0 ** -7 * o.double().abs())
    assert torch.all((torch.cat([x for _, x in outs], 2) - lse).abs() <= 2e-3)


def test_decode_as_it_is_used():
    """A prompt is written in two pieces, then tokens one by one; after each the attention of
    the new tokens over what the cache holds is the oracle's."""
    pool = Pool(70, 2, 2, 64, 32, 5)
    dev = pool.dev()
    length = np.array([0, 0])
    for new in ([50, 33], [20, 1], [1, 1], [1, 1], [1, 0], [3, 2]):
        T = max(new)
        length = length + new
        k, kv = bf16(pool.rng, (2, 2, T, 64))
        v, vv = bf16(pool.rng, (2, 2, T, 64), amp=1.0 + T)
        q, qv = bf16(pool.rng, (2, 6, T, 64))
        lens = length.tolist()
        api.cache_append(k, v, *dev, i32(lens), new_lens=i32(new))
        o, lse = api.fwd_cache(q, *dev, i32(lens), q_lens=i32(new), window_left=45, sinks=4)
        check_clean()
        streaming.cache_append(kv, vv, pool.k, pool.v, pool.ks, pool.vs, pool.table, lens, new)
        assert np.array_equal(dev[0].cpu().numpy(), pool.k) and np.array_equal(dev[1].cpu().numpy(), pool.v)
        check_out(o, lse, streaming.cache_forward(qv, pool.k, pool.v, pool.ks, pool.vs, pool.table, lens, new,
                                                  64 ** -0.5, 45, 4))


@pytest.mark.parametrize("T", [1, 70])
def test_calls_that_follow_copies_and_other_streams(T):
    """What a call reads was written just before it: by a copy, by a kernel of another stream
    that it waits for, by the call before it; eager and captured, many times over."""
    import torch
    torch.manual_seed(5)
    B, H, Hk, d, page, n = 3, 8, 2, 64, 32, 400
    kp, vp = (torch.randint(0, 0x70, (40, Hk, page, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((40, Hk), 2.0 ** -6, device="cuda") for _ in range(2))
    table = torch.randperm(39, device="cuda", dtype=torch.int32).view(3, 13)
    k, q = (torch.randn(B, h, T, d, device="cuda").bfloat16() for h in (Hk, H))
    want_lens = [i32([n, 71, 133]), i32([150, n, 70])]
    lens, q_in = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros_like(q)
    pages = [x.clone() for x in (kp, vp, ks, vs)]
    side, o = torch.cuda.Stream(), [torch.empty_like(q) for _ in want_lens]
    lse = [torch.empty(B, H, T, device="cuda") for _ in want_lens]

    def steps():
        here = torch.cuda.current_stream()
        for i, w in enumerate(want_lens):
            lens.copy_(w)
            api.cache_append(k, k, *pages, table, lens)
            side.wait_stream(here)
            with torch.cuda.stream(side):
                q_in.copy_(q)
                q_in.mul_(1 - 2 * i)
            here.wait_stream(side)
            api.fwd_cache(q_in, *pages, table, lens, o=o[i], lse=lse[i])
            q_in.zero_()
            lens.zero_()

    def reset():
        for x, y in zip(pages, (kp, vp, ks, vs)):
            x.copy_(y)

    # one step at a time
    want = []
    reset()
    for i, w in enumerate(want_lens):
        api.cache_append(k, k, *pages, table, w)
        torch.cuda.synchronize()
        want.append([x.clone() for x in api.fwd_cache(q * (1 - 2 * i), *pages, table, w)])
        torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    reset()
    with torch.cuda.graph(g, stream=s):
        steps()
    for run in [steps] * 20 + [g.replay] * 20:
        reset()
        for x in (*o, *lse):
            x.fill_(3.0)
        run()
        for (wo, wl), go, gl in zip(want, o, lse):
            assert torch.equal(wo.view(torch.int16), go.view(torch.int16)) and torch.equal(wl, gl)
    check_clean()


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_calls_read_in_python_and_compiled_are_the_same(layout, monkeypatch):
    """The two halves of the binding make the same call of the same arguments: with outputs
    and workspaces given and not, and NumPy's integers, which only the one in Python takes."""
    import torch
    assert api._compiled_calls() is not None
    torch.manual_seed(3)
    B, H, Hk, T, d = 2, 4, 2, 5, 64
    shape = lambda h, n: (B, h, n, d) if layout == "bhnd" else (B, n, h, d)
    new = lambda h, n: torch.randn(shape(h, n), device="cuda").bfloat16()
    kp, vp = (torch.randint(0, 0x70, (12, Hk, 32, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = [torch.full((12, Hk), 2.0 ** -6, device="cuda") for _ in range(2)]
    table, lens, ql = torch.arange(12, device="cuda", dtype=torch.int32).view(2, 6), i32([100, 7]), i32([5, 3])
    q, k, v = new(H, T), new(Hk, T), new(Hk, T)
    qs, ks, vs, do = new(H, 150), new(Hk, 150), new(Hk, 150), new(H, 150)
    room = torch.empty(max(api.fwd_cache_workspace_bytes(B, H, Hk, T, d), api.bwd_sinks_workspace_bytes(B, H, Hk, 150, d, 3)),
                       dtype=torch.uint8, device="cuda")

    def run(three, given):
        pages = [x.clone() for x in (kp, vp, *scales)]
        o, lse = (torch.empty_like(q), torch.empty(B, H, T, device="cuda")) if given else (None, None)
        og, lg = (torch.empty_like(qs), torch.empty(B, H, 150, device="cuda")) if given else (None, None)
        grads = [torch.empty_like(x) if given else None for x in (qs, ks, vs)]
        ws = room if given else None
        api.cache_append(k, v, *pages, table, lens, new_lens=ql, layout=layout)
        if not given:  # makes the kept workspace
            api.fwd_cache(q, *pages, table, lens, q_lens=ql, layout=layout)
        # rows behind the last query are left as they were: only those that there are count
        r = api.fwd_cache(q, *pages, table, lens, q_lens=ql, layout=layout, scale=0.2, window_left=three * 9, sinks=three,
                          o=o, lse=lse, workspace=ws)
        assert not given or (r[0] is o and r[1] is lse)
        there = r[0][1, :, :3] if layout == "bhnd" else r[0][1, :3]
        s = api.fwd_sinks(qs, ks, vs, three * 9, three, layout=layout, o=og, lse=lg)
        g = api.bwd_sinks(qs, ks, vs, s[0], do, s[1], three * 9, three, layout=layout, dq=grads[0], dk=grads[1],
                          dv=grads[2], workspace=ws)
        assert not given or all(x is y for x, y in zip(g, grads))
        # dQ is summed by fp32 reductions whose order changes, the others are the same bit for bit
        return [*pages, r[0][0], r[1][0], there, r[1][1, :, :3], *s, *g[1:]]

    want = run(3, True)
    for three, given in ((3, False), (np.int64(3), True)):
        for x, y in zip(want, run(three, given)):
            assert torch.equal(x, y)
    monkeypatch.setattr(api, "_compiled_calls", lambda: None)
    for given in (True, False):
        for x, y in zip(want, run(3, given)):
            assert torch.equal(x, y)
    check_clean()

