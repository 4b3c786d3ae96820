"""attn_fwd_cache_prefix in two parts as a server runs it: what the call reads is written just before it.
Results are compared bit for bit with those of calls that have the device to themselves, or with the
fp64 oracle (tolerances: test_gpu_cache)."""

import numpy as np
import pytest

from exact_attention_52_gb300 import api

from oracle import streaming

from .test_gpu_cache import bf16, check_clean, check_out, i32
from .test_gpu_prefix import run, shared_pool, wide

pytestmark = pytest.mark.gpu


def versions(n):
    """Inputs of n calls of the same sizes, and the pools' tensors on the device."""
    import torch
    B, H, Hk, T, d, page = 12, 16, 2, 2, 128, 64
    out = []
    for i in range(n):
        rng = np.random.default_rng(100 + i)
        firsts = [0, 5 + i % 3, 12]
        prefixes = [256 + 128 * (i % 3), 512 - 128 * (i % 2)]
        lens = [prefixes[b >= firsts[1]] + T + int(rng.integers(0, 200)) for b in range(B)]
        pool = shared_pool(200 + i, B, Hk, d, page, firsts, prefixes, lens)
        table = np.full((B, 16), 10 ** 6, dtype=np.int32)
        table[:, :pool.table.shape[1]] = pool.table
        pages = 16 * B + 3
        k, v = (np.zeros((pages, Hk, page, d), dtype=np.uint8) for _ in range(2))
        ks, vs = (np.ones((pages, Hk)) for _ in range(2))
        for big, small in ((k, pool.k), (v, pool.v), (ks, pool.ks), (vs, pool.vs)):
            big[:small.shape[0]] = small
        pool.table = table
        ql = [int(x) for x in rng.integers(1, T + 1, B)]
        out.append([torch.randn(B, H, T, d, device="cuda").bfloat16(), *(torch.from_numpy(x).cuda() for x in (k, v)),
                    *(torch.from_numpy(x).float().cuda() for x in (ks, vs)), i32(wide(table, pool)), i32(lens), i32(prefixes),
                    i32(firsts), i32(ql)])
    return out


def call(x, **kw):
    return api.fwd_cache_prefix(*x[:8], group_first=x[8], q_lens=x[9], **kw)


def outputs(like):
    import torch
    return torch.zeros_like(like[0]), torch.zeros(like[0].shape[:3], device="cuda")


def check_same(got, ref):
    import torch
    assert torch.equal(got[0].view(torch.int16), ref[0].view(torch.int16))
    assert torch.equal(got[1].view(torch.int32), ref[1].view(torch.int32))


def references(data):
    import torch
    refs = []
    for x in data:
        o, lse = outputs(x)
        torch.cuda.synchronize()
        call(x, o=o, lse=lse)
        torch.cuda.synchronize()
        refs.append((o, lse))
    check_clean()
    return refs


def test_a_call_sees_what_was_written_just_before_it():
    """Every input changes between calls that follow each other without a pause, and calls of another
    kind share the workspace that is kept for the stream."""
    import torch
    data = versions(4)
    refs = references(data)
    live, got = [t.clone() for t in data[0]], []
    for step in range(40):
        for t, new in zip(live, data[step % 4]):
            t.copy_(new)
        o, lse = outputs(live)
        call(live, o=o, lse=lse)
        got.append((o, lse))
        if step % 3 == 0:
            api.fwd_cache(*live[:7], q_lens=live[9])
    for step, x in enumerate(got):
        check_same(x, refs[step % 4])
    check_clean()


def test_captured_calls_that_share_a_workspace():
    """Two graphs, each of copies and calls, replayed in turn with one workspace, which other calls write
    over in between; a replayed call is the same call again."""
    import torch
    data = versions(4)
    refs = references(data)
    B, H, T, d = data[0][0].shape
    ws = torch.full((api.fwd_cache_prefix_workspace_bytes(B, H, 2, T, d),), 255, dtype=torch.uint8, device="cuda")
    live, graphs = [t.clone() for t in data[0]], []
    call(live, workspace=ws)
    torch.cuda.synchronize()
    for pair in ((0, 1), (2, 3)):
        g, outs = torch.cuda.CUDAGraph(), [outputs(live) for _ in pair]
        with torch.cuda.graph(g):
            for i, (o, lse) in zip(pair, outs):
                for t, new in zip(live, data[i]):
                    t.copy_(new)
                call(live, o=o, lse=lse, workspace=ws)
        graphs.append((g, pair, outs))
    for step in range(12):
        g, pair, outs = graphs[step % 2]
        for o, lse in outs:
            o.zero_(), lse.zero_()
        g.replay()
        for i, out in zip(pair, outs):
            check_same(out, refs[i])
        if step % 3 == 0:
            ws.fill_(step)
        elif step % 3 == 1:
            call(data[step % 4], workspace=ws)
    check_clean()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,prompt,shared", [(16, 300, 300), (64, 200, 200), (128, 320, 320), (128, 320, 256),
                                                (256, 400, 256), (512, 1100, 1024), (1024, 900, 0)])
def test_decoding_behind_a_prompt_that_ends_inside_a_page(page, prompt, shared, d):
    """Full pages are shared; of the page in which the prompt ends each sequence has a copy, which its own
    tokens go to, with values that make the page's scale grow at another step in each."""
    import torch
    B, H, Hk, steps = 6, 8, 2, 6
    rng = np.random.default_rng(prompt + d)
    full = prompt // page
    pool = shared_pool(page + d, B, Hk, d, page, [0, B], [full * page], [prompt + 2 * steps] * B)
    dev = pool.dev()
    dev[4] = i32(wide(pool.table, pool))
    new = lambda b, t, amp=1.0: torch.from_numpy((amp * rng.standard_normal((b, Hk, t, d))).astype(np.float32)).bfloat16().cuda()
    # the prompt, as the first sequence's, and the copies of its last page
    api.cache_append(new(1, prompt), new(1, prompt), *dev[:4], dev[4][:1], i32([prompt]))
    for x in dev[:4]:
        for b in range(1, B):
            x[int(pool.table[b, full])] = x[int(pool.table[0, full])]
    start = [x.clone() for x in dev[:4]]
    lens = np.full(B, prompt)
    for step in range(steps):
        T = 1 + step % 2
        k, v = new(B, T), new(B, T)
        k[step] *= 1000.0
        v[(step + 3) % B] *= 1000.0
        lens = lens + T
        seq = i32(lens)
        api.cache_append(k, v, *dev, seq)
        q, qv = bf16(rng, (B, H, T, d), amp=2.0 ** -10)  # scores of the large keys stay below 32
        o, lse = api.fwd_cache_prefix(q, *dev, seq, i32([shared]))
        check_clean()
        kc, vc = (x.cpu().numpy() for x in dev[:2])
        ks, vs = (x.double().cpu().numpy() for x in dev[2:4])
        check_out(o, lse, streaming.cache_forward(qv, kc, vc, ks, vs, pool.table, lens, [T] * B, d ** -0.5))
    for pid in pool.table[0, :full]:  # what is shared has stayed as it was
        assert all(torch.equal(x[int(pid)], y[int(pid)]) for x, y in zip(dev[:4], start))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T", [(65, 8, 1), (70, 4, 2), (200, 8, 1), (200, 32, 3)])
def test_more_sequences_than_a_warp_takes(B, H, T, d):
    """Above 64 sequences a block's threads find its share together, above 128 with several sequences
    each; lengths are ragged, slots are empty, a group may be."""
    rng = np.random.default_rng(B + T + d)
    cuts = sorted(int(x) for x in rng.integers(0, B + 1, 4))
    firsts = [0, *cuts, cuts[-1], B]  # an empty group
    prefixes = [int(x) for x in rng.choice([128, 256, 300, 640], len(firsts) - 1)]
    ql = [int(x) for x in rng.integers(0, T + 1, B)]
    lens = [0] * B
    for g, n in enumerate(prefixes):
        for b in range(firsts[g], firsts[g + 1]):
            lens[b] = n + T + int(rng.integers(0, 250)) if ql[b] or rng.integers(0, 2) else 0
    pool = shared_pool(B, B, 2, d, 32, firsts, prefixes, lens)
    run(pool, H, T, firsts, prefixes, lens, ql)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("groups,B", [(33, 240), (64, 400), (100, 610)])
def test_more_groups_than_lanes(groups, B, d):
    """More than 32 groups: a lane of the prefixes' launch adds several up.  Some are empty, some share
    nothing, some have more than a pair of query tiles."""
    rng = np.random.default_rng(groups + d)
    inner = sorted(int(x) for x in rng.integers(0, B - 130, groups - 2))
    firsts = [0, *inner, B - 129, B]  # 129 sequences of 2 rows in the last group
    prefixes = [int(x) for x in rng.choice([0, 100, 128, 200, 384], groups - 1)] + [256]
    ql = [int(x) for x in rng.integers(0, 2, B)]
    lens = [0] * B
    for g, n in enumerate(prefixes):
        for b in range(firsts[g], firsts[g + 1]):
            lens[b] = n + 1 + int(rng.integers(0, 40))
    pool = shared_pool(groups, B, 1, d, 16, firsts, prefixes, lens)
    run(pool, 2, 1, firsts, prefixes, lens, ql)


@pytest.mark.parametrize("compiled", [True, False])
def test_the_columns_in_use_of_a_wide_table(compiled, monkeypatch):
    """A view of a wide table's first columns is the narrow table: the same path and the same bits."""
    import torch
    if not compiled:
        monkeypatch.setattr(api, "_read", lambda *a: (None, None, None))
    lens = [300 + 11 * b for b in range(8)]
    pool = shared_pool(41, 8, 2, 128, 64, [0, 8], [256], lens)
    q, dev = torch.randn(8, 16, 1, 128, device="cuda").bfloat16(), pool.dev()
    ref = api.fwd_cache(q, *dev, i32(lens))
    whole = i32(wide(pool.table, pool))
    check_same(api.fwd_cache_prefix(q, *dev[:4], whole[:, :dev[4].shape[1]], i32(lens), i32([256])), ref)
    o, lse = api.fwd_cache_prefix(q, *dev[:4], whole, i32(lens), i32([256]))  # in two parts
    check_clean()
    host = [x.cpu().numpy() for x in dev[:2]] + [x.double().cpu().numpy() for x in dev[2:4]]
    check_out(o, lse, streaming.cache_forward(q.double().cpu().numpy(), *host, pool.table, lens, [1] * 8, 128 ** -0.5))
