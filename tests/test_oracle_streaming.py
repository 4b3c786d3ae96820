"""Pins of the streaming oracle (CPU): the mask against its definition, E4M3 encoding
against PyTorch's, the cache against dense attention, gradients against differences."""

import numpy as np
import pytest

import oracle
from oracle import streaming


@pytest.mark.parametrize("left,sinks,right", [(-1, 0, 0), (3, 0, 0), (3, 2, 0), (0, 1, 0), (2, 4, 1), (2, 1, -1)])
def test_visible_by_definition(left, sinks, right):
    vis = streaming.sink_visible(np.arange(4, 13), 13, left, sinks, right)
    for i, p in enumerate(range(4, 13)):
        for j in range(13):
            want = (right < 0 or j <= p + right) and (left < 0 or j >= p - left or j < sinks)
            assert vis[i, j] == want
    if sinks == 0:
        full = streaming.sink_visible(np.arange(13), 13, left, 0, right)
        assert np.array_equal(full, oracle.window_visible(13, 13, (left, right)))


def test_encode_matches_torch_and_roundtrips():
    import torch
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert np.array_equal(streaming.e4m3_encode(oracle.e4m3_to_f64(codes)), codes)
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 9, 4000),
                        np.arange(-80, 81) * 2.0 ** -10]).clip(-448, 448).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(streaming.e4m3_encode(y), want)
    assert streaming.e4m3_encode(np.array([1e9, -np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7F]


def test_append_exponent():
    for amax, e in ((448.0, 0), (449.0, 1), (224.0, -1), (1.75, -8), (1.76, -7), (0.0, -100), (1e-40, -100)):
        assert streaming.append_exponent(amax) == e


def test_cache_forward_is_dense_attention_of_what_was_appended():
    rng = np.random.default_rng(2)
    B, H, Hk, page, d, n = 2, 4, 2, 16, 8, 37
    q, k, v = (rng.standard_normal((B, h, n, d)) for h in (H, Hk, Hk))
    table = rng.permutation(6).reshape(B, 3)
    kp, vp = (np.zeros((6, Hk, page, d), dtype=np.uint8) for _ in range(2))
    ks, vs = (np.ones((6, Hk)) for _ in range(2))
    for end, m in ((20, 20), (21, 1), (n, 16)):
        streaming.cache_append(k[:, :, end - m:end], v[:, :, end - m:end], kp, vp, ks, vs, table, [end] * B, [m] * B)
    dense = [np.zeros((B, Hk, n, d)) for _ in range(2)]
    for b in range(B):
        for j in range(n):
            pid = table[b, j // page]
            for out, pages, sc in zip(dense, (kp, vp), (ks, vs)):
                out[b, :, j] = oracle.e4m3_to_f64(pages[pid, :, j % page]) * sc[pid][:, None]
    assert np.abs(dense[0] - k).max() < 0.0625 * np.abs(k).max() and np.abs(dense[1] - v).max() < 0.0625 * np.abs(v).max()
    o, lse, _, there = streaming.cache_forward(q[:, :, -5:], kp, vp, ks, vs, table, [n] * B, [5] * B, 0.3, left=4, sinks=2)
    o_ref, lse_ref = streaming.sinks_forward(q, *dense, 0.3, 4, 2)
    assert there.all() and np.allclose(o, o_ref[:, :, -5:]) and np.allclose(lse, lse_ref[:, :, -5:])


def test_rows_that_see_nothing():
    q = np.ones((1, 1, 2, 4))
    pages, sc = np.zeros((1, 1, 16, 4), dtype=np.uint8), np.ones((1, 1))
    o, lse, _, _ = streaming.cache_forward(q, pages, pages, sc, sc, [[0]], [1], [2], 1.0)
    assert np.all(o[0, 0, 0] == 0) and np.isposinf(lse[0, 0, 0]) and np.isfinite(lse[0, 0, 1])


@pytest.mark.parametrize("left,sinks", [(2, 1), (3, 5), (0, 2)])
def test_sinks_gradients_match_differences(left, sinks):
    rng = np.random.default_rng(3)
    q, k, v, do = (rng.standard_normal((1, h, 11, 4)) for h in (2, 1, 1, 2))
    grads = streaming.sinks_backward(q, k, v, do, 0.4, left, sinks)
    loss = lambda: float(np.sum(streaming.sinks_forward(q, k, v, 0.4, left, sinks)[0] * do))
    for x, g in zip((q, k, v), grads):
        for _ in range(12):
            at = tuple(rng.integers(0, s) for s in x.shape)
            keep, h = x[at], 1e-5
            x[at] = keep + h
            up = loss()
            x[at] = keep - h
            down = loss()
            x[at] = keep
            assert abs((up - down) / (2 * h) - g[at]) < 1e-7
