"""attn_rope, attn_rope_bwd and attn_cache_append_rope refuse bad arguments before the device is
looked at (no GPU needed)."""

import ctypes
import os

import pytest

from exact_attention_52_gb300 import api

from .test_compiled_calls import CALLS, module  # noqa: F401

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return api.load_library()


def test_bad_arguments_are_refused(lib):
    fake = ctypes.c_void_p(1 << 20)
    st = api.Strides(64 * 8, 64 * 8, 64)

    def view(turns=1 << 20, qw=0, kw=0, bf=0, rot=64, inter=0, factor=1.0, eps=1e-6):
        return api._ROPE.pack(turns, qw, kw, bf, rot, inter, factor, eps)

    def call(v, q=fake, qs=st, H=1, Hk=1, N=8, d=64, step=0, pos=None):
        return lib.attn_rope(v, q, qs, fake, st, fake, st, fake, st, pos, step, 1, H, Hk, N, d, None)
    for v in (view(turns=0), view(turns=(1 << 20) + 8), view(rot=0), view(rot=8), view(rot=24), view(rot=80), view(inter=2),
              view(bf=2), view(factor=float("nan")), view(qw=8), view(kw=1 << 20, eps=0.0), None):
        assert call(v) == -1
    for kw in (dict(q=None), dict(q=ctypes.c_void_p((1 << 20) + 8)), dict(qs=api.Strides(64, 64, 63)), dict(H=0), dict(Hk=-1),
               dict(H=65535), dict(N=0), dict(step=-1), dict(pos=ctypes.c_void_p(2))):
        assert call(view(), **kw) == -1
    assert call(view(), d=96) == -2
    bwd = lambda v, x, ws: lib.attn_rope_bwd(v, x, st, fake, st, fake, st, fake, fake, st, fake, st, fake, st, fake, ws, None,
                                             0, 1, 1, 1, 8, 64, None)
    assert bwd(view(qw=1 << 20), None, fake) == -1
    assert bwd(view(qw=1 << 20), fake, None) == -1
    assert bwd(view(qw=1 << 20), fake, ctypes.c_void_p((1 << 20) + 16)) == -1
    assert lib.attn_rope_bwd_workspace_bytes(1, 1, -1, 8, 64) == 0
    assert lib.attn_rope_bwd_workspace_bytes(0, 1, 1, 8, 64) == 0
    assert lib.attn_rope_bwd_workspace_bytes(1, 1, 0, 8, 128) > 0


def test_a_bad_append_is_refused(lib):
    fake, st = ctypes.c_void_p(1 << 20), api.Strides(64, 64, 64)
    table = api._ROPE.pack(1 << 20, 0, 0, 0, 64, 0, 1.0, 1e-6)

    def call(cache=None, rope=table, q=fake, k=fake, qs=st, H=1, d=64, page=16, ks=64):
        if cache is None:
            cache = api._CACHE.pack(*[1 << 20] * 2, *[ks] * 6, *[1 << 20] * 3, 1, 1 << 20, 1, page, 1)
        return lib.attn_cache_append_rope(cache, rope, q, qs, fake, st, k, st, fake, st, None, 1, H, 1, 1, d, None)
    for kw in (dict(rope=None), dict(q=None), dict(k=None), dict(H=0), dict(H=65536), dict(page=24), dict(page=8), dict(ks=0),
               dict(rope=api._ROPE.pack(1 << 20, 0, 0, 0, 128, 0, 1.0, 1e-6))):
        assert call(**kw) == -1, kw
    assert call(d=96) == -2


def test_calls_without_a_gpu_name_the_argument():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 2, 4, 64).bfloat16()
    table = api.rope_table(64, device="cpu")
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        api.rope(q, q, table)
    with pytest.raises(ValueError, match="dq_out must be a CUDA tensor"):
        api.rope_bwd(q, q, table)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        api.cache_append_rope(q, q, q, table, q, q, q, q, q, q)
    with pytest.raises(ValueError, match="unknown layout"):
        api.rope(q, q, table, layout="nbhd")


def test_a_bad_prefix_is_refused(lib):
    fake, st = ctypes.c_void_p(1 << 20), api.Strides(64, 64, 64)
    cache = api._CACHE.pack(*[1 << 20] * 2, *[64] * 6, *[1 << 20] * 3, 1, 1 << 20, 1, 16, 1)

    def call(first=fake, lens=fake, groups=1, B=1, T=1, d=64, scale=0.125, ws=fake, q=fake):
        return lib.attn_fwd_cache_prefix(cache, first, lens, groups, q, st, fake, st, fake, ws, None, B, 1, 1, T, d, scale, None)
    for kw in (dict(lens=None), dict(lens=ctypes.c_void_p(2)), dict(first=ctypes.c_void_p((1 << 20) + 2)), dict(groups=0),
               dict(groups=2), dict(groups=-1), dict(B=0), dict(T=0), dict(scale=0.0), dict(ws=None),
               dict(ws=ctypes.c_void_p((1 << 20) + 16)), dict(q=None)):
        assert call(**kw) == -1, kw
    assert call(d=96) == -2
    sizes = lib.attn_fwd_cache_prefix_workspace_bytes
    assert sizes(1, 3, 2, 1, 64) == 0 and sizes(0, 1, 1, 1, 64) == 0 and sizes(1, 1, 1, 1, 96) == 0
    # both launches' segments, the items' CTAs, and fp32 rows with their statistics, twice
    r256 = lambda x: (x + 255) // 256 * 256
    seg = lambda T: lib.attn_fwd_cache_workspace_bytes(1, 1, 1, T, 128)
    for B, H, Hk, T in ((64, 32, 8, 2), (3, 40, 2, 3), (1, 1, 1, 1)):
        G, rows = H // Hk, B * T * H
        fin = r256(rows * 128 * 4) + r256(rows * 8)
        want = (seg(200) + r256((B * T * G // 256 + B + 1) * Hk * 8) + fin
                + seg(1) + r256(B * Hk * ((T * G + 7) // 8) * 8) + fin)
        assert sizes(B, H, Hk, T, 128) == want
    assert sizes(3, 40, 2, 70, 128) == lib.attn_fwd_cache_workspace_bytes(3, 40, 2, 70, 128)  # prompts


def test_the_compiled_half_gives_back_what_it_does_not_take(module):
    import torch
    functions = ((module.rope, 14), (module.rope_bwd, 19), (module.cache_append_rope, 20), (module.fwd_cache_prefix, 17))
    q = torch.zeros(1, 2, 4, 64).bfloat16()
    for f, n in functions:
        for t in (q, None, 3, "x", q.float(), q[0], torch.zeros(0)):
            assert f(*[t] * (n - 2), 0, 0) is None
        for m in (0, 1, n - 1, n + 1):
            assert f(*[None] * m) is None
    assert not CALLS
