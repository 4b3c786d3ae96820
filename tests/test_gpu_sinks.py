"""Sliding window with first tokens that stay visible (attn_fwd_sinks / attn_bwd_sinks)
against the fp64 oracle, forward and backward, at the tolerances of the window tests:
the kernels and their roundings (P and dS to bf16, fp32 sums) are the same.  A gradient
past its relative bound is held to the roundings' own, element by element
(rounding_bounds)."""

import numpy as np
import pytest

import oracle
from exact_attention_52_gb300 import api
from exact_attention_52_gb300.inputs import make_inputs_gqa
from oracle import streaming

from .helpers import (TOL_GRAD_RELFRO, TOL_LSE_ABS, TOL_O_MAXABS, bf16_out_err, bf16_to_device,
                      decoded, device_bf16_to_f64, device_f32_to_f64, grad_rel_err, max_abs, rel_fro)

pytestmark = pytest.mark.gpu


def check_clean():
    rc, site = api.check_device_error()
    assert rc == 0, f"device error {rc} at site {site:#x}"


def order(t, layout):
    return t if layout == "bhnd" else t.permute(0, 2, 1, 3).contiguous()


def check(B, H, Hk, N, d, left, sinks, right=0, layout="bhnd", backward=True, seed=0):
    inp = make_inputs_gqa(B, H, Hk, N, d, seed=seed + N + d + sinks + left, with_grad=True)
    q, k, v, do = (order(bf16_to_device(x), layout) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits))
    o, lse = api.fwd_sinks(q, k, v, left, sinks, right, layout=layout)
    check_clean()
    qf, kf, vf, dof = decoded(inp)
    scale = 1.0 / np.sqrt(d)
    o_ref, lse_ref = streaming.sinks_forward(qf, kf, vf, scale, left, sinks, right)
    host = lambda t: device_bf16_to_f64(order(t, layout))
    assert bf16_out_err(host(o), o_ref) <= TOL_O_MAXABS
    assert max_abs(device_f32_to_f64(lse), lse_ref) <= TOL_LSE_ABS
    if not backward:
        return
    grads = api.bwd_sinks(q, k, v, o, do, lse, left, sinks, right, layout=layout)
    check_clean()
    ref = streaming.sinks_backward(qf, kf, vf, dof, scale, left, sinks, right)
    bounds = None
    for i, (name, g, r) in enumerate(zip(("dq", "dk", "dv"), grads, ref)):
        err = grad_rel_err(host(g), r)
        if err > TOL_GRAD_RELFRO:  # rows of which little is left: each element by its own bound
            bounds = bounds or rounding_bounds(qf, kf, vf, dof, scale, left, sinks, right)
            assert np.all(np.abs(host(g) - r) <= bounds[i]), (name, err)


def rounding_bounds(q, k, v, do, scale, left, sinks, right):
    """How far roundings alone can move each element of dQ, dK and dV.  With u = 2^-8, half a
    bf16 step relative to a value: the forward rounds P (once in the product, once in its
    normaliser) and O, so |dO| = u |O| + 2 u P |V|; the backward takes D = sum dO * O from that O,
    off by E = sum |dO| (u |O| + 2 u P |V|); dS = P (dP - D) is off by P E, then rounded:
    e = P E + u (|dS| + P E).  Then dQ is off by scale e |K| + u |dQ|, dK by scale e^T |Q| + u |dK|,
    dV (P rounded) by u P^T |dO| + u |dV|.  A quarter more covers products of two roundings and
    the fp32 sums (2^-14 and less).  Where a row sees few keys dP - D is a small difference and
    these bounds pass 2 % of it."""
    u, vis = 2.0 ** -8, streaming.sink_visible(np.arange(q.shape[2]), q.shape[2], left, sinks, right)
    out = [np.zeros_like(x) for x in (q, k, v)]
    full = [np.zeros_like(x) for x in (k, v)]
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            g = oracle.kv_head_of(h, q.shape[1], k.shape[1])
            o, _, p, mag = streaming.masked_head(q[b, h], k[b, g], v[b, g], scale, vis)
            dp = do[b, h] @ v[b, g].T
            ds = p * (dp - np.sum(p * dp, axis=1, keepdims=True))
            pe = p * np.sum(np.abs(do[b, h]) * (u * np.abs(o) + 2 * u * mag), axis=1, keepdims=True)
            e = pe + u * (np.abs(ds) + pe)
            out[0][b, h] = scale * e @ np.abs(k[b, g]) + u * np.abs(scale * ds @ k[b, g])
            out[1][b, g] += scale * e.T @ np.abs(q[b, h])
            out[2][b, g] += u * p.T @ np.abs(do[b, h])
            full[0][b, g] += scale * ds.T @ q[b, h]
            full[1][b, g] += p.T @ do[b, h]
    out[1] += u * np.abs(full[0])
    out[2] += u * np.abs(full[1])
    return [1.25 * x for x in out]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left,sinks", [(64, 4), (0, 1), (200, 130), (127, 128), (129, 300), (5, 100000), (300, 0),
                                        (-1, 7), (100000, 3)])
@pytest.mark.parametrize("N,H,Hk", [(700, 2, 2), (513, 4, 1)])
def test_sinks_match_oracle(N, H, Hk, left, sinks, d):
    check(1, H, Hk, N, d, left, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 255, 257, 385])
def test_sinks_lengths(N, d):
    check(2, 2, 1, N, d, 40, 3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left,right,sinks", [(30, 50, 2), (200, 1, 140), (64, -1, 5), (0, 300, 1)])
def test_sinks_right_bounds(left, right, sinks, d):
    check(1, 2, 2, 600, d, left, sinks, right)


@pytest.mark.parametrize("d", [64, 128])
def test_sinks_token_major_layout(d):
    check(2, 4, 2, 450, d, 100, 6, layout="bnhd")


# Items of a sink tile visit every later query tile: split into parts where few heads
# leave CTAs idle (2 heads: parts of 16 steps; 40 heads: fewer parts a head; 260 items of
# sink tiles: none), and several sink tiles a head.
@pytest.mark.parametrize("B,H,Hk,N,left,sinks", [(1, 2, 2, 8192, 200, 4), (1, 8, 1, 2500, 255, 1),
                                                 (1, 40, 40, 4096, 100, 2), (1, 2, 2, 6000, 130, 513)])
def test_sinks_split_backward(B, H, Hk, N, left, sinks):
    """Against oracle heads; dK and dV the same bits in two runs."""
    import torch
    d = 128
    inp = make_inputs_gqa(B, H, Hk, N, d, seed=N + H, with_grad=True)
    q, k, v, do = (bf16_to_device(x) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits))
    o, lse = api.fwd_sinks(q, k, v, left, sinks)
    dq, dk, dv = api.bwd_sinks(q, k, v, o, do, lse, left, sinks)
    again = api.bwd_sinks(q, k, v, o, do, lse, left, sinks)
    check_clean()
    assert torch.equal(dk.view(torch.int16), again[1].view(torch.int16))
    assert torch.equal(dv.view(torch.int16), again[2].view(torch.int16))
    qf, kf, vf, dof = decoded(inp)
    G, g = H // Hk, Hk - 1  # the last key/value head and its query heads
    hs = slice(g * G, H)
    part = (qf[:, hs], kf[:, g:], vf[:, g:])
    o_ref, lse_ref = streaming.sinks_forward(*part, d ** -0.5, left, sinks)
    assert bf16_out_err(device_bf16_to_f64(o[:, hs]), o_ref) <= TOL_O_MAXABS
    assert max_abs(device_f32_to_f64(lse[:, hs]), lse_ref) <= TOL_LSE_ABS
    ref = streaming.sinks_backward(*part, dof[:, hs], d ** -0.5, left, sinks)
    for name, x, r in zip(("dq", "dk", "dv"), (dq[:, hs], dk[:, g:], dv[:, g:]), ref):
        err = grad_rel_err(device_bf16_to_f64(x), r)
        assert err <= TOL_GRAD_RELFRO, (name, err)


def test_many_sink_items_are_not_split():
    check(5, 52, 52, 300, 128, 100, 4, backward=True)


def test_no_sinks_is_the_window_call():
    """sinks = 0, and a window that covers the sequence, give the window's and the causal call's bits."""
    import torch
    inp = make_inputs_gqa(1, 4, 2, 900, 128, seed=3, with_grad=True)
    q, k, v, do = (bf16_to_device(x) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits))
    for (left, sinks), (o2, lse2), back in (
            ((70, 0), api.fwd_window(q, k, v, 70, 0), lambda o, l: api.bwd_window(q, k, v, o, do, l, 70, 0)),
            ((899, 9), api.fwd(q, k, v, causal=True), lambda o, l: api.bwd(q, k, v, o, do, l, causal=True))):
        o, lse = api.fwd_sinks(q, k, v, left, sinks)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
        g, g2 = api.bwd_sinks(q, k, v, o, do, lse, left, sinks), back(o2, lse2)
        for a, b in zip(g[1:], g2[1:]):  # dQ's summation order is free
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    check_clean()


def test_sinks_debug_build():
    """Coordinates and tensor-memory addresses of the range-checked library stay clear."""
    saved = api._lib
    api._lib = api.load_library(api.DEBUG_LIB_PATH)
    try:
        for d in (64, 128):
            check(1, 4, 2, 777, d, 100, 130)
        check(1, 2, 2, 2900, 128, 130, 4)
    finally:
        api._lib = saved


def test_sinks_gradients_against_differences():
    """Directional differences of the kernel's own forward, in the sum over O * dO."""
    import torch
    B, H, Hk, N, d, left, sinks = 1, 2, 1, 260, 64, 50, 3
    inp = make_inputs_gqa(B, H, Hk, N, d, seed=9, with_grad=True)
    q, k, v, do = (bf16_to_device(x) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits))
    o, lse = api.fwd_sinks(q, k, v, left, sinks)
    grads = api.bwd_sinks(q, k, v, o, do, lse, left, sinks)
    rng = np.random.default_rng(4)
    for i, g in enumerate(grads):
        step = torch.from_numpy(rng.standard_normal(tuple(g.shape))).cuda() * 0.25
        ends, moved = [], []
        for sign in (1, -1):
            args = [q, k, v]
            args[i] = (args[i].double() + sign * step).bfloat16()
            moved.append(args[i].double())
            ends.append((api.fwd_sinks(*args, left, sinks)[0].double() * do.double()).sum())
        # the loss moves by the gradient along what the rounded inputs really moved; the forward
        # rounds O to bf16 (relative 2^-8 an element, independent: 2^-8 of the norms), and the
        # second differences of the softmax stay below a tenth at this step
        along = (g.double() * (moved[0] - moved[1])).sum().item()
        noise = 2.0 ** -8 * 2 * (o.double() * do.double()).norm().item()
        size = g.double().norm().item() * (moved[0] - moved[1]).norm().item()
        assert abs((ends[0] - ends[1]).item() - along) <= noise + 0.1 * max(abs(along), size / np.sqrt(g.numel()) * 4)


def test_sinks_in_a_replayed_graph_and_on_another_stream():
    import torch
    inp = make_inputs_gqa(1, 4, 2, 1500, 128, seed=5, with_grad=True)
    q, k, v, do = (bf16_to_device(x) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits))
    o, lse = torch.empty_like(q), torch.empty((1, 4, 1500), device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(api.bwd_sinks_workspace_bytes(1, 4, 2, 1500, 128, 4), dtype=torch.uint8, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.fwd_sinks(q, k, v, 200, 4, o=o, lse=lse)
        api.bwd_sinks(q, k, v, o, do, lse, 200, 4, dq=dq, dk=dk, dv=dv, workspace=ws)
    for _ in range(2):
        q.copy_(q.flip(2))
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = api.fwd_sinks(q, k, v, 200, 4, stream=side)
        g2 = api.bwd_sinks(q, k, v, o2, do, lse2, 200, 4, stream=side)
        side.synchronize()
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
        assert torch.equal(dk.view(torch.int16), g2[1].view(torch.int16))
        assert torch.equal(dv.view(torch.int16), g2[2].view(torch.int16))
        assert rel_fro(device_bf16_to_f64(dq), device_bf16_to_f64(g2[0])) <= 1e-3
    check_clean()


def test_sinks_refusals():
    import torch
    q, k = (torch.zeros(1, h, 64, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    o, lse = api.fwd_sinks(q, k, k, 10, 2)
    for args in ((q.float(), k, k), (q, k, k[:, :, :32]), (q, k[:, :, :32], k[:, :, :32]), (q.cpu(), k, k),
                 (q[..., :32], k[..., :32], k[..., :32]), (q[:, :3], k, k)):
        with pytest.raises((ValueError, api.AttnError)):
            api.fwd_sinks(*args, 10, 2)
    for left, sinks, right in ((-2, 1, 0), (10, -1, 0), (10, 1, -2)):
        with pytest.raises((ValueError, api.AttnError)):
            api.fwd_sinks(q, k, k, left, sinks, right)
        with pytest.raises((ValueError, api.AttnError)):
            api.bwd_sinks(q, k, k, o, q, lse, left, sinks, right)
    with pytest.raises(ValueError):
        api.bwd_sinks(q, k, k, o, q, lse, 10, 2, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        api.bwd_sinks(q, k, k, o, q, lse[:, :2], 10, 2)
    check_clean()


@pytest.mark.parametrize("big", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 10 ** 20])
def test_bounds_past_a_c_int(big):
    """A window or a number of sinks beyond every length, whatever its low 32 bits are: the
    causal call, in each call that takes one."""
    import torch
    inp = make_inputs_gqa(1, 2, 2, 300, 64, seed=6, with_grad=True)
    q, k, v, do = (bf16_to_device(x) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits))
    o, lse = api.fwd(q, k, v, causal=True)
    _, dk, dv = api.bwd(q, k, v, o, do, lse, causal=True)
    for o2, lse2 in (api.fwd_sinks(q, k, v, big, 3), api.fwd_window(q, k, v, big, 0),
                     api.fwd_strided(q, k, v, layout="bhnd", window=(big, 0)), api.fwd_sinks(q, k, v, 10, big)):
        # every key a sink: the mask is the causal one, its sums are in another order
        assert (o2.double() - o.double()).abs().max() <= 2.0 ** -7 * o.double().abs().max()
        assert (lse2 - lse).abs().max() <= TOL_LSE_ABS
    for g in (api.bwd_sinks(q, k, v, o, do, lse, big, 3), api.bwd_window(q, k, v, o, do, lse, big, 0),
              api.bwd_strided(q, k, v, o, do, lse, layout="bhnd", window=(big, 0)),
              api.bwd_sinks(q, k, v, o, do, lse, 10, big)):
        assert rel_fro(device_bf16_to_f64(g[1]), device_bf16_to_f64(dk)) <= TOL_GRAD_RELFRO
        assert rel_fro(device_bf16_to_f64(g[2]), device_bf16_to_f64(dv)) <= TOL_GRAD_RELFRO
    check_clean()


@pytest.mark.parametrize("N", [1, 150])
def test_strides_over_one_element_are_not_looked_at(N):
    """One sequence of one head (and of one token): those dimensions may have any stride."""
    import torch
    inp = make_inputs_gqa(1, 1, 1, N, 64, seed=8, with_grad=True)
    dense = [bf16_to_device(x) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits)]
    odd = [x.as_strided(x.shape, (3, 1, 5 if N == 1 else 64, 1)) for x in dense]
    for fwd, bwd in ((lambda q, k, v: api.fwd_sinks(q, k, v, 20, 2), lambda *a: api.bwd_sinks(*a, 20, 2)),
                     (lambda q, k, v: api.fwd_strided(q, k, v, layout="bhnd", window=(20, 0)),
                      lambda *a: api.bwd_strided(*a, layout="bhnd", window=(20, 0)))):
        o, lse = fwd(*dense[:3])
        g = bwd(*dense[:3], o, dense[3], lse)
        o2, lse2 = fwd(*odd[:3])
        g2 = bwd(*odd[:3], o2, odd[3], lse2)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])
    check_clean()


@pytest.mark.parametrize("B,H,Hk,N,left,sinks", [(1, 2, 2, 8192, 200, 4), (1, 8, 1, 2500, 255, 1),
                                                 (1, 40, 40, 4096, 100, 2), (1, 2, 2, 6000, 130, 513)])
def test_sinks_split_backward_of_narrow_heads(B, H, Hk, N, left, sinks):
    """test_sinks_split_backward at d = 64, whose launch is another: a CTA a part, the last ones
    first, parts that begin in the middle of a query head (test_sink_parts.py says that these
    shapes are split).  Every key/value head's dK and dV the same bits in three runs."""
    import torch
    d = 64
    inp = make_inputs_gqa(B, H, Hk, N, d, seed=N + H, with_grad=True)
    q, k, v, do = (bf16_to_device(x) for x in (inp.q_bits, inp.k_bits, inp.v_bits, inp.do_bits))
    o, lse = api.fwd_sinks(q, k, v, left, sinks)
    dq, dk, dv = api.bwd_sinks(q, k, v, o, do, lse, left, sinks)
    for _ in range(2):
        again = api.bwd_sinks(q, k, v, o, do, lse, left, sinks)
        assert torch.equal(dk.view(torch.int16), again[1].view(torch.int16))
        assert torch.equal(dv.view(torch.int16), again[2].view(torch.int16))
    check_clean()
    qf, kf, vf, dof = decoded(inp)
    G = H // Hk
    for g in {0, Hk - 1}:  # the first and last key/value head and their query heads
        hs, ks = slice(g * G, g * G + G), slice(g, g + 1)
        part = (qf[:, hs], kf[:, ks], vf[:, ks])
        o_ref, lse_ref = streaming.sinks_forward(*part, d ** -0.5, left, sinks)
        assert bf16_out_err(device_bf16_to_f64(o[:, hs]), o_ref) <= TOL_O_MAXABS
        assert max_abs(device_f32_to_f64(lse[:, hs]), lse_ref) <= TOL_LSE_ABS
        ref = streaming.sinks_backward(*part, dof[:, hs], d ** -0.5, left, sinks)
        for name, x, r in zip(("dq", "dk", "dv"), (dq[:, hs], dk[:, ks], dv[:, ks]), ref):
            err = grad_rel_err(device_bf16_to_f64(x), r)
            assert err <= TOL_GRAD_RELFRO, (name, err)


def test_many_sink_items_of_narrow_heads_are_not_split():
    check(5, 52, 52, 300, 64, 100, 4, backward=True)
