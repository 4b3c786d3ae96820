"""The oracle of rotary positions and head norms against closed forms and differences, and the
frequency tables, on the CPU."""

import math
from fractions import Fraction

import numpy as np
import pytest

from exact_attention_52_gb300 import api
from oracle import rope


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_rotation_is_a_complex_factor(interleaved):
    rng = np.random.default_rng(0)
    x, theta, pos = rng.standard_normal((2, 3, 5, 64)), rng.uniform(0, 3, 16), rng.integers(-9, 1000, (2, 5))
    a = rope.angles(pos, theta)[:, None]
    y = rope.turn(x, a, 1.5, 32, interleaved)
    p1, p2 = rope.pairs(32, interleaved)
    z = (x[..., p1] + 1j * x[..., p2]) * 1.5 * np.exp(1j * pos[:, None, :, None] * theta)
    assert np.allclose(y[..., p1], z.real, atol=1e-11) and np.allclose(y[..., p2], z.imag, atol=1e-11)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    # scores depend on the distance of positions alone
    k = rng.standard_normal((1, 1, 1, 32))
    at = lambda v, p: rope.turn(v, rope.angles(p, theta), 1.0, 32, interleaved).ravel()
    assert np.isclose(at(x[:1, :1, :1, :32], 70) @ at(k, 50), at(x[:1, :1, :1, :32], 1020) @ at(k, 1000))


def test_far_positions_keep_their_angles():
    theta, pos = [1.0, 10000.0 ** -0.5, 3e-5], 2 ** 31 - 1
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    for t, a in zip(theta, rope.angles(pos, theta)):
        exact = Fraction(t) * pos / (2 * pi)
        exact = float((exact - round(exact)) * 2 * pi)
        assert abs(a - exact) < 2.0 ** -30


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_are_the_differences(interleaved, norm):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 2, 3, 16)), rng.standard_normal((2, 2, 3, 16))
    a = rope.angles(np.arange(3), rng.uniform(0, 2, 4))[None, None]
    w = rng.uniform(0.5, 2, 16) if norm else None
    f = lambda x, w: np.sum(dy * rope.forward(x, a, 1.25, 8, interleaved, w, 1e-3)[0])
    dx, dw, _, _ = rope.backward(dy, a, 1.25, 8, interleaved, x, w, 1e-3)
    h = 1e-5
    for at in ((0, 1, 2, 0), (1, 0, 0, 5), (1, 1, 1, 15), (0, 0, 1, 4)):
        e = np.zeros_like(x)
        e[at] = h
        assert math.isclose((f(x + e, w) - f(x - e, w)) / (2 * h), dx[at], rel_tol=1e-6, abs_tol=1e-8)
    for i in range(16) if norm else ():
        e = np.zeros(16)
        e[i] = h
        assert math.isclose((f(x, w + e) - f(x, w - e)) / (2 * h), dw[i], rel_tol=1e-6, abs_tol=1e-8)


def test_frequencies():
    plain, one = api.rope_frequencies(128, 10000.0)
    assert one == 1.0 and plain[0] == 1.0 and math.isclose(plain[63], 10000.0 ** (-126 / 128))
    linear, one = api.rope_frequencies(128, 10000.0, "linear", 4.0)
    assert one == 1.0 and all(math.isclose(4 * x, y) for x, y in zip(linear, plain))
    ntk, one = api.rope_frequencies(128, 10000.0, "ntk", 4.0)  # fastest as it was, slowest by the factor
    assert one == 1.0 and ntk[0] == 1.0 and math.isclose(4 * ntk[63], plain[63], rel_tol=1e-12)
    yarn, m = api.rope_frequencies(128, 10000.0, "yarn", 4.0, 4096)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1.0)
    for x, y in zip(yarn, plain):
        turns = 4096 * y / (2 * math.pi)
        want = y if turns > 32 else y / 4 if turns < 1 else y * ((turns - 1) / 31 * 0.75 + 0.25)
        assert math.isclose(x, want, rel_tol=1e-12)
    assert api.rope_frequencies(64, scaling=None, factor=7.0) == api.rope_frequencies(64)


def test_the_table_holds_turns():
    torch = pytest.importorskip("torch")
    theta = [1.0, 0.5, 1e-5, 0.0, -0.25, 6.5, 2 * math.pi, 1e300]
    t = api.rope_table(16, frequencies=theta, interleaved=True, magnitude=1.5, device="cpu")
    assert (t.rot, t.interleaved, t.magnitude, t.turns.dtype, tuple(t.turns.shape)) == (16, True, 1.5, torch.int64, (8,))
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    for n, th in zip(t.turns.tolist(), theta[:7]):
        off = (Fraction(n, 2 ** 64) - Fraction(th) / (2 * pi)) % 1
        assert min(off, 1 - off) <= Fraction(1, 2 ** 65)
    d = api.rope_table(32, base=500000.0, scaling="yarn", factor=8.0, original_len=8192, device="cpu")
    assert d.rot == 32 and math.isclose(d.magnitude, 0.1 * math.log(8.0) + 1.0) and not d.interleaved


@pytest.mark.parametrize("args", [
    dict(rot=24), dict(rot=0), dict(rot=-16), dict(rot=16.0), dict(rot=16, scaling="sqrt"), dict(rot=16, base=0.0),
    dict(rot=16, base=float("inf")), dict(rot=16, scaling="linear", factor=0.0), dict(rot=16, scaling="yarn", factor=2.0),
    dict(rot=16, scaling="yarn", factor=2.0, original_len=10, beta_fast=1.0), dict(rot=16, frequencies=[1.0] * 7),
    dict(rot=16, frequencies=[float("nan")] * 8), dict(rot=16, magnitude=float("inf"))])
def test_tables_that_are_refused(args):
    pytest.importorskip("torch")
    with pytest.raises(ValueError):
        api.rope_table(device="cpu", **args)
