"""fp64 CPU oracle of rotary positions and head norms.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  With w the weight (None: no norm),
  n = x r w,  r = (mean_i x_i^2 + eps)^(-1/2)   (n = x without a weight),
and the first rot elements of n turned in pairs by a = position * theta_i,
  y1 = f (n1 cos a - n2 sin a),  y2 = f (n2 cos a + n1 sin a);
pairs are elements (i, i + rot/2), or (2i, 2i + 1) where interleaved.  Angles are reduced in
extended precision, so that positions near 2^31 keep 2^-30 radians.
"""

from __future__ import annotations

import numpy as np

TWO_PI = 2 * np.longdouble("3.14159265358979323846264338327950288419716939937510582")


def angles(positions, theta):
    """[..., rot/2] angles of integer positions, within a turn."""
    a = np.asarray(positions)[..., None].astype(np.longdouble) * np.asarray(theta, dtype=np.longdouble)
    return (a - TWO_PI * np.rint(a / TWO_PI)).astype(np.float64)


def pairs(rot, interleaved):
    """Indices of the first and second elements of the pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, a, f, rot, interleaved):
    """x [..., d] with its pairs turned by a [..., rot/2]."""
    p1, p2 = pairs(rot, interleaved)
    y = np.array(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        y[..., p1] = f * (x[..., p1] * np.cos(a) - x[..., p2] * np.sin(a))
        y[..., p2] = f * (x[..., p2] * np.cos(a) + x[..., p1] * np.sin(a))
    return y


def reach(x, f, rot, interleaved):
    """f (|x1| + |x2|) at both elements of a pair, |x| elsewhere: what a rounding error of the
    rotation is relative to."""
    p1, p2 = pairs(rot, interleaved)
    y = np.abs(x)
    y[..., p1] = y[..., p2] = abs(f) * (np.abs(x[..., p1]) + np.abs(x[..., p2]))
    return y


def rnorm(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def forward(x, a, f, rot, interleaved, w=None, eps=1e-6):
    """x [B, heads, N, d], a [B or 1, 1, N, rot/2]; (y, what its errors are relative to)."""
    n = x if w is None else x * rnorm(x, eps) * w
    return turn(n, a, f, rot, interleaved), reach(n, f, rot, interleaved)


def backward(dy, a, f, rot, interleaved, x=None, w=None, eps=1e-6):
    """(dx, dw or None, what dx's errors are relative to, what dw's are)."""
    dn, size = turn(dy, -a, f, rot, interleaved), reach(dy, f, rot, interleaved)
    if w is None:
        return dn, None, size, None
    d, r = x.shape[-1], rnorm(x, eps)
    u = x * r
    g = dn * w
    dx = r * (g - u * np.mean(g * u, axis=-1, keepdims=True))
    big = size * np.abs(w)
    dx_size = r * (big + np.abs(u) * np.mean(big * np.abs(u), axis=-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, np.sum(dn * u, axis=axes), dx_size, np.sum(size * np.abs(u), axis=axes)
