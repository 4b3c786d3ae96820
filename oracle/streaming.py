"""fp64 CPU oracle of streaming attention: sliding window with first tokens that
stay visible (sinks), and a paged key/value cache held as E4M3 codes.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Definitions:

* with ``sinks`` first tokens and window (left, right), key j is visible to
  position p iff j <= p + right (no bound for right < 0) and (left < 0, or
  j >= p - left, or j < sinks);
* cache: token j of sequence b is slot j % page of page table[b][j // page];
  its value is scale[page, head] * decode(code);
* append: the scale of a page is 2^e, the smallest e >= -100 with every finite new
  magnitude <= 448 * 2^e, or the one it has where older tokens are in it and that
  suffices; a code is the E4M3 number nearest to the fp32 quotient value / scale (ties to
  even, saturating), which is exact where the scale is a power of two.
"""

from __future__ import annotations

import math

import numpy as np

from .attention import _E4M3, kv_head_of, softmax_rows



def e4m3_encode(y: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code of each y by search over the table: ties to the even code, beyond
    448 the largest, NaN the NaN code 0x7F."""
    y = np.asarray(y, dtype=np.float64)
    mags = _E4M3[:127]
    a = np.minimum(np.abs(y), 448.0)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - mags[lo], mags[hi] - a
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.signbit(y), code | 0x80, code).astype(np.uint8)
    return np.where(np.isnan(y), np.uint8(0x7F), code)


def append_exponent(amax: float) -> int:
    """Smallest e >= -100 with amax <= 448 * 2^e."""
    e = -100
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def cache_append(k, v, k_pages, v_pages, k_scale, v_scale, table, seq_lens, new_lens):
    """In place on uint8 pages [P, Hk, page, d] and scales [P, Hk]; k, v are fp64 [B, Hk, T, d]."""
    page = k_pages.shape[2]
    for x, pages, scale in ((k, k_pages, k_scale), (v, v_pages, v_scale)):
        for b, (length, m) in enumerate(zip(seq_lens, new_lens)):
            by_page = {}
            for t in range(m):
                pos = length - m + t
                if pos >= 0:
                    by_page.setdefault(pos // page, []).append((pos % page, t))
            for pg, slots in by_page.items():
                pid = table[b][pg]
                for h in range(x.shape[1]):
                    new = np.stack([x[b, h, t] for _, t in slots])
                    fin = np.abs(new[np.isfinite(new)])
                    amax = float(fin.max()) if fin.size else 0.0
                    s = 2.0 ** append_exponent(amax)
                    old = slots[0][0]
                    if old and float(scale[pid, h]) >= 2.0 ** -100 and amax <= 448.0 * float(scale[pid, h]):
                        s = float(scale[pid, h])
                    elif old:
                        ratio = np.float32(float(scale[pid, h]) / s)  # not 1 and no power of two only for a user's scale
                        pages[pid, h, :old] = e4m3_encode(_E4M3[pages[pid, h, :old]].astype(np.float32) * ratio)
                    scale[pid, h] = s
                    for (slot, t), row in zip(slots, new):
                        with np.errstate(invalid="ignore", over="ignore"):
                            pages[pid, h, slot] = e4m3_encode(row.astype(np.float32) / np.float32(s))


def sink_visible(pos: np.ndarray, nk: int, left: int, sinks: int, right: int = 0) -> np.ndarray:
    """Boolean [len(pos), nk]: True where position pos sees key j."""
    j = np.arange(nk)[None, :]
    p = np.asarray(pos)[:, None]
    vis = np.ones((len(pos), nk), dtype=bool) if right < 0 else j <= p + right
    if left >= 0:
        vis = vis & ((j >= p - left) | (j < sinks))
    return vis


def masked_head(q, k, v, scale, vis):
    """One head under a visibility mask; hidden keys take no part, whatever they hold.
    Returns (O, LSE, P, sum_j P_ij |V_j|)."""
    seen = vis.any(axis=0)
    kk, vv = np.where(seen[:, None], k, 0.0), np.where(seen[:, None], v, 0.0)
    with np.errstate(invalid="ignore", over="ignore"):
        p, lse = softmax_rows(np.where(vis, float(scale) * (q @ kk.T), -np.inf))
    if np.isfinite(vv).all():
        return p @ vv, lse, p, p @ np.abs(vv)
    o, mag = np.zeros_like(q), np.zeros_like(q)
    for i in range(len(q)):
        o[i], mag[i] = p[i, vis[i]] @ vv[vis[i]], p[i, vis[i]] @ np.abs(vv[vis[i]])
    return o, lse, p, mag


def cache_forward(q, k_pages, v_pages, k_scale, v_scale, table, seq_lens, q_lens, scale, left=-1, sinks=0):
    """q fp64 [B, H, T, d].  Returns (O, LSE, sum P|V|, there [B, T]): rows behind q_lens are
    not there."""
    B, H, T, d = q.shape
    Hk, page = k_pages.shape[1], k_pages.shape[2]
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, H, T))
    there = np.arange(T)[None, :] < np.asarray(q_lens)[:, None]
    for b, (length, m) in enumerate(zip(seq_lens, q_lens)):
        if m == 0:
            continue
        pos = length - m + np.arange(m)
        vis = sink_visible(pos, length, left, sinks)
        keys = np.flatnonzero(vis.any(axis=0))
        pid = np.asarray(table[b])[keys // page]  # only pages that some query sees
        for h in range(H):
            g = kv_head_of(h, H, Hk)
            k, v = (_E4M3[pages[pid, g, keys % page]] * sc[pid, g].astype(np.float64)[:, None]
                    for pages, sc in ((k_pages, k_scale), (v_pages, v_scale)))
            o[b, h, :m], lse[b, h, :m], _, mag[b, h, :m] = masked_head(
                q[b, h, :m], k, v, scale, vis[:, keys]) if len(keys) else (0.0, math.inf, None, 0.0)
    return o, lse, mag, there


def sinks_forward(q, k, v, scale, left, sinks, right=0):
    """Whole sequences, [B, H, N, d] and [B, Hk, N, d] fp64: (O, LSE)."""
    B, H, N, _ = q.shape
    vis = sink_visible(np.arange(N), N, left, sinks, right)
    o, lse = np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        for h in range(H):
            g = kv_head_of(h, H, k.shape[1])
            o[b, h], lse[b, h], _, _ = masked_head(q[b, h], k[b, g], v[b, g], scale, vis)
    return o, lse


def sinks_backward(q, k, v, do, scale, left, sinks, right=0):
    """Gradients of sum(O * do): (dQ, dK, dV), dK and dV summed over the heads that share them."""
    B, H, N, _ = q.shape
    vis = sink_visible(np.arange(N), N, left, sinks, right)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        for h in range(H):
            g = kv_head_of(h, H, k.shape[1])
            _, _, p, _ = masked_head(q[b, h], k[b, g], v[b, g], scale, vis)
            dp = do[b, h] @ v[b, g].T
            ds = p * (dp - np.sum(p * dp, axis=1, keepdims=True))
            dq[b, h] = scale * (ds @ k[b, g])
            dk[b, g] += scale * (ds.T @ q[b, h])
            dv[b, g] += p.T @ do[b, h]
    return dq, dk, dv
