"""Microscaled 4-bit storage (E2M1 elements, one power-of-two factor per 32 columns), products
with it and the routed expert layer, from their definitions in 64 bits.

The element rounding is a search over the eight magnitudes, so it shares nothing with a
hardware conversion.  Parity unpinned beyond the hand-derived rounding cases of the tests.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest_code(a: np.ndarray) -> np.ndarray:
    """Magnitude code nearest to a >= 0 (ties to the even code, 7 above the top)."""
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    even_first = np.where(d == best, np.arange(8) % 2, 2)
    return even_first.argmin(-1)


def _pad(w, fill=0.0):
    rows, cols = w.shape
    g = -(-cols // BLOCK)
    p = np.full((rows, g * BLOCK), fill, np.float64)
    p[:, :cols] = w
    return p.reshape(rows, g, BLOCK)


def factor(e):
    return np.where(np.asarray(e) == 255, np.nan, np.ldexp(1.0, np.asarray(e, np.int64) - 127))


def quantize(w, rule="floor", colw=None):
    """(codes [rows x 16 G] u8, scales [rows x G] u8) of a float32-valued matrix."""
    w = np.asarray(w, np.float32).astype(np.float64)
    rows, cols = w.shape
    b = _pad(w)
    finite = np.isfinite(b).all(2)
    b = np.where(finite[..., None], b, 0.0)
    top = np.abs(b).max(2)
    _, ex = np.frexp(np.where(top > 0, top, 1.0))     # top = m 2^ex, 1/2 <= m < 1
    e = np.where(top > 0, np.maximum(ex - 1 - 2 + 127, 0), 0)
    q = nearest_code(np.abs(b) / factor(e)[..., None])
    if rule == "least":
        h = _pad(np.ones((1, cols)) if colw is None else np.asarray(colw, np.float64)[None])
        up = nearest_code(np.abs(b) / factor(e + 1)[..., None])
        err = [((np.abs(b) - MAGNITUDES[c] * factor(s)[..., None]) ** 2 * h).sum(2)
               for c, s in ((q, e), (up, e + 1))]
        # 4 x 2^126 = 2^128 is no fp32 number: a block that would round there keeps E
        finite_up = (MAGNITUDES[up] * factor(e + 1)[..., None] <= np.finfo(np.float32).max).all(2)
        better = (err[1] < err[0]) & finite_up
        e, q = np.where(better, e + 1, e), np.where(better[..., None], up, q)
    code = q + 8 * np.signbit(b)
    code = np.where(finite[..., None], code, 0)
    inside = (np.arange(b.shape[1] * BLOCK) < cols).reshape(1, -1, BLOCK)
    code = np.where(inside, code, 0).reshape(rows, -1).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(finite, e, 255).astype(np.uint8)


def elements(codes, cols):
    """Signed element values (without the factor) [... x cols]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)[..., :cols]
    return MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)


def values(codes, scales, cols):
    return elements(codes, cols) * np.repeat(factor(scales), BLOCK, -1)[..., :cols]


def route(x, router, top_k, renorm):
    """(experts by descending logit, ties to the lower index; their weights)."""
    logits = np.asarray(x, np.float64) @ np.asarray(router, np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    p = np.exp(logits - logits.max(1, keepdims=True))
    w = np.take_along_axis(p, ids, 1)
    return ids, w / (w if renorm else p).sum(1, keepdims=True)


def moe(x, router, gate_up, down, top_k, renorm):
    """y, ids, weights; gate_up [E x 2f x d] and down [E x d x f] as values."""
    x = np.asarray(x, np.float64)
    ids, w = route(x, router, top_k, renorm)
    f = gate_up.shape[1] // 2
    y = np.zeros((x.shape[0], down.shape[1]))
    for t in range(x.shape[0]):
        for r, e in enumerate(ids[t]):
            g, u = gate_up[e, :f] @ x[t], gate_up[e, f:] @ x[t]
            y[t] += w[t, r] * (down[e] @ (g / (1 + np.exp(-g)) * u))
    return y, ids, w
