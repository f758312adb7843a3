"""8-bit integer rows (one fp32 scale each), products with them, routing, and the routed expert layer,
from their definitions in 64 bits.

Parity unpinned beyond the hand-derived cases of the tests.
"""
from __future__ import annotations

import numpy as np


def pitch(cols):
    return -(-cols // 128) * 128


def padded(codes):
    out = np.zeros((codes.shape[0], pitch(codes.shape[1])), np.int8)
    out[:, :codes.shape[1]] = codes
    return out


def quantize(x, colf=None):
    """(codes [rows x cols] int8, scales [rows] float32) of a float32-valued matrix."""
    v = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if colf is not None:
            v = v * np.asarray(colf, np.float32)
        s = np.abs(v).max(1) * (np.float32(1) / np.float32(127))
        # 24-bit quotients are 2^-25 or more from a half that they do not equal: 64 bits decide
        q = v.astype(np.float64) / s.astype(np.float64)[:, None]
    finite = np.isfinite(v).all(1)
    q = np.where((finite & (s > 0))[:, None], np.clip(np.rint(q), -127, 127), 0)
    return q.astype(np.int8), np.where(finite, s, np.float32(np.nan)).astype(np.float32)


def levels(codes, zeros=None):
    """Whole numbers that a row's scale is multiplied by."""
    c = codes.astype(np.int64)
    return c if zeros is None else c + 128 - zeros.astype(np.int64)[..., None]


def product(xcodes, xscales, codes, scales, zeros=None, bias=None):
    y = (xcodes.astype(np.float64) @ levels(codes, zeros).astype(np.float64).T)
    y = y * xscales.astype(np.float64)[:, None] * scales.astype(np.float64)
    return y if bias is None else y + bias


def route(logits, top_k, scores="softmax", bias=None, groups=1, top_groups=1, group_best=1, renorm=True,
          scale=1.0):
    """(ids [n x k], weights [n x k] float64), one token and one expert at a time."""
    n, E = logits.shape
    size = E // groups
    sigmoid = lambda v: 1.0 / (1.0 + np.exp(-v)) if v > -700 else np.exp(v)  # noqa: E731
    ids, weights = np.zeros((n, top_k), np.int32), np.zeros((n, top_k))
    for t in range(n):
        x = [float(v) for v in logits[t]]
        held = [v > -np.inf for v in x]          # False for NaN too
        if scores == "sigmoid":
            score = [sigmoid(v) if h else 0.0 for v, h in zip(x, held)]
        else:
            top = max([v for v, h in zip(x, held) if h], default=0.0)
            e = [0.0 if not h else 1.0 if v == top else np.exp(v - top) for v, h in zip(x, held)]
            total = sum(e)
            score = [v / total if total > 0 else 0.0 for v in e]
        choice = []
        for e in range(E):
            c = score[e] + (0.0 if bias is None else float(bias[e]))
            choice.append(c if held[e] and c == c else -np.inf)
        value = []
        for g in range(groups):
            best = sorted((c for c in choice[g * size:(g + 1) * size] if c > -np.inf), reverse=True)[:group_best]
            value.append(sum(best) if best else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        order = sorted((e for e in range(E) if e // size in kept), key=lambda e: (-choice[e], e))[:top_k]
        w = np.array([score[e] for e in order])
        if renorm:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t], weights[t] = order, w * scale
    return ids, weights


def gated(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def moe(x, ids, weights, gu, dn, f):
    """(y, slack): the layer in 64 bits, and how far y moves where a hidden code next to a half rounds
    the other way.  gu, dn: (codes [E x rows x cols], scales, zeros or None).

    h in fp32 is off by less than (24 + 4 |g|) 2^-24 of itself: three roundings in each of g and u
    (silu multiplies g's by at most 1 + |g|), a few last bits of the exponential, the quotient and the
    product; the row's largest the same, so a quotient of at most 127 is off by twice that."""
    n, k = ids.shape
    E = gu[0].shape[0]
    qx, sx = quantize(x)
    pick = lambda m, e: (m[0][e], m[1][e], None if m[2] is None else m[2][e])  # noqa: E731
    y, slack = np.zeros((n, dn[0].shape[1])), np.zeros((n, dn[0].shape[1]))
    for e in range(E):
        t, r = np.nonzero(ids == e)
        if not len(t):
            continue
        v = product(qx[t], sx[t], *pick(gu, e))
        g, u = v[:, :f], v[:, f:]
        h = gated(g, u)
        s = np.abs(h).max(1, keepdims=True) / 127
        q = np.divide(h, s, out=np.zeros_like(h), where=s > 0)
        code = np.clip(np.rint(q), -127, 127)
        off = 2 * (24 + 4 * np.abs(g).max(1, keepdims=True)) * 2.0 ** -24 * np.abs(q)
        near = np.abs(np.abs(q - np.trunc(q)) - 0.5) <= off
        w = weights[t, r].astype(np.float64)[:, None]
        c, ws, z = pick(dn, e)
        level = levels(c, z).astype(np.float64).T
        main = code @ level
        np.add.at(y, t, w * ws * s * main)
        np.add.at(slack, t, np.abs(w) * ws * s * (near @ np.abs(level)
                                                  + (off.max(1, keepdims=True) / 127 + 2.0 ** -20) * np.abs(main)))
    return y, slack
