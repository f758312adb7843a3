"""GPU: the gate of the 8-bit integer expert layer, silu(g) = g / (1 + e^-g), to its last bits.

One column of x and the same row of W for every hidden element, so that gate g, up value u and hidden value
h = silu(g) u of a token are known numbers, and its code is 127.  Results leave in bf16, so a second expert, whose
gate is so large that silu(g) = g, is weighted to take the first one's result away: what is left shows the first
one's error.

In units of 2^-24 of the first result: silu 8 (e^-g 3: the hardware's power of two is a last bit off, and a step behind
it; 1 + e^-g 1; its reciprocal 2, a last bit; a product 1, and for gates beyond 80 one more with fewer before it), u times
it 1, the scale 1, 127 times the scale 1.  The second one's sum is reckoned here in 32 bits, its weighting rounds once.
A silu below 2^-126 (gates below -91) is a multiple of 2^-149: half of that, times u, more."""
import numpy as np
import pytest

from gpu_util import qz, to_dev, to_host
from oracle import i8

pytestmark = pytest.mark.gpu

F32 = np.float32


def _levels(x, code, scale):
    """scale (127 code) sx as the products round it."""
    sx = x * (F32(1) / F32(127))
    return (F32(127 * code) * sx) * F32(scale)


@pytest.mark.parametrize("n,f", [(4, 300), (100, 40), (300, 300), (2500, 520)])
def test_gates_to_the_last_bits(n, f):
    q = qz()
    import torch
    rng = np.random.default_rng(n)
    size = np.where(rng.random(n) < 0.3, 86 + 22 * rng.random(n), np.exp(rng.uniform(np.log(0.03), np.log(88), n)))
    size[:2] = 89, 95
    x = size.astype(F32)
    up = F32(2.0 ** 64 / 127)
    # experts: gates -x, x and 1024 x; up values 2^64 x and, of the last, x
    gate = [(-127, F32(1 / 127)), (127, F32(1 / 127)), (127, F32(1024 / 127))]
    ups = [(127, up), (127, up), (127, F32(1 / 127))]
    gu = np.zeros((3, 2 * f, 128), np.int8)
    gs = np.zeros((3, 2 * f), F32)
    for e in range(3):
        gu[e, :f, 0], gs[e, :f] = gate[e]
        gu[e, f:, 0], gs[e, f:] = ups[e]
    dn = np.zeros((3, 1, i8.pitch(f)), np.int8)
    dn[:, 0, f // 2] = 1
    ids = np.stack([np.where(np.arange(n) % 4 == 3, 1, 0), np.full(n, 2)], 1).astype(np.int32)
    g = np.where(ids[:, 0] == 1, _levels(x, *gate[1]), _levels(x, *gate[0]))
    u = _levels(x, *ups[0])
    assert (_levels(x, *gate[2]) > 20).all()                       # e^-20 < 2^-25
    c = F32(1) / F32(127)
    far = F32(127) * (_levels(x, *gate[2]) * _levels(x, *ups[2]) * c)
    g64 = g.astype(np.float64)
    true = 127 * float(c) * (g64 * np.exp(np.minimum(g64, 0)) / (1 + np.exp(-np.abs(g64)))) * u
    w = np.stack([np.ones(n, F32), (-true / far).astype(F32)], 1)
    want = true + w[:, 1].astype(np.float64) * far
    got = q.qz_i8_moe(to_dev(x[:, None]), to_dev(ids), to_dev(w), to_dev(gu), to_dev(gs), to_dev(dn),
                      to_dev(np.ones((3, 1), F32)))
    got = got.double().cpu().numpy()[:, 0]
    e = 2.0 ** -24 * (1 + 2.0 ** -10) * 12 * np.abs(true) + 2.0 ** -150 * (1 + 2.0 ** -10) * np.abs(u.astype(np.float64)) \
        + 2.0 ** -8 * np.abs(want)
    off = np.abs(got - want)
    e += 2.0 ** -8 * off                                            # what is left is rounded to bf16
    print("largest error over bound:", float((off / e).max()), "at gate", g[np.argmax(off / e)])
    bad = off > e
    assert not bad.any(), [(float(g[i]), got[i], want[i], e[i], true[i]) for i in np.flatnonzero(bad)[:6]]


@pytest.mark.parametrize("n", [1, 30, 500])
def test_rows_of_gates_far_below_zero(n):
    """A hidden row all of whose gates are below -88.7, under large up values, has a scale and codes of its own."""
    q = qz()
    rng = np.random.default_rng(n)
    d, f, E = 64, 96, 2
    x = np.abs(rng.standard_normal((n, d))).astype(F32) + F32(0.1)
    # gates between -100 and -89: all tokens are alike, so that a row's scale makes its gate
    x[:] = x[0]
    xq, sx = i8.quantize(x)
    wg = -rng.integers(90, 128, (E, f, 1)).astype(np.int8) * np.ones((1, 1, d), np.int8)
    wu = rng.integers(-127, 128, (E, f, d)).astype(np.int8)
    total = (wg.astype(np.int64) @ xq[0].astype(np.int64)).astype(np.float64) * sx[0]
    gs = np.empty((E, 2 * f), F32)
    gs[:, :f] = -rng.uniform(89, 100, (E, f)) / total
    gs[:, f:] = 2.0 ** 70
    gu = (np.concatenate([wg, wu], 1), gs, None)
    dn = (rng.integers(-127, 128, (E, d, f)).astype(np.int8), np.ones((E, d), F32), None)
    ids = np.tile(np.array([[0, 1]], np.int32), (n, 1))
    w = np.ones((n, 2), F32)
    y, slack = i8.moe(x, ids, w, gu, dn, f)
    assert np.abs(y).max() > 0
    pad = lambda m: to_dev(i8.padded(m.reshape(-1, m.shape[2])).reshape(E, m.shape[1], -1))  # noqa: E731
    got = q.qz_i8_moe(to_dev(x), to_dev(ids), to_dev(w), pad(gu[0]), to_dev(gu[1]), pad(dn[0]), to_dev(dn[1]))
    got = got.double().cpu().numpy()
    # as for any layer: the halves' window that the oracle leaves for a gate of 100 is 5e-5 of a quotient, and half of
    # 2^-149 times u is 4e-7 of a code where the row's largest silu is about 2e-37
    e = 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(y) + slack * (1 + 2.0 ** -8)
    bad = np.abs(got - y) > e
    print("largest result", np.abs(y).max(), "bound", e.max())
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], y[bad][:4])
