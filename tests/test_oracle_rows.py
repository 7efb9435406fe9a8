"""CPU pins of oracle/rows.py: the row operators against brute force, their
gradients against differences, the MXFP4 quantiser against its definition in
exact rational arithmetic, the product against a triple loop."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import formats as F
from oracle import rows as R

GRID = [Fraction(v) for v in (0, 0.5, 1, 1.5, 2, 3, 4, 6)]


def _case(seed, T=5, k=3, H=4):
    g = np.random.default_rng(seed)
    S = T * k
    routed = g.random(S) > 0.3
    pos = np.full(S, -1)
    pos[routed] = g.permutation(int(routed.sum()))
    inv = pos.reshape(T, k)
    return inv, g.normal(size=(T, H)), g.normal(size=(S, H)), g.normal(size=(T, k)), g


@pytest.mark.parametrize("seed", range(4))
def test_permute_and_unpermute_by_brute_force(seed):
    inv, x, rows, w, g = _case(seed)
    T, k = inv.shape
    got = R.permute(x, inv, rows)
    for p in range(T * k):
        owner = [t for t in range(T) for j in range(k) if inv[t, j] == p]
        np.testing.assert_array_equal(got[p], x[owner[0]] if owner else rows[p])
    out = R.unpermute(rows, inv, w)
    for t in range(T):
        want = sum((w[t, j] * rows[inv[t, j]] for j in range(k) if inv[t, j] >= 0), np.zeros(4))
        np.testing.assert_allclose(out[t], want, rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("seed", range(4))
def test_gradients_against_differences(seed):
    """Both operators are (bi)linear: a central difference of <out, g> is exact
    up to rounding."""
    inv, x, rows, w, g = _case(seed)
    dout = g.normal(size=x.shape)
    drows, dw = R.unpermute_backward(dout, rows, inv, w, np.zeros_like(rows))
    h = 0.5
    for p in range(len(rows)):
        for c in range(rows.shape[1]):
            up, dn = rows.copy(), rows.copy()
            up[p, c] += h
            dn[p, c] -= h
            d = ((R.unpermute(up, inv, w) - R.unpermute(dn, inv, w)) * dout).sum() / (2 * h)
            assert abs(d - drows[p, c]) < 1e-12
    for t in range(inv.shape[0]):
        for j in range(inv.shape[1]):
            up, dn = w.copy(), w.copy()
            up[t, j] += h
            dn[t, j] -= h
            d = ((R.unpermute(rows, inv, up) - R.unpermute(rows, inv, dn)) * dout).sum() / (2 * h)
            assert abs(d - dw[t, j]) < 1e-12
    # permute's gradient is the sum with weights 1.
    gr = g.normal(size=rows.shape)
    dx = R.unpermute(gr, inv, np.ones_like(w))
    routed = inv.reshape(-1)[inv.reshape(-1) >= 0]
    mask = np.zeros((len(rows), 1))
    mask[routed] = 1
    for t in range(x.shape[0]):
        for c in range(x.shape[1]):
            up, dn = x.copy(), x.copy()
            up[t, c] += h
            dn[t, c] -= h
            z = np.zeros_like(rows)
            d = ((R.permute(up, inv, z) - R.permute(dn, inv, z)) * gr).sum() / (2 * h)
            assert abs(d - dx[t, c]) < 1e-12


def _rational_block(vals):
    v = [Fraction(float(a)) for a in vals]
    amax = max(abs(a) for a in v)
    n = -127
    while amax > 6 * Fraction(2) ** n:
        n += 1
    codes = []
    for a, raw in zip(v, vals):
        y = abs(a) / Fraction(2) ** n
        best = min(range(8), key=lambda c: (abs(GRID[c] - y), c % 2))
        codes.append(best | (8 if np.signbit(raw) else 0))
    return n, codes


def _hard_blocks():
    g = np.random.default_rng(7)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)
    out = [ties, -ties, np.zeros(32), -np.zeros(32), np.nextafter(ties, 10), np.nextafter(ties, 0)]
    for e in (-149, -140, -133, -127, -126, -125, -40, 0, 60, 125):
        b = np.zeros(32)
        b[3] = 2.0 ** e
        out += [b, 1.5 * b, 1.5 * b * (1 + 2.0 ** -23)]
    for s in (1e-38, 1e-6, 1.0, 1e30):
        out.append(g.normal(size=32) * s)
    return [np.float32(b).astype(np.float64) for b in out]


@pytest.mark.parametrize("i", range(len(_hard_blocks())))
def test_quantiser_against_its_definition(i):
    b = _hard_blocks()[i]
    codes, scales = R.quantize_mxfp4(b[None])
    n, want = _rational_block(b)
    assert scales[0, 0] == n + 127
    np.testing.assert_array_equal(F.unpack_e2m1_pairs(codes)[0], want)
    # and back
    got = R.dequantize_mxfp4(codes, scales)[0]
    val = [float((-1 if c & 8 else 1) * GRID[c & 7] * Fraction(2) ** n) for c in want]
    np.testing.assert_array_equal(got, val)


def test_quantiser_of_blocks_that_are_not_finite():
    x = np.ones((3, 96))
    x[0, 40] = np.nan
    x[1, 0] = np.inf
    x[2, 95] = -np.inf
    codes, scales = R.quantize_mxfp4(x)
    np.testing.assert_array_equal(scales == 255, [[False, True, False], [True, False, False],
                                                  [False, False, True]])
    v = R.dequantize_mxfp4(codes, scales)
    assert np.isnan(v[0, 32:64]).all() and np.isfinite(v[0, :32]).all()


def test_quantiser_equals_the_input_recipe():
    """Above the recipe's floor (amax 1e-4) the rule is the one the layer's MXFP4
    weights are made by."""
    import torch

    from workloads.synth import _quant_e2m1_rows
    g = np.random.default_rng(3)
    x = np.float32(g.normal(size=(64, 256)) * 0.02)
    c, s = _quant_e2m1_rows(torch.from_numpy(x))
    codes, scales = R.quantize_mxfp4(x.astype(np.float64))
    np.testing.assert_array_equal(codes, c.numpy())
    np.testing.assert_array_equal(scales, s.numpy())


def test_group_major_layout():
    s = np.arange(3 * 5, dtype=np.uint8).reshape(3, 5)
    g = R.group_major(s)
    assert g.shape == (2, 3, 4)
    for r in range(3):
        for b in range(8):
            assert g[b // 4, r, b % 4] == (s[r, b] if b < 5 else 0)


def test_grouped_product_by_triple_loop():
    g = np.random.default_rng(5)
    a, w = g.normal(size=(7, 6)), g.normal(size=(3, 4, 6))
    out = R.grouped_product(a, w, [0, 2, 2, 6], np.full((7, 4), 9.0))
    for r in range(7):
        e = 0 if r < 2 else 2 if r < 6 else None
        for n in range(4):
            want = 9.0 if e is None else sum(a[r, c] * w[e, n, c] for c in range(6))
            assert abs(out[r, n] - want) < 1e-13
    # Offsets that run backwards or out of range cover nothing twice.
    out = R.grouped_product(a, w, [3, -4, 99, 5], np.zeros((7, 4)))
    np.testing.assert_allclose(out[:3], 0)
    np.testing.assert_allclose(out[3:], a[3:] @ w[1].T)
