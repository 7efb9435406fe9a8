"""The row operators and the MXFP4 operators in float64, straight from their
formulas (TEST INFRASTRUCTURE ONLY, see the package docstring).

  permute:    rows[inv[t, j]] = x[t]            (rows no slot names keep `rows`)
  unpermute:  out[t] = sum_j w[t, j] * rows[inv[t, j]]
  gradients:  dx[t] = sum_j drows[inv[t, j]]; drows[inv[t, j]] = w[t, j] * dout[t];
              dw[t, j] = <dout[t], rows[inv[t, j]]>
  quantise:   per 32 elements, n = the smallest integer >= -127 with
              amax <= 6 * 2^n; E2M1 of x / 2^n to nearest, ties to even
  product:    out[r] = a[r] @ w[e]^T for offsets[e] <= r < offsets[e + 1]

Parity: pinned by brute force, by differences (the gradients) and by exact
rational arithmetic (the quantiser) in tests/test_oracle_rows.py.
"""
import numpy as np

from .formats import decode_e2m1, decode_ue8m0, unpack_e2m1_pairs


def slots(inv, S):
    """(t, j, position) of every routed slot, t then j ascending."""
    T, k = inv.shape
    return [(t, j, int(inv[t, j])) for t in range(T) for j in range(k) if 0 <= inv[t, j] < S]


def permute(x, inv, rows):
    out = np.array(rows)
    for t, _, p in slots(inv, len(out)):
        out[p] = x[t]
    return out


def unpermute(rows, inv, w):
    rows, w = np.asarray(rows, np.float64), np.asarray(w, np.float64)
    out = np.zeros((inv.shape[0], rows.shape[1]))
    for t, j, p in slots(inv, len(rows)):
        out[t] += w[t, j] * rows[p]
    return out


def unpermute_backward(dout, rows, inv, w, drows):
    """(drows with the routed rows written, dw)."""
    dout, rows = np.asarray(dout, np.float64), np.asarray(rows, np.float64)
    drows = np.array(drows, np.float64)
    dw = np.zeros(inv.shape)
    for t, j, p in slots(inv, len(rows)):
        drows[p] = np.float64(w[t, j]) * dout[t]
        dw[t, j] = dout[t] @ rows[p]
    return drows, dw


def quantize_mxfp4(x):
    """x [R, K] -> (packed codes u8 [R, K/2], scale bytes u8 [R, K/32])."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    m, e = np.frexp(amax)                        # amax = m * 2^e, m in [0.5, 1)
    n = np.where(m <= 0.75, e - 3, e - 2)        # 6 = 0.75 * 2^3
    n = np.maximum(np.where(amax == 0, -127, n), -127)
    y = np.ldexp(b, -n[:, :, None])
    a = np.abs(y)
    # Spacing of the E2M1 grid: 0.5 below 2, then 1 and 2; rint takes ties to
    # even, which on this grid is the even code.
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    mag = np.rint(a / step) * step
    code = np.searchsorted(np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0]), mag).astype(np.uint8)
    code = np.where(np.signbit(y), code | 8, code).astype(np.uint8)
    code[bad] = 0
    code = code.reshape(R, K)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), \
        np.where(bad, 255, n + 127).astype(np.uint8)


def dequantize_mxfp4(codes, scales):
    """Packed codes [R, K/2] and row-major scale bytes [R, K/32] -> float64."""
    return decode_e2m1(unpack_e2m1_pairs(codes)) * np.repeat(decode_ue8m0(scales), 32, axis=-1)


def group_major(scales):
    """Scale bytes [R, K/32] -> [ceil(K/128), R, 4], 0 past K."""
    R, nb = scales.shape
    g = -(-nb // 4)
    out = np.zeros((R, 4 * g), np.uint8)
    out[:, :nb] = scales
    return np.ascontiguousarray(out.reshape(R, g, 4).transpose(1, 0, 2))


def grouped_product(a, w, offsets, out):
    """a [R, K], w [E, N, K] -> out [R, N] with the rows of every group written."""
    out = np.array(out, np.float64)
    top = 0
    for e in range(len(w)):
        lo = max(top, min(max(int(offsets[e]), 0), len(a)))
        hi = max(lo, min(max(int(offsets[e + 1]), 0), len(a)))
        top = hi
        out[lo:hi] = a[lo:hi] @ w[e].T
    return out
