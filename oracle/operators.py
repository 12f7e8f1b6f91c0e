"""CPU references of the gradients and the 4-bit operators -- TEST INFRASTRUCTURE ONLY.

Binary64, one expert at a time, written from the formulas; nothing here uses the
HIP library. bf16 arrays are bit patterns (uint16), as in ``oracle``.

* ``dgrad``: dA[r] = dC[r] @ B[e].T, and the sum of magnitudes of its terms.
* ``wgrad``: dB[e] = A_e.T @ dC_e, and the sum of magnitudes of its terms.
* ``swiglu_grad``: with H = silu(gate) * up on interleaved columns and dH given,
  the gradient of the columns and H itself; ``swiglu_grad_error`` bounds what a
  binary32 evaluation with exp2 and reciprocal of one ulp may be off by.
* ``mx4_encode`` / ``mx4_values``: blocks of 32 values to E2M1 codes and E8M0
  scale bytes by the format's rule, and back.
* ``mx4_product``: the grouped product of the decoded values.
"""

from __future__ import annotations

import numpy as np

from oracle import _bf16_to_f64

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _spans(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def dgrad(dC, B, offsets):
    """(dA, S) [M, K] for dC [M, N] bits, B [E, K, N] bits; rows outside every group are NaN."""
    d = _bf16_to_f64(dC)
    out = np.full((d.shape[0], B.shape[1]), np.nan)
    S = out.copy()
    for e, lo, hi in _spans(offsets):
        b = _bf16_to_f64(B[e]).T
        out[lo:hi] = d[lo:hi] @ b
        S[lo:hi] = np.abs(d[lo:hi]) @ np.abs(b)
    return out, S


def wgrad(A, dC, offsets):
    """(dB, S) [E, K, N] for A [M, K] bits, dC [M, N] bits."""
    a, d = _bf16_to_f64(A), _bf16_to_f64(dC)
    out = np.zeros((len(offsets) - 1, a.shape[1], d.shape[1]))
    S = out.copy()
    for e, lo, hi in _spans(offsets):
        out[e] = a[lo:hi].T @ d[lo:hi]
        S[e] = np.abs(a[lo:hi]).T @ np.abs(d[lo:hi])
    return out, S


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu_grad(dH, C):
    """(dC, H) for dH [M, I] and interleaved gate / up columns C [M, 2I] (binary64)."""
    g, u = C[:, 0::2], C[:, 1::2]
    s = _sigmoid(g)
    d = np.empty_like(C)
    d[:, 0::2] = dH * u * s * (1.0 + g * (1.0 - s))
    d[:, 1::2] = dH * g * s
    return d, g * s * u


def swiglu_grad_error(dH, dH_err, C):
    """Bounds (on dC, on H) of an fp32 evaluation from a dH that is off by dH_err.

    With u = 2^-23 (one ulp): sigmoid is off by at most (|g| + 3) u relative
    (the rounded exponent |g| log2(e) moves e^-g by |g| u, exp2, the sum and
    the reciprocal add one ulp at most each). 1 - s then is off by s (|g| + 3) u
    + u, so t = 1 + g (1 - s) by |g| (s (|g| + 3) + 1) u and two roundings of
    numbers up to 1 + |g|. The products add at most one ulp each. Twice the sum
    of the first-order terms covers the higher ones. Where s is below
    2^-126 it is 0 instead: 2^-100 of everything it multiplies.
    """
    u = 2.0 ** -23
    g, up = np.abs(C[:, 0::2]), np.abs(C[:, 1::2])
    s = _sigmoid(C[:, 0::2])
    t = np.abs(1.0 + C[:, 0::2] * (1.0 - s))
    rel_s = (g + 3.0) * u
    t_err = g * (s * (g + 3.0) + 1.0) * u + 2.0 * (1.0 + g) * u
    h = np.abs(dH)
    tiny = 2.0 ** -100 * (1.0 + g)
    err = np.empty_like(C)
    err[:, 0::2] = up * (dH_err * s * t + h * (s * t * (rel_s + 4.0 * u) + s * t_err)) + tiny * h * up
    err[:, 1::2] = g * s * (dH_err + h * (rel_s + 3.0 * u)) + tiny * h
    return 2.0 * err, 2.0 * g * s * up * (rel_s + 3.0 * u) + 2.0 * tiny * up


def mx4_encode(x):
    """bf16 bits [..., M, K] -> codes [..., M, K/2], scale bytes [..., ceil(K/256), M, 8]."""
    shape = x.shape
    K = shape[-1]
    v = _bf16_to_f64(x).reshape(shape[:-1] + (K // 32, 32))
    neg = (x.reshape(v.shape) >> 15).astype(np.uint8)
    bad = ~np.isfinite(v).all(-1)
    mag = np.abs(np.where(bad[..., None], 0.0, v))
    top = mag.max(-1)
    _, ex = np.frexp(top)                      # top = f * 2^ex, f in [0.5, 1)
    e = np.where(top > 0, np.maximum(ex - 1 - 2, -127), -127)
    y = np.ldexp(mag, -e[..., None])           # exact: powers of two
    # the nearest value; at a border the code that is even
    code = np.zeros(y.shape, dtype=np.uint8)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code[(y > mid) | ((y == mid) & (i % 2 == 1))] = i + 1
    code |= neg << 3
    code[bad] = 0
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    code = code.reshape(shape)
    slices = -(-K // 256)
    padded = np.zeros(shape[:-1] + (8 * slices,), dtype=np.uint8)
    padded[..., : K // 32] = scale
    padded = padded.reshape(shape[:-1] + (slices, 8))
    return code[..., 0::2] | code[..., 1::2] << 4, np.ascontiguousarray(np.swapaxes(padded, -3, -2))


def mx4_values(q, scales):
    """The binary64 values of codes [..., M, K/2] and scale bytes [..., ceil(K/256), M, 8]."""
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[:-1] + (-1,))
    K = code.shape[-1]
    by_row = np.swapaxes(scales, -3, -2)
    by_row = by_row.reshape(by_row.shape[:-2] + (-1,))[..., : K // 32].astype(np.int64)
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    v = np.ldexp(v.reshape(v.shape[:-1] + (K // 32, 32)), (by_row - 127)[..., None])
    v = np.where((by_row == 255)[..., None], np.nan, v)
    return v.reshape(code.shape)


def mx4_product(Aq, a_scale, Bq, b_scale, offsets):
    """(C, S) [M, N]; rows outside every group are NaN."""
    a = mx4_values(Aq, a_scale)
    out = np.full((a.shape[0], Bq.shape[1]), np.nan)
    S = out.copy()
    for e, lo, hi in _spans(offsets):
        b = mx4_values(Bq[e], b_scale[e]).T
        out[lo:hi] = a[lo:hi] @ b
        S[lo:hi] = np.abs(a[lo:hi]) @ np.abs(b)
    return out, S
