"""CPU references of what surrounds the experts' products -- TEST INFRASTRUCTURE ONLY.

Binary64, written from the formulas; nothing here uses the HIP library. bf16 arrays
are bit patterns (uint16), as in ``oracle``.

* ``fp8_rows`` / ``fp8_weights``: blocks of 128 (128 x 128) values to E4M3 codes and
  fp32 scales; ``fp8_row_values`` / ``fp8_weight_values``: what they stand for.
* ``fp8_product``: the grouped product of the values, with the sums that bound it.
* ``sort``: a router's choices grouped by expert, one choice after the other.
* ``spread``, ``combine``, ``combine_grad``: rows to their experts and back.
* ``norm`` and ``norm_grad``: the root-mean-square norm and its gradient.
"""

from __future__ import annotations

import numpy as np

from oracle import _bf16_to_f64, decode_e4m3, round_to_bf16

BLOCK, TOP, LEAST = 128, 448.0, 2.0 ** -100
# the finite magnitudes in order: code i stands for GRID[i]
GRID = decode_e4m3(np.arange(0x7F, dtype=np.uint8)).astype(np.float64)


def multiplier(top):
    """448 / top cut to 16 significant bits; NaN where top is not finite."""
    top = np.asarray(top, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        f, e = np.frexp(TOP / np.maximum(top, LEAST))
        m = np.ldexp(np.floor(f * 65536.0), e - 16)
    return np.where(np.isfinite(top), m, np.nan)


def to_e4m3(y):
    """The code nearest to y (binary64), ties to the even code, magnitudes over 448 to 448."""
    y = np.asarray(y, dtype=np.float64)
    mag = np.abs(y)
    hi = np.clip(np.searchsorted(GRID, mag), 1, len(GRID) - 1)
    lo = hi - 1
    mid = (GRID[lo] + GRID[hi]) / 2           # exact
    code = np.where((mag > mid) | ((mag == mid) & (hi % 2 == 0)), hi, lo)
    code = np.where(mag >= TOP, len(GRID) - 1, code)
    return (code | (np.signbit(y) << 7)).astype(np.uint8)


def _encode(x, m):
    """x over blocks whose multipliers are m, already of x's shape: codes (0 where m is NaN)."""
    bad = np.isnan(m)
    with np.errstate(invalid="ignore"):
        return np.where(bad, 0, to_e4m3(np.where(bad, 0.0, x * m))).astype(np.uint8)


def _tops(x, height):
    """Largest magnitudes of blocks height x 128 of x [rows, K] (infinity for an infinity or a NaN)."""
    mag = np.where(np.isfinite(x), np.abs(x), np.inf)
    a = np.maximum.reduceat(mag, np.arange(0, x.shape[1], BLOCK), axis=1)
    return a if height == 1 else np.maximum.reduceat(a, np.arange(0, x.shape[0], height), axis=0)


def _spread_blocks(v, rows, K, height):
    return np.repeat(np.repeat(v, height, axis=0)[:rows], BLOCK, axis=1)[:, :K]


def _blocks(x, height):
    m = multiplier(_tops(x, height))
    with np.errstate(divide="ignore"):
        scale = (1.0 / m).astype(np.float32)
    return _encode(x, _spread_blocks(m, *x.shape, height)), scale


def fp8_rows_of(x):
    """binary64 [M, K] -> codes [M, K], fp32 scales [ceil(K/128), M]."""
    if x.shape[0] == 0:
        return np.zeros(x.shape, np.uint8), np.zeros((-(-x.shape[1] // BLOCK), 0), np.float32)
    q, s = _blocks(x, 1)
    return q, np.ascontiguousarray(s.T)


def fp8_rows(bits):
    return fp8_rows_of(_bf16_to_f64(bits))


def fp8_weights(B, for_grad=False):
    """bf16 bits [E, K, N] -> codes [E, N, K] and scales [E, ceil(N/128), ceil(K/128)], or as they lie."""
    out = []
    for b in B:
        x = _bf16_to_f64(b)
        out.append(_blocks(x if for_grad else np.ascontiguousarray(x.T), BLOCK))
    return np.stack([q for q, _ in out]), np.stack([s for _, s in out])


def _values(q):
    return decode_e4m3(q).astype(np.float64)


def fp8_row_values(q, scales):
    return _values(q) * np.repeat(scales.T.astype(np.float64), BLOCK, axis=1)[:, :q.shape[1]]


def fp8_weight_values(q, scales):
    return np.stack([_values(w) * _spread_blocks(s.astype(np.float64), *w.shape, BLOCK)
                     for w, s in zip(q, scales)])


def fp8_product(Aq, a_scale, Bq, b_scale, offsets, bounds=True):
    """(C, S, G) [M, N]: the product and (with bounds) the sum of its terms' magnitudes and
    that over eight neighbouring terms of the largest one. Rows outside every group are NaN."""
    qa = _values(Aq)
    out = np.full((qa.shape[0], Bq.shape[1]), np.nan)
    S, G = out.copy(), out.copy()
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        out[lo:hi] = S[lo:hi] = G[lo:hi] = 0.0
        for i, k in enumerate(range(0, qa.shape[1], BLOCK)):
            # a block's sum first, then its scales: exact in binary64, whatever the others' scales
            a, b = qa[lo:hi, k:k + BLOCK], _values(Bq[e][:, k:k + BLOCK]).T
            scale = (a_scale[i, lo:hi, None].astype(np.float64)
                     * np.repeat(b_scale[e, :, i].astype(np.float64), BLOCK)[None, :Bq.shape[1]])
            out[lo:hi] += scale * (a @ b)
            if not bounds:
                continue
            S[lo:hi] += np.abs(scale) * (np.abs(a) @ np.abs(b))
            for j in range(0, a.shape[1], 8):
                G[lo:hi] += np.abs(scale) * np.max(np.abs(a[:, j:j + 8, None] * b[None, j:j + 8]), axis=1)
    return out, S, G


def fp8_product_error(S, G, K):
    """What the fp8 matrix cores and fp32 sums may be off by.

    A group of eight loses less than 2^-12 of its largest product for each of the
    other seven. A block's 16 group sums are added with an error of at most one unit
    (2^-23) of the sum of magnitudes each; the two scales' product and the scaled
    addition round once more a block: 18 + ceil(K/128) units in all.
    """
    return 7 * 2.0 ** -12 * G + (18 + -(-K // BLOCK)) * 2.0 ** -23 * S


def sort(experts, E, weights=None):
    """(offsets, rows, pos, row_weights) of choices [T, k]."""
    T, k = experts.shape
    groups = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if 0 <= experts[t, j] < E:
                groups[experts[t, j]].append((t, j))
    offsets = np.zeros(E + 1, np.int32)
    rows = np.full(T * k, -1, np.int32)
    pos = np.full((T, k), -1, np.int32)
    row_w = np.zeros(T * k, np.float32)
    r = 0
    for e in range(E):
        for t, j in groups[e]:
            rows[r], pos[t, j] = t, r
            if weights is not None:
                row_w[r] = weights[t, j]
            r += 1
        offsets[e + 1] = r
    return offsets, rows, pos, row_w


def spread(x, pos, out):
    """out with out[pos[t, j]] = x[t] (any arrays of rows)."""
    out = out.copy()
    for t in range(pos.shape[0]):
        for at in pos[t]:
            if 0 <= at < out.shape[0]:
                out[at] = x[t]
    return out


def combine(y, pos, w):
    """(out, S) [T, N] for rows y [M, N] (binary64) and weights w [T, k]."""
    out = np.zeros((pos.shape[0], y.shape[1]))
    S = out.copy()
    for t in range(pos.shape[0]):
        for j, at in enumerate(pos[t]):
            if 0 <= at < y.shape[0]:
                out[t] += w[t, j] * y[at]
                S[t] += np.abs(w[t, j] * y[at])
    return out, S


def combine_grad(dO, y, pos, w):
    """(dY, dw, Sw): dY [M, N] with NaN in rows that no choice names; Sw the sum of |dO * y|."""
    dY = np.full(y.shape, np.nan)
    dw = np.zeros(pos.shape)
    Sw = np.zeros(pos.shape)
    for t in range(pos.shape[0]):
        for j, at in enumerate(pos[t]):
            if 0 <= at < y.shape[0]:
                dY[at] = w[t, j] * dO[t]
                dw[t, j] = dO[t] @ y[at]
                Sw[t, j] = np.abs(dO[t]) @ np.abs(y[at])
    return dY, dw, Sw


def norm(x, residual, g, eps):
    """(z, y) [T, K] in binary64: z the bf16 sum, y the normalised and weighted z."""
    z = x if residual is None else round_to_bf16((x + residual).astype(np.float32).astype(np.float64))
    r = 1.0 / np.sqrt((z * z).mean(1, keepdims=True) + eps)
    return z, z * r * g


# Sums over a row: each square rounds once, and at most 118 additions follow one
# another on the way to the whole (64 of a lane's values, its wave's 6 steps, and those
# of up to 16 waves, with room); the square root halves the relative error, and the
# mean, the sum with eps, the root, the inverse and the product with z g (which is
# exact in fp32) add one rounding of 2^-24 each.
NORM_REL = (119 / 2 + 5) * 2.0 ** -24


def norm_grad(dy, z, g, d_residual, eps):
    """(dz, dg, dz_err, dg_abs): the gradient, what fp32 may be off by in dz, and the sum
    of the magnitudes of dg's terms."""
    r = 1.0 / np.sqrt((z * z).mean(1, keepdims=True) + eps)
    u = dy * g
    a = r * u
    b = z * r ** 3 * (u * z).mean(1, keepdims=True)
    dz = a - b + (0.0 if d_residual is None else d_residual)
    b_abs = np.abs(z) * r ** 3 * (np.abs(u * z)).mean(1, keepdims=True)
    # r^3 triples r's error, the mean of u z adds a sum of its own (u rounds first)
    err = 2 * (NORM_REL * np.abs(a) + (3 * NORM_REL + 125 * 2.0 ** -24) * b_abs)
    err += 2.0 ** -22 * (np.abs(a) + b_abs + (0.0 if d_residual is None else np.abs(d_residual)))
    terms = dy * z * r
    return dz, terms.sum(0), err, np.abs(terms).sum(0)


# dg: at most 256 additions follow one another (rows of a workgroup, then the
# workgroups' shares), after the error of r and two products.
NORM_DG_REL = NORM_REL + 260 * 2.0 ** -24
