"""The root-mean-square norm in 8 bits, and its gradient, on the GPU against binary64 (needs an MI355X)."""

import numpy as np
import pytest

import oracle
import oracle.layer as ref
import workloads as wl
from tests import operators as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SHAPES = [(1, 16), (1, 6144), (2, 128), (3, 144), (7, 2048), (5, 2064), (33, 1040), (9, 4112), (4, 6160), (3, 8208),
          (2, 16384), (130, 272)]


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _inputs(rng, T, K):
    heat = np.exp(0.8 * rng.standard_normal(K))
    x, res = (wl.f32_to_bf16_bits((rng.standard_normal((T, K)) * heat).astype(np.float32)) for _ in range(2))
    return x, res, wl.f32_to_bf16_bits((1 + 0.2 * rng.standard_normal(K)).astype(np.float32))


def check_fp8(q, scales, y, rel):
    """8 bits of a y that is within `rel` of the given one: a block's multiplier lies between
    those of the ends of its largest value's interval (it is 1 / scale, whose 16 bits the
    rounding of the scale leaves standing), and a code between the codes of the ends of its
    value's interval, as rounding is monotone."""
    T, K = y.shape
    tops = ref._tops(y, 1)
    m = 1.0 / scales.T.astype(np.float64)
    f, e = np.frexp(m)
    m = np.ldexp(np.round(f * 65536), e - 16)
    assert (m >= ref.multiplier(tops * (1 + rel))).all() and (m <= ref.multiplier(tops * (1 - rel))).all()
    assert ((1.0 / m).astype(np.float32) == scales.T).all()
    v = y * ref._spread_blocks(m, T, K, 1)
    ends = [oracle.decode_e4m3(ref.to_e4m3(v * (1 + s * rel))) for s in (-1, 1)]
    got = oracle.decode_e4m3(q)
    assert (got >= np.minimum(*ends)).all() and (got <= np.maximum(*ends)).all()


@pytest.mark.parametrize("T,K", SHAPES)
def test_norm(gg, T, K):
    rng = np.random.default_rng(T * K)
    x, res, g = _inputs(rng, T, K)
    X, R, W = (oracle._bf16_to_f64(a) for a in (x, res, g))
    for residual in (None, R):
        z, y = ref.norm(X, residual, W, 1e-5)
        got = gg.rms_norm_fp8(ops.to_dev(x), ops.to_dev(g), residual=None if residual is None else ops.to_dev(res),
                              eps=1e-5, with_norm=True)
        assert got[0].dtype == torch.float8_e4m3fn
        check_fp8(got[0].view(torch.uint8).cpu().numpy(), ops.host(got[1]), y, ref.NORM_REL)
        if residual is not None:
            assert np.array_equal(ops.host(got[2]), z)
        ops.check_bf16(ops.host(got[-1]), y, ref.NORM_REL * np.abs(y), "norm")
        plain = gg.rms_norm_fp8(ops.to_dev(x), ops.to_dev(g), residual=None if residual is None else ops.to_dev(res),
                                eps=1e-5)
        assert len(plain) == len(got) - 1
        assert torch.equal(plain[0].view(torch.uint8), got[0].view(torch.uint8)) and torch.equal(plain[1], got[1])


def test_norm_of_no_rows(gg):
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    q, s, z, y = gg.rms_norm_fp8(x, w, residual=x, with_norm=True)
    assert q.shape == z.shape == y.shape == (0, 64) and s.shape == (1, 0)
    dz, dg = gg.rms_norm_grad(x, x, w)
    assert dz.shape == (0, 64) and (dg == 0).all()


def test_sum_in_place(gg):
    rng = np.random.default_rng(1)
    x, res, g = _inputs(rng, 21, 400)
    want = gg.rms_norm_fp8(ops.to_dev(x), ops.to_dev(g), residual=ops.to_dev(res))
    for which in (0, 1):
        X, R = ops.to_dev(x), ops.to_dev(res)
        got = gg.rms_norm_fp8(X, ops.to_dev(g), residual=R, out_sum=(X, R)[which])
        assert got[2] is (X, R)[which]
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_rows_of_zeros_and_extremes(gg):
    # zeros (eps > 0: codes 0 at the least scale; eps = 0: NaN), infinities and NaN stay in their rows, and
    # values whose squares leave fp32 give 0 / NaN as the formula in fp32 does
    K = 272
    x = np.zeros((6, K), np.float32)
    rng = np.random.default_rng(2)
    x[1], x[2], x[3] = rng.standard_normal((3, K))
    x[2, 5], x[3, 7] = np.inf, np.nan
    x[4] = 2.0 ** -120
    x[5] = 1.0
    g = np.ones(K, np.float32)
    q, s, y = gg.rms_norm_fp8(ops.to_dev(wl.f32_to_bf16_bits(np.where(np.isnan(x), 0, x))), ops.to_dev(wl.f32_to_bf16_bits(g)),
                              eps=1e-6, with_norm=True)
    bits = ops.to_dev(wl.f32_to_bf16_bits(np.where(np.isfinite(x), x, 0)))
    bits[2, 5], bits[3, 7] = float("inf"), float("nan")
    q, s, y = gg.rms_norm_fp8(bits, ops.to_dev(wl.f32_to_bf16_bits(g)), eps=1e-6, with_norm=True)
    q, s, y = q.view(torch.uint8).cpu().numpy(), ops.host(s), ops.host(y)
    assert (q[0] == 0).all() and (y[0] == 0).all() and (s[:, 0] == np.float32(2.0 ** -100 / 448)).all()
    # an infinity: its row's r is 0, so it is NaN (infinity times 0) and the rest 0 of either sign; a NaN: all NaN
    assert np.isnan(s[0, 2]) and (oracle.decode_e4m3(q[2]) == 0).all() and np.isnan(y[2, 5]) and (np.delete(y[2], 5) == 0).all()
    assert np.isnan(s[:, 3]).all() and (q[3] == 0).all() and np.isnan(y[3]).all()
    assert np.isfinite(s[:, [0, 1, 4, 5]]).all() and np.isfinite(y[[0, 1, 4, 5]]).all()
    check_fp8(q[4:], s[:, 4:], ref.norm(oracle._bf16_to_f64(wl.f32_to_bf16_bits(x[4:])), None, g, 1e-6)[1], ref.NORM_REL)


@pytest.mark.parametrize("T,K", SHAPES + [(3000, 48), (1500, 2064)])
def test_gradient(gg, T, K):
    rng = np.random.default_rng(T * K + 1)
    z, res, g = _inputs(rng, T, K)
    dy = ops.bits(rng, T, K, scale=0.02)
    Z, R, W, D = (oracle._bf16_to_f64(a) for a in (z, res, g, dy))
    for r in (None, R):
        want, dg, err, mags = ref.norm_grad(D, Z, W, r, 1e-5)
        dz, dw = gg.rms_norm_grad(ops.to_dev(dy), ops.to_dev(z), ops.to_dev(g), eps=1e-5,
                                  d_residual=None if r is None else ops.to_dev(res))
        ops.check_bf16(ops.host(dz), want, err, "dz")
        ops.check_f32(ops.host(dw), dg, ref.NORM_DG_REL * mags, "dg")
        again = gg.rms_norm_grad(ops.to_dev(dy), ops.to_dev(z), ops.to_dev(g), eps=1e-5,
                                 d_residual=None if r is None else ops.to_dev(res))
        assert torch.equal(again[0], dz) and torch.equal(again[1], dw)


def test_rows_past_2_to_the_32_bytes(gg):
    T, K = 2 ** 17 + 3, 16384  # 4.3e9 bytes of bf16
    rng = np.random.default_rng(3)
    pick = [0, T // 2, T - 2, T - 1]
    x, res, g = _inputs(rng, len(pick), K)
    X = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    X[pick] = ops.to_dev(x)
    q, s, y = gg.rms_norm_fp8(X, ops.to_dev(g), with_norm=True)
    _, want = ref.norm(oracle._bf16_to_f64(x), None, oracle._bf16_to_f64(g), 1e-6)
    check_fp8(q[pick].view(torch.uint8).cpu().numpy(), ops.host(s[:, pick]), want, ref.NORM_REL)
    ops.check_bf16(ops.host(y[pick]), want, ref.NORM_REL * np.abs(want), "norm")
    del q, s, y
    dY = torch.zeros_like(X)
    dY[pick] = ops.to_dev(res)
    dz, dg = gg.rms_norm_grad(dY, X, ops.to_dev(g))
    w, wg, err, mags = ref.norm_grad(oracle._bf16_to_f64(res), oracle._bf16_to_f64(x), oracle._bf16_to_f64(g), None, 1e-6)
    ops.check_bf16(ops.host(dz[pick]), w, err, "dz")
    ops.check_f32(ops.host(dg), wg, ref.NORM_DG_REL * mags, "dg")


# powers of two that rows lie at: their squares, and the cube of 1 / rms, leave fp32 on both sides
FAR = [-120, -100, -70, -45, -13, 0, 20, 47, 50, 70, 100, 118]


def _far(rng, K, g_powers=(0,)):
    """Rows near 2^FAR and a weight near the given powers of two, column by column."""
    x = rng.standard_normal((len(FAR), K)) * np.exp2(FAR)[:, None]
    g = (1 + 0.2 * rng.standard_normal(K)) * np.exp2(rng.choice(g_powers, K))
    return wl.f32_to_bf16_bits(x.astype(np.float32)), wl.f32_to_bf16_bits(g.astype(np.float32))


@pytest.mark.parametrize("g_powers", [(0,), (-40, 0), (50, 20)])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("K", [272, 6144, 8208])
def test_gradient_of_rows_far_from_one(gg, K, eps, g_powers):
    # dY about as far out as the rows' root mean square: the gradient is near the weight whatever the row,
    # while dY * weight, its products with Z, Z's squares and r^3 are not
    rng = np.random.default_rng(K + len(g_powers))
    z, g = _far(rng, K, g_powers)
    rms = np.log2(np.sqrt(np.exp2(2.0 * np.array(FAR)) + eps))
    out = np.clip(rms, -100, 90)
    dy, res = (wl.f32_to_bf16_bits((rng.standard_normal((len(FAR), K)) * np.exp2(p)[:, None]).astype(np.float32))
               for p in (out, out - rms))
    Z, W, D, R = (oracle._bf16_to_f64(a) for a in (z, g, dy, res))
    for r in (None, R):
        want, dg, err, mags = ref.norm_grad(D, Z, W, r, eps)
        dz, dw = gg.rms_norm_grad(ops.to_dev(dy), ops.to_dev(z), ops.to_dev(g), eps=eps,
                                  d_residual=None if r is None else ops.to_dev(res))
        for t in range(len(FAR)):
            ops.check_bf16(ops.host(dz[t]), want[t], err[t], "dz of a row at 2^%d" % FAR[t])
        ops.check_f32(ops.host(dw), dg, ref.NORM_DG_REL * mags, "dg")
    # a row at a time, so that none hides behind the largest one's share of dg
    for t in range(len(FAR)):
        _, dg, _, mags = ref.norm_grad(D[t:t + 1], Z[t:t + 1], W, None, eps)
        if mags[mags > 0].min() < 2.0 ** -120:
            continue  # (eps outweighs the row: no normal fp32 numbers)
        dw = gg.rms_norm_grad(ops.to_dev(dy[t:t + 1]), ops.to_dev(z[t:t + 1]), ops.to_dev(g), eps=eps)[1]
        ops.check_f32(ops.host(dw), dg, ref.NORM_DG_REL * mags, "dg of a row at 2^%d" % FAR[t])


@pytest.mark.parametrize("K", [144, 2064, 8208])
def test_gradient_where_rows_begin_to_be_far(gg, K):
    # rows and gradients on both sides of the powers of two up to which a row's sums are taken in
    # fp32, half of dY zeros, and a row without any gradient
    rng = np.random.default_rng(K)
    rows = [(z, d) for z in (-22, -21, -20, -19, -10, 0, 19, 20, 21) for d in (-118, -100, -90, -82, -60, 0, 55, 62)
            if d - z >= -100] + [(0, None)]
    z = wl.f32_to_bf16_bits((rng.standard_normal((len(rows), K)) * np.exp2([[p] for p, _ in rows])).astype(np.float32))
    g = wl.f32_to_bf16_bits((1 + 0.2 * rng.standard_normal(K)).astype(np.float32))
    dy = rng.standard_normal((len(rows), K)) * [[0 if p is None else 2.0 ** p] for _, p in rows] * rng.integers(0, 2, (len(rows), K))
    dy = wl.f32_to_bf16_bits(dy.astype(np.float32))
    Z, W, D = (oracle._bf16_to_f64(a) for a in (z, g, dy))
    want, dg, err, mags = ref.norm_grad(D, Z, W, None, 0.0)
    dz, dw = gg.rms_norm_grad(ops.to_dev(dy), ops.to_dev(z), ops.to_dev(g), eps=0.0)
    for t, row in enumerate(rows):
        ops.check_bf16(ops.host(dz[t]), want[t], err[t], "dz of %s" % (row,))
    ops.check_f32(ops.host(dw), dg, ref.NORM_DG_REL * mags, "dg")


def test_gradient_of_zeros_without_eps_is_nan(gg):
    z = torch.zeros((2, 272), dtype=torch.bfloat16, device=DEV)
    z[1] = 2.0 ** -100
    dy, w = torch.ones_like(z), torch.ones(272, dtype=torch.bfloat16, device=DEV)
    dz, dg = gg.rms_norm_grad(dy, z, w, eps=0.0)
    assert dz[0].isnan().all() and dg.isnan().all()
    assert (dz[1].abs() <= 2.0 ** 100 * 2.0 ** -14).all()  # 2^100 (1 - 1): what fp32 leaves of it


@pytest.mark.parametrize("g_powers", [(0,), (-60, 0), (70, 20)])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("K", [272, 6144, 8208, 16384])
def test_norm_of_rows_far_from_one(gg, K, eps, g_powers):
    # squares that leave fp32 on both sides, 1 / rms near its ends, and z * weight beyond them
    rng = np.random.default_rng(K + 3 * len(g_powers))
    x, g = _far(rng, K, g_powers)
    res = wl.f32_to_bf16_bits((rng.standard_normal(x.shape) * np.exp2(FAR)[:, None]).astype(np.float32))
    X, R, W = (oracle._bf16_to_f64(a) for a in (x, res, g))
    for residual in (None, R):
        z, y = ref.norm(X, residual, W, eps)
        got = gg.rms_norm_fp8(ops.to_dev(x), ops.to_dev(g), residual=None if residual is None else ops.to_dev(res),
                              eps=eps, with_norm=True)
        if residual is not None:
            assert np.array_equal(ops.host(got[2]), z)
        q, s, norm = got[0].view(torch.uint8).cpu().numpy(), ops.host(got[1]), ops.host(got[-1])
        assert np.isfinite(s).all()
        for t in range(len(FAR)):
            check_fp8(q[t:t + 1], s[:, t:t + 1], y[t:t + 1], ref.NORM_REL)
            # (half a step of a subnormal bf16 number besides, where eps outweighs a row by far)
            ops.check_bf16(norm[t], y[t], ref.NORM_REL * np.abs(y[t]) + 2.0 ** -134, "norm of a row at 2^%d" % FAR[t])


@pytest.mark.parametrize("K", [144, 2064, 16384])
def test_norm_where_a_product_with_the_weight_leaves_fp32(gg, K):
    # ordinary rows but for a few values and weights so far out that their product is subnormal or
    # beyond fp32 while the normalised value is neither
    rng = np.random.default_rng(K + 1)
    x, _, g = _inputs(rng, 9, K)
    X, W = oracle._bf16_to_f64(x), oracle._bf16_to_f64(g)
    for row, (scale, value, weight) in enumerate([(2.0 ** 40, 2.0 ** 41, 2.0 ** 90), (2.0 ** -40, 2.0 ** -41, 2.0 ** -90),
                                                  (2.0 ** -30, 2.0 ** -60, 2.0 ** -75), (1.0, 2.0 ** -100, 2.0 ** -20)]):
        at = int(rng.integers(0, K))
        X[row] *= scale
        X[row, at] = value
        W[at] = weight
    X[5, ::2] = 0.0
    X[6] = 0.0
    X[7, : K // 2] = 0.0
    x, g = wl.f32_to_bf16_bits(X.astype(np.float32)), wl.f32_to_bf16_bits(W.astype(np.float32))
    _, y = ref.norm(oracle._bf16_to_f64(x), None, oracle._bf16_to_f64(g), 1e-30)
    q, s, norm = gg.rms_norm_fp8(ops.to_dev(x), ops.to_dev(g), eps=1e-30, with_norm=True)
    check_fp8(q.view(torch.uint8).cpu().numpy(), ops.host(s), y, ref.NORM_REL)
    ops.check_bf16(ops.host(norm), y, ref.NORM_REL * np.abs(y) + 2.0 ** -134, "norm")


def test_norm_of_zeros_without_eps_is_nan(gg):
    x = torch.zeros((3, 272), dtype=torch.bfloat16, device=DEV)
    x[1], x[2] = 2.0 ** -120, -2.0 ** 120
    q, s, y = gg.rms_norm_fp8(x, torch.ones(272, dtype=torch.bfloat16, device=DEV), eps=0.0, with_norm=True)
    assert s[:, 0].isnan().all() and (q[0].view(torch.uint8) == 0).all() and y[0].isnan().all()
    assert (y[1] == 1).all() and (y[2] == -1).all() and (s[:, 1:] == np.float32(1 / 448)).all()
    # eps alone decides: r = 0, and everything finite is 0
    q, s, y = gg.rms_norm_fp8(x, torch.full((272,), 2.0 ** 100, dtype=torch.bfloat16, device=DEV), eps=float("inf"), with_norm=True)
    assert (y == 0).all() and (s == np.float32(2.0 ** -100 / 448)).all()


@pytest.mark.parametrize("K", [272, 6144, 16384])
def test_gradient_with_weights_and_gradients_of_zero(gg, K):
    # weights of 0 (as a layer begins with) in all columns and in runs of them, gradients of 0 in rows and runs
    rng = np.random.default_rng(K + 2)
    z, _, g = _inputs(rng, 6, K)
    dy = ops.bits(rng, 6, K, scale=0.02)
    dy[1], dy[2, 8:40], z[3, 64:96] = 0, 0, 0
    for weight in (np.zeros_like(g), np.where(np.arange(K) // 16 % 3 == 0, 0, g).astype(g.dtype)):
        Z, W, D = (oracle._bf16_to_f64(a) for a in (z, weight, dy))
        want, dg, err, mags = ref.norm_grad(D, Z, W, None, 1e-6)
        dz, dw = gg.rms_norm_grad(ops.to_dev(dy), ops.to_dev(z), ops.to_dev(weight))
        ops.check_bf16(ops.host(dz), want, err, "dz")
        ops.check_f32(ops.host(dw), dg, ref.NORM_DG_REL * mags, "dg")


def test_far_rows_among_others_in_a_workgroup(gg):
    # rows of one workgroup in turn far and not, more rows than workgroups: each row's result is its own
    rng = np.random.default_rng(4)
    T, K = 5000, 272
    z, _, g = _inputs(rng, T, K)
    dy = ops.bits(rng, T, K, scale=0.02)
    Z, D = oracle._bf16_to_f64(z), oracle._bf16_to_f64(dy)
    far = rng.integers(0, 3, T)
    Z *= np.array([1.0, 2.0 ** 60, 2.0 ** -60])[far][:, None]
    D *= np.array([1.0, 2.0 ** 60, 2.0 ** -60])[far][:, None]
    z, dy = (wl.f32_to_bf16_bits(a.astype(np.float32)) for a in (Z, D))
    dz, _ = gg.rms_norm_grad(ops.to_dev(dy), ops.to_dev(z), ops.to_dev(g), eps=0.0)
    q, s, y = gg.rms_norm_fp8(ops.to_dev(z), ops.to_dev(g), eps=0.0, with_norm=True)
    W = oracle._bf16_to_f64(g)
    want, _, err, _ = ref.norm_grad(D, Z, W, None, 0.0)
    ops.check_bf16(ops.host(dz), want, err, "dz")
    _, want = ref.norm(Z, None, W, 0.0)
    check_fp8(q.view(torch.uint8).cpu().numpy(), ops.host(s), want, ref.NORM_REL)
    ops.check_bf16(ops.host(y), want, ref.NORM_REL * np.abs(want), "norm")
    for _ in range(3):
        again = gg.rms_norm_grad(ops.to_dev(dy), ops.to_dev(z), ops.to_dev(g), eps=0.0)[0]
        assert torch.equal(again, dz)
