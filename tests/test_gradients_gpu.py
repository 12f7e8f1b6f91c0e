"""The gradients of the grouped product on the GPU against binary64 (needs an MI355X)."""

import numpy as np
import pytest

import oracle
import oracle.operators as ref
import workloads as wl
from tests import operators as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BMS = [0, 16, 32, 64, 128, 256]
DTYPES = ["fp32", "bf16"]


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _check(out, *args):
    (ops.check_f32 if out == "fp32" else ops.check_bf16)(*args)


def _dgrad_case(gg, sizes, K, N, bm, out, seed, spare=3, draw=ops.bits):
    rng = np.random.default_rng(seed)
    off = ops.offsets_of(sizes)
    M = int(off[-1])
    dC, B = draw(rng, M + spare, N), draw(rng, len(sizes), K, N)
    got = torch.full((M + spare, K), float("nan"), dtype=_dt(out), device="cuda:0")
    ret = gg.grouped_gemm_dgrad(ops.to_dev(dC), ops.to_dev(B), ops.to_dev(off), out=got, bm=bm)
    assert ret is got
    got = ops.host(got)
    want, S = ref.dgrad(dC, B, off)
    assert np.isnan(got[M:]).all(), "rows past the last group were written"
    return got[:M], want[:M], S[:M]


# empty and one-row experts, an expert of several tiles, lengths that end
# inside a slice (64 columns), inside a 16-byte piece's tile (8) and inside a
# 128- or 256-wide tile
SHAPES = [([0, 1, 17, 130, 0, 300], 328, 392), ([5], 8, 8), ([1], 136, 64), ([16, 16, 16], 1032, 72),
          ([300, 0, 45, 517], 200, 776), ([0, 0, 3], 264, 1000), ([33, 64, 65, 2], 512, 128)]


@pytest.mark.parametrize("bm", BMS)
@pytest.mark.parametrize("sizes,K,N", SHAPES)
def test_dgrad(gg, sizes, K, N, bm):
    for i, out in enumerate(DTYPES):
        got, want, S = _dgrad_case(gg, sizes, K, N, bm, out, 100 + i)
        _check(out, got, want, ops.sum_bound(N, S), "dgrad %s bm=%d %s" % (sizes, bm, out))


@pytest.mark.parametrize("copies", [1, 3, 4, 6, 12])
def test_dgrad_heights_of_a_launch(gg, copies):
    # heights of 16 to 256 together; from a few tiles, whose heights are cut to fill
    # the CUs, over half a round of the narrowest to several rounds of the widest
    sizes = [300, 20, 0, 700, 64, 130] * copies
    got, want, _ = _dgrad_case(gg, sizes, 1032, 72, 0, "fp32", 8, draw=ops.int_bits)
    assert (got == want).all()
    got, want, _ = _dgrad_case(gg, sizes, 72, 136, 0, "bf16", 9, draw=ops.int_bits)
    assert (got == oracle.round_to_bf16(want)).all()


@pytest.mark.parametrize("bm", BMS)
def test_dgrad_integers_are_exact(gg, bm):
    # every partial sum is an integer below 2^24
    got, want, _ = _dgrad_case(gg, [5, 0, 40, 129, 16], 264, 512, bm, "fp32", 7, draw=ops.int_bits)
    assert (got == want).all()


def test_dgrad_all_groups_empty(gg):
    got, want, _ = _dgrad_case(gg, [0, 0], 64, 64, 0, "fp32", 1)
    assert got.shape == (0, 64)


def test_dgrad_no_rows_at_all(gg):
    dC = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda:0")
    B = torch.ones((2, 32, 64), dtype=torch.bfloat16, device="cuda:0")
    off = torch.zeros(3, dtype=torch.int32, device="cuda:0")
    assert gg.grouped_gemm_dgrad(dC, B, off).shape == (0, 32)


def test_dgrad_nonfinite_stays_in_its_rows(gg):
    # an infinity or NaN in one row or one expert's weights reaches only the
    # results that sum over it; spare rows of NaN reach none
    rng = np.random.default_rng(3)
    off = ops.offsets_of([20, 30, 5])
    dC, B = ops.bits(rng, 60, 200), ops.bits(rng, 3, 136, 200)
    dC[55:] = 0x7FC0
    dC[7, 3] = 0x7F80
    B[1, 9, 150] = 0x7FC0
    for bm in BMS:
        got = ops.host(gg.grouped_gemm_dgrad(ops.to_dev(dC), ops.to_dev(B), ops.to_dev(off), bm=bm))
        clean = np.ones((55, 136), dtype=bool)
        clean[7] = False
        clean[20:50, 9] = False
        assert np.isfinite(got[:55][clean]).all()
        assert not np.isfinite(got[7]).any()
        assert np.isnan(got[20:50, 9]).all()


def _swiglu_case(gg, sizes, K, N, bm, seed, with_h, gate_scale=2.0, spare=2, in_place=False):
    rng = np.random.default_rng(seed)
    off = ops.offsets_of(sizes)
    M = int(off[-1])
    dY, B = ops.bits(rng, M + spare, N, scale=0.5), ops.bits(rng, len(sizes), K, N, scale=0.2)
    C = ops.bits(rng, M + spare, 2 * K, scale=gate_scale)
    tC = ops.to_dev(C)
    nan = float("nan")
    out = tC if in_place else torch.full((M + spare, 2 * K), nan, dtype=torch.bfloat16, device="cuda:0")
    h = torch.full((M + spare, K), nan, dtype=torch.bfloat16, device="cuda:0") if with_h else None
    gg.grouped_gemm_dgrad_swiglu(ops.to_dev(dY), ops.to_dev(B), ops.to_dev(off), tC, out=out, out_h=h,
                                 bm=bm)
    c64 = oracle._bf16_to_f64(C)[:M]
    dh, S = ref.dgrad(dY, B, off)
    dh, dh_err = dh[:M], ops.sum_bound(N, S[:M])
    want, want_h = ref.swiglu_grad(dh, c64)
    err, err_h = ref.swiglu_grad_error(dh, dh_err, c64)
    got = ops.host(out)
    what = "dgrad_swiglu %s K=%d N=%d bm=%d" % (sizes, K, N, bm)
    ops.check_bf16(got[:M], want, err, what)
    if in_place:
        assert (ops.bits_of(out)[M:] == C[M:]).all()
    else:
        assert np.isnan(got[M:]).all()
    if with_h:
        gh = ops.host(h)
        ops.check_bf16(gh[:M], want_h, err_h, what + " H")
        assert np.isnan(gh[M:]).all()


@pytest.mark.parametrize("bm", BMS)
@pytest.mark.parametrize("sizes,K,N", SHAPES)
def test_dgrad_swiglu(gg, sizes, K, N, bm):
    _swiglu_case(gg, sizes, K, N, bm, 200, True)


@pytest.mark.parametrize("bm", [0, 16, 128, 256])
def test_dgrad_swiglu_without_h_and_in_place(gg, bm):
    _swiglu_case(gg, [3, 0, 150, 40], 296, 104, bm, 201, False)
    _swiglu_case(gg, [3, 0, 150, 40], 296, 104, bm, 202, True, in_place=True)


def test_dgrad_swiglu_large_gates(gg):
    # gates out to +-200: e^-gate overflows, sigmoid is 0 or 1
    _swiglu_case(gg, [70, 9], 128, 64, 0, 203, True, gate_scale=60.0)


def test_dgrad_swiglu_large_factors(gg):
    # dH * up lies beyond fp32, the sigmoid's factor brings the gradient back: finite
    # results are the formula's, and 0 where the sigmoid is 0 (gates below -87.3)
    # (beside large values at the steepest slope, 1.0998 at 2.4)
    big = 2.0 ** 126
    gates = np.repeat([-100.0, -95.0, -60.0, -40.0, -60.0, -60.0, 2.40625, 2.40625], 8)
    ups = np.repeat([2.0 ** 70, -2.0 ** 100, 2.0 ** 70, 2.0 ** 64, 2.0 ** 100, -2.0 ** 30, big, -big], 8)
    dhs = np.repeat([2.0 ** 70, 2.0 ** 60, 2.0 ** 70, -2.0 ** 65, 2.0 ** 60, 2.0 ** 120, 2.0 ** -2, -2.0 ** -3], 8)
    I = gates.size
    C = wl.f32_to_bf16_bits(np.stack([gates, ups], axis=-1).reshape(1, 2 * I).astype(np.float32))
    dY, eye = wl.f32_to_bf16_bits(dhs[None].astype(np.float32)), wl.f32_to_bf16_bits(np.eye(I, dtype=np.float32))
    got = ops.host(gg.grouped_gemm_dgrad_swiglu(ops.to_dev(dY), ops.to_dev(eye[None]), ops.to_dev(ops.offsets_of([1])),
                                                ops.to_dev(C))).astype(np.float64)
    want, _ = ref.swiglu_grad(dhs[None], np.stack([gates, ups], axis=-1).reshape(1, 2 * I))
    live = np.repeat(gates > -88, 2)[None]
    # sigmoid is off by |gate| + 3 ulps, its complement's sum and the products by less than
    # 8 more (62 * 2^-23 = 2^-17 at gate = -60, and 2^-17 covers the rest), then one rounding to bf16
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want))[live].all()
    assert (got[~live] == 0).all()


def test_dgrad_swiglu_where_the_sigmoid_ends(gg):
    # s of gates from -87.5 on would be subnormal and is 0; before that it is there
    gates = np.array([-86.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -100.0])
    I, h = gates.size, 2.0 ** 60
    C = wl.f32_to_bf16_bits(np.stack([gates, np.full(I, h)], axis=-1).reshape(1, 2 * I).astype(np.float32))
    dY = wl.f32_to_bf16_bits(np.full((1, I), h, dtype=np.float32))
    eye = wl.f32_to_bf16_bits(np.eye(I, dtype=np.float32))[None]
    d, H = (ops.host(t).astype(np.float64)[0] for t in gg.grouped_gemm_dgrad_swiglu(
        ops.to_dev(dY), ops.to_dev(eye), ops.to_dev(ops.offsets_of([1])), ops.to_dev(C), with_h=True))
    want, want_h = ref.swiglu_grad(np.full((1, I), h), np.stack([gates, np.full(I, h)], axis=-1).reshape(1, 2 * I))
    for got, exact, scale in ((d[0::2], want[0, 0::2], h * h), (d[1::2], want[0, 1::2], h), (H, want_h[0], h)):
        assert (got[3:] == 0).all() and (np.abs(exact[3:]) < 1.1e-36 * scale).all()
        # |gate| + 3 ulps of s and a few of the products, one rounding to bf16
        assert (np.abs(got - exact)[:3] <= (2.0 ** -8 + 2.0 ** -16) * np.abs(exact[:3])).all()


def test_dgrad_swiglu_differences(gg):
    # the gradient against central differences of sum(dH * silu(gate) * up) in
    # binary64; K = N with identity weights, so that dH = dY
    rng = np.random.default_rng(9)
    M, I = 12, 64
    C, dY = ops.bits(rng, M, 2 * I, scale=1.5), ops.bits(rng, M, I)
    eye = wl.f32_to_bf16_bits(np.eye(I, dtype=np.float32))[None]
    got = ops.host(gg.grouped_gemm_dgrad_swiglu(ops.to_dev(dY), ops.to_dev(eye),
                                                ops.to_dev(ops.offsets_of([M])), ops.to_dev(C)))
    c, d = oracle._bf16_to_f64(C), oracle._bf16_to_f64(dY)
    loss = lambda x: d * oracle.swiglu_pairs(x)  # noqa: E731
    h = 2.0 ** -14
    for which in (0, 1):
        step = np.zeros_like(c)
        step[:, which::2] = h
        diff = (loss(c + step) - loss(c - step)) / (2 * h)
        # the third derivative times h^2 / 6 (|silu'''| < 1), the cancellation in
        # binary64, and the rounding to bf16
        err = np.abs(d) * np.maximum(np.abs(c[:, 1::2]), 1) * h * h + 1e-10 + 2.0 ** -8 * np.abs(diff)
        assert (np.abs(got[:, which::2] - diff) <= err + 2.0 ** -22).all()


def _wgrad_case(gg, sizes, K, N, out, seed, spare=3, draw=ops.bits, accumulate=False, A=None, dC=None):
    rng = np.random.default_rng(seed)
    off = ops.offsets_of(sizes)
    M = int(off[-1])
    A = draw(rng, M + spare, K) if A is None else A
    dC = draw(rng, M + spare, N) if dC is None else dC
    old = rng.standard_normal((len(sizes), K, N)).astype(np.float32)
    got = ops.to_dev(old) if accumulate else torch.full((len(sizes), K, N), float("nan"), dtype=_dt(out),
                                                        device="cuda:0")
    gg.grouped_gemm_wgrad(ops.to_dev(A), ops.to_dev(dC), ops.to_dev(off), out=got, accumulate=accumulate)
    want, S = ref.wgrad(A, dC, off)
    n = np.asarray(sizes)[:, None, None]
    err = ops.sum_bound(n, S)
    if accumulate:
        want = want + old
        err = err + ops.ULP * (np.abs(want) + err)
        err[np.asarray(sizes) == 0] = 0
    return ops.host(got), want, err


# K and N below, at and past the tiles' 64, 128 and 256; enough experts for the
# large tiles in the last ones; row counts around the slices' 32
WSHAPES = [([0, 1, 17, 130, 0, 300], 328, 392), ([5], 8, 8), ([1], 136, 72), ([31, 32, 33, 64, 65], 200, 264),
           ([97], 1032, 16), ([1000, 0, 333, 31], 72, 136),
           ([3, 0, 40, 7] * 16, 264, 520), ([0] * 70 + [50, 1], 256, 776)]


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("sizes,K,N", WSHAPES)
def test_wgrad(gg, sizes, K, N, out):
    got, want, err = _wgrad_case(gg, sizes, K, N, out, 300)
    _check(out, got, want, err, "wgrad %s K=%d N=%d %s" % (sizes[:8], K, N, out))
    for e, m in enumerate(sizes):
        if m == 0:
            assert (got[e] == 0).all()


@pytest.mark.parametrize("sizes,K,N", WSHAPES)
def test_wgrad_accumulate(gg, sizes, K, N):
    got, want, err = _wgrad_case(gg, sizes, K, N, "fp32", 301, accumulate=True)
    ops.check_f32(got, want, err, "wgrad accumulate")


@pytest.mark.parametrize("sizes,K,N", [([5, 0, 40, 129, 16], 264, 512), ([9, 60, 0, 33] * 20, 256, 520), ([777], 40, 72)])
def test_wgrad_integers_are_exact(gg, sizes, K, N):
    got, want, _ = _wgrad_case(gg, sizes, K, N, "fp32", 302, draw=ops.int_bits)
    assert (got == want).all()


# long groups whose tiles of 64 x 64 are 65 to 256: waves share the rows
LONG = [([3100], 600, 456), ([6200, 1], 264, 520), ([0, 9001, 0], 520, 200)]


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("sizes,K,N", LONG)
def test_wgrad_long_groups(gg, sizes, K, N, out):
    got, want, err = _wgrad_case(gg, sizes, K, N, out, 306)
    _check(out, got, want, err, "wgrad %s K=%d N=%d %s" % (sizes, K, N, out))
    for accumulate in (False, True) if out == "fp32" else ():
        got, want, err = _wgrad_case(gg, sizes, K, N, out, 307, draw=ops.int_bits, accumulate=accumulate)
        assert (np.abs(got - want) <= (err if accumulate else 0)).all()


def test_wgrad_many_experts_and_ties(gg):
    # 1024 experts of 0 .. 40 rows: the order by size has ties everywhere
    rng = np.random.default_rng(5)
    sizes = rng.integers(0, 41, size=1024).tolist()
    got, want, _ = _wgrad_case(gg, sizes, 24, 40, "fp32", 303, draw=ops.int_bits)
    assert (got == want).all()
    got, want, _ = _wgrad_case(gg, sizes[:130], 264, 520, "fp32", 304, draw=ops.int_bits)
    assert (got == want).all()


@pytest.mark.parametrize("E", [64, 65, 200, 256, 257])
def test_wgrad_expert_counts(gg, E):
    # one, two and more votes of 64 experts; large tiles
    sizes = np.random.default_rng(E).integers(0, 20, size=E)
    sizes[E // 2] = 300
    got, want, _ = _wgrad_case(gg, sizes.tolist(), 256, 264, "fp32", 305, draw=ops.int_bits)
    assert (got == want).all()


@pytest.mark.parametrize("N", [256, 264])
@pytest.mark.parametrize("out", DTYPES)
def test_wgrad_output_off_a_line(gg, N, out):
    # a gradient that starts 16 bytes into a line, as a part of a larger buffer
    # does, with and without accumulation; its surroundings stay as they were
    rng = np.random.default_rng(N)
    sizes, K = [33, 0, 90] * 30, 136
    off = ops.offsets_of(sizes)
    A, dC = ops.int_bits(rng, int(off[-1]), K), ops.int_bits(rng, int(off[-1]), N)
    want, _ = ref.wgrad(A, dC, off)
    n, pad = want.size, 16 // _dt(out).itemsize
    buf = torch.full((n + 2 * pad,), 3.0, dtype=_dt(out), device="cuda:0")
    view = buf[pad:pad + n].view(want.shape)
    assert view.data_ptr() % 128 == 16
    args = [ops.to_dev(t) for t in (A, dC, off)]
    gg.grouped_gemm_wgrad(*args, out=view)
    got = ops.host(view)
    assert (got == (want if out == "fp32" else oracle.round_to_bf16(want))).all()
    if out == "fp32":
        gg.grouped_gemm_wgrad(*args, out=view, accumulate=True)
        assert (ops.host(view) == 2 * want).all()
    assert (buf[:pad] == 3).all() and (buf[-pad:] == 3).all()


def test_rows_beyond_4_gigabytes(gg):
    # the last group's rows lie past 2^32 bytes of dC and past 2^31 of dA
    M, N, K, last = 560_000, 4096, 64, 70
    off = torch.tensor([0, M - last, M], dtype=torch.int32, device="cuda:0")
    rng = np.random.default_rng(14)
    dC = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda:0")
    A = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda:0")
    tail, a_tail, B = ops.int_bits(rng, last, N), ops.int_bits(rng, last, K), ops.int_bits(rng, 2, K, N)
    dC[M - last:] = ops.to_dev(tail)
    A[M - last:] = ops.to_dev(a_tail)
    want, _ = ref.dgrad(tail, B[1:], np.array([0, last]))
    for bm in (0, 16):
        got = gg.grouped_gemm_dgrad(dC, ops.to_dev(B), off, bm=bm)
        assert (ops.host(got[M - last:]) == want).all() and not got[:M - last].any()
    dB = ops.host(gg.grouped_gemm_wgrad(A, dC, off))
    assert (dB[1] == ref.wgrad(a_tail, tail, np.array([0, last]))[0][0]).all() and (dB[0] == 0).all()
    del dC, A, got
    torch.cuda.empty_cache()


def _signs(*shape, seed):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda:0", dtype=torch.int8).to(torch.bfloat16)


@pytest.mark.parametrize("rows,K,N", [(3, 264, 2 ** 21), (300, 8, 2 ** 21), (20, 2 ** 24, 8)])
def test_dgrad_longest_rows(gg, rows, K, N):
    # -1, 0 and 1: sums of at most 2^21 of them are exact in fp32
    dC, B = _signs(rows, N, seed=1), _signs(1, K, N, seed=2)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda:0")
    want = dC.float() @ B[0].float().t()
    for bm in (0, 256):
        assert torch.equal(gg.grouped_gemm_dgrad(dC, B, off, bm=bm), want)
    torch.cuda.empty_cache()


def test_dgrad_swiglu_longest_rows(gg):
    # gate 0 and up in -1, 0, 1: d gate = dH * up / 2 is a bf16 value, d up = 0
    rows, K, N = 18, 2 ** 24, 8
    dY, B, up = _signs(rows, N, seed=3), _signs(1, K, N, seed=4), _signs(rows, K, seed=5)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda:0")
    C = torch.zeros((rows, K, 2), dtype=torch.bfloat16, device="cuda:0")
    C[..., 1] = up
    dC = gg.grouped_gemm_dgrad_swiglu(dY, B, off, C.view(rows, 2 * K)).view(rows, K, 2)
    assert torch.equal(dC[..., 0].float(), (dY.float() @ B[0].float().t()) * up.float() / 2)
    assert not dC[..., 1].any()
    del C, dC
    torch.cuda.empty_cache()


@pytest.mark.parametrize("K,N", [(2 ** 22, 8), (8, 2 ** 22)])
def test_wgrad_longest_rows(gg, K, N):
    A, dC = _signs(70, K, seed=6), _signs(70, N, seed=7)
    off = torch.tensor([0, 33, 70], dtype=torch.int32, device="cuda:0")
    want = torch.stack([A[:33].float().t() @ dC[:33].float(), A[33:].float().t() @ dC[33:].float()])
    for out in DTYPES:
        assert torch.equal(gg.grouped_gemm_wgrad(A, dC, off, out_dtype=_dt(out)).float(), want)
    torch.cuda.empty_cache()


def test_wgrad_neighbours_rows_stay_out(gg):
    # NaN in an expert's rows reaches that expert's gradient only
    rng = np.random.default_rng(6)
    for sizes, K, N in (([20, 30, 5], 136, 200), ([20, 30, 5] * 30, 256, 264)):
        off = ops.offsets_of(sizes)
        A, dC = ops.bits(rng, int(off[-1]) + 4, K), ops.bits(rng, int(off[-1]) + 4, N)
        A[off[-1]:] = 0x7FC0
        dC[off[-1]:] = 0x7F80
        A[off[1]:off[2]] = 0x7FC0
        got = ops.host(gg.grouped_gemm_wgrad(ops.to_dev(A), ops.to_dev(dC), ops.to_dev(off)))
        assert np.isnan(got[1]).all()
        assert np.isfinite(np.delete(got, 1, axis=0)).all()


def test_wgrad_no_rows_at_all(gg):
    off = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    A = torch.empty((0, 72), dtype=torch.bfloat16, device="cuda:0")
    dC = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda:0")
    got = torch.full((3, 72, 40), float("nan"), device="cuda:0")
    gg.grouped_gemm_wgrad(A, dC, off, out=got)
    assert (got == 0).all()


def test_same_bits_twice(gg):
    rng = np.random.default_rng(8)
    off = ops.to_dev(ops.offsets_of([40, 300, 0, 7]))
    A, dC = ops.to_dev(ops.bits(rng, 347, 264)), ops.to_dev(ops.bits(rng, 347, 392))
    B = ops.to_dev(ops.bits(rng, 4, 264, 392))
    for f in (lambda: gg.grouped_gemm_wgrad(A, dC, off), lambda: gg.grouped_gemm_dgrad(dC, B, off)):
        assert torch.equal(f(), f())


def test_arrays_side_by_side(gg):
    # inputs and outputs that meet end to start inside one buffer are apart
    rng = np.random.default_rng(16)
    M, K, N, E = 40, 72, 136, 2
    off = ops.to_dev(ops.offsets_of([33, 7]))
    parts = [(M, N), (M, K), (E, K, N), (E, K, N), (M, 2 * K), (M, 2 * K), (M, K)]
    dC, dA, B, dB, C, d, H = torch.zeros(sum(int(np.prod(p)) for p in parts), dtype=torch.bfloat16,
                                         device="cuda:0").split([int(np.prod(p)) for p in parts])
    dC, dA, B, dB, C, d, H = (t.view(p) for t, p in zip((dC, dA, B, dB, C, d, H), parts))
    for t in (dC, B, C):
        t.copy_(ops.to_dev(ops.bits(rng, *t.shape)))
    want = gg.grouped_gemm_dgrad(dC, B, off, out_dtype=torch.bfloat16)
    assert torch.equal(gg.grouped_gemm_dgrad(dC, B, off, out=dA), want)
    want_d, want_h = gg.grouped_gemm_dgrad_swiglu(dC, B, off, C, with_h=True)
    gg.grouped_gemm_dgrad_swiglu(dC, B, off, C, out=d, out_h=H)
    assert torch.equal(d, want_d) and torch.equal(H, want_h)
    want = gg.grouped_gemm_wgrad(dA, dC, off, out_dtype=torch.bfloat16)
    assert torch.equal(gg.grouped_gemm_wgrad(dA, dC, off, out=dB), want)


def test_outputs_over_inputs_are_refused(gg):
    off = ops.to_dev(ops.offsets_of([40]))
    X = torch.zeros((40, 64), dtype=torch.bfloat16, device="cuda:0")
    B = torch.zeros((1, 64, 64), dtype=torch.bfloat16, device="cuda:0")
    C = torch.zeros((41, 128), dtype=torch.bfloat16, device="cuda:0")
    for call in (lambda: gg.grouped_gemm_dgrad(X, B, off, out=X),
                 lambda: gg.grouped_gemm_dgrad_swiglu(X, B, off, C[:40], out=C[1:]),
                 lambda: gg.grouped_gemm_dgrad_swiglu(X, B, off, C[:40], out_h=X),
                 lambda: gg.grouped_gemm_wgrad(B[0][:40], X, off, out=B)):
        with pytest.raises(gg.GroupedGemmError, match="status 1 .*shares memory"):
            call()


@pytest.mark.parametrize("offs", [[0, 9, 4, 30], [-5, 10, 20, 30], [0, 10, 99, 30], [7, 7, 7, 7],
                                  [30, 20, 10, 0]])
def test_malformed_offsets_stay_inside(gg, offs):
    # clamped offsets; what is written lies inside the arrays, guarded on both sides
    rng = np.random.default_rng(10)
    M, K, N = 30, 72, 136
    dC, A, B = ops.bits(rng, M, N), ops.bits(rng, M, K), ops.bits(rng, 3, K, N)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda:0")

    def guarded(rows, cols):
        buf = torch.full((rows + 64, cols), -7.0, device="cuda:0")
        return buf, buf[32:32 + rows]

    for bm in (0, 16, 256):
        buf, out = guarded(M, K)
        gg.grouped_gemm_dgrad(ops.to_dev(dC), ops.to_dev(B), off, out=out, bm=bm)
        assert (buf[:32] == -7).all() and (buf[-32:] == -7).all()
    buf, out = guarded(3 * K, N)
    gg.grouped_gemm_wgrad(ops.to_dev(A), ops.to_dev(dC), off, out=out.view(3, K, N))
    assert (buf[:32] == -7).all() and (buf[-32:] == -7).all() and torch.isfinite(out).all()


def test_training_step_of_a_layer(gg):
    # an expert layer's forward and backward by these operators alone, against
    # binary64 autograd: loss = sum(Y * W)
    rng = np.random.default_rng(11)
    sizes, D, I = [37, 0, 70, 1, 21], 136, 72
    off = ops.offsets_of(sizes)
    M, E = int(off[-1]), len(sizes)
    X, W = ops.bits(rng, M, D), ops.bits(rng, M, D)
    B1, B2 = ops.bits(rng, E, D, 2 * I, scale=D ** -0.5), ops.bits(rng, E, I, D, scale=I ** -0.5)
    tX, tdY, tB1, tB2, toff = (ops.to_dev(t) for t in (X, W, B1, B2, off))

    C = gg.grouped_gemm(tX, tB1, toff, out_dtype=torch.bfloat16)
    dC, H = gg.grouped_gemm_dgrad_swiglu(tdY, tB2, toff, C, with_h=True)
    dB2 = gg.grouped_gemm_wgrad(H, tdY, toff)
    dX = gg.grouped_gemm_dgrad(dC, tB1, toff)
    dB1 = gg.grouped_gemm_wgrad(tX, dC, toff)

    leaf = lambda b: torch.from_numpy(oracle._bf16_to_f64(b)).requires_grad_()  # noqa: E731
    x, b1, b2 = leaf(X), leaf(B1), leaf(B2)
    w = torch.from_numpy(oracle._bf16_to_f64(W))
    loss = 0.0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        c = x[lo:hi] @ b1[e]
        h = torch.nn.functional.silu(c[:, 0::2]) * c[:, 1::2]
        loss = loss + (h @ b2[e] * w[lo:hi]).sum()
    loss.backward()
    # Roundings to bf16 on the way, each of at most 2^-8 of the value: gate, up,
    # the gradient of either, H.
    for got, want in ((dX, x.grad), (dB1, b1.grad), (dB2, b2.grad)):
        want = want.numpy()
        rel = np.linalg.norm(ops.host(got) - want) / np.linalg.norm(want)
        assert rel < 4 * 2.0 ** -8, rel


def test_graph_replays_follow_the_offsets(gg):
    # captured once, replayed on other rows, weights and group sizes
    rng = np.random.default_rng(12)
    K, N, M = 136, 264, 96
    sets = [([90, 0, 6], 1), ([0, 96, 0], 2), ([30, 31, 35], 3)]
    A, dC = (torch.zeros((M, c), dtype=torch.bfloat16, device="cuda:0") for c in (K, N))
    B = torch.zeros((3, K, N), dtype=torch.bfloat16, device="cuda:0")
    off = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    C = torch.zeros((M, 2 * K), dtype=torch.bfloat16, device="cuda:0")

    def step():
        return (gg.grouped_gemm_dgrad(dC, B, off), gg.grouped_gemm_wgrad(A, dC, off),
                *gg.grouped_gemm_dgrad_swiglu(dC, B, off, C, with_h=True))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for sizes, seed in sets * 2:
        r = np.random.default_rng(seed)
        A.copy_(ops.to_dev(ops.bits(r, M, K)))
        dC.copy_(ops.to_dev(ops.bits(r, M, N)))
        B.copy_(ops.to_dev(ops.bits(r, 3, K, N)))
        C.copy_(ops.to_dev(ops.bits(r, M, 2 * K)))
        off.copy_(ops.to_dev(ops.offsets_of(sizes)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want)


def test_two_streams_at_once(gg):
    rng = np.random.default_rng(15)
    sets = []
    for seed in range(2):
        off = ops.to_dev(ops.offsets_of([500 + seed, 12, 90]))
        A, dC = ops.to_dev(ops.bits(rng, 602 + seed, 264)), ops.to_dev(ops.bits(rng, 602 + seed, 1032))
        B, C = ops.to_dev(ops.bits(rng, 3, 264, 1032)), ops.to_dev(ops.bits(rng, 602 + seed, 528))
        sets.append((A, dC, B, off, C))

    def step(A, dC, B, off, C, s=None):
        return (gg.grouped_gemm_dgrad(dC, B, off, stream=s), gg.grouped_gemm_wgrad(A, dC, off, stream=s),
                *gg.grouped_gemm_dgrad_swiglu(dC, B, off, C, with_h=True, stream=s))

    want = [step(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[step(*x, s=s) for x, s in zip(sets, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for turn in got:
        for g, w in zip(turn, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_tensors_dropped_after_a_call_on_another_stream(gg):
    # a busy stream runs the call long after its inputs and outputs were dropped and their
    # memory could be handed out again: nothing of it may be, until the stream is through
    off = ops.to_dev(ops.offsets_of([256, 256]))
    ones = lambda *shape: torch.ones(shape, dtype=torch.bfloat16, device="cuda:0")  # noqa: E731
    rows, weights = (lambda: ones(512, 512)), (lambda: ones(2, 512, 512))
    codes = lambda: (*gg.mx4_quantize(rows()), *gg.mx4_quantize_weights(weights()))  # noqa: E731
    calls = [
        (lambda: (rows(), weights()), lambda s, a, b: gg.grouped_gemm_dgrad(a, b, off, stream=s), 512.0),
        (lambda: (rows(), rows()), lambda s, a, b: gg.grouped_gemm_wgrad(a, b, off, stream=s), 256.0),
        (lambda: (rows(), weights(), torch.zeros((512, 1024), dtype=torch.bfloat16, device="cuda:0")),
         lambda s, a, b, c: gg.grouped_gemm_dgrad_swiglu(a, b, off, c, with_h=True, stream=s)[1], 0.0),
        (lambda: (rows(),), lambda s, a: gg.mx4_dequantize(*gg.mx4_quantize(a, stream=s), stream=s), 1.0),
        (lambda: (weights(),), lambda s, a: gg.mx4_dequantize(*gg.mx4_quantize_weights(a, stream=s), stream=s), 1.0),
        (codes, lambda s, *c: gg.grouped_gemm_mx4(*c, off, stream=s), 512.0),
        (codes, lambda s, *c: gg.grouped_gemm_mx4_swiglu(*c, off, stream=s), 512.0 ** 2)]
    for make, call, want in calls:
        call(None, *make())  # a kernel's first launch loads it, which takes its time

        def attempt(s):
            torch.cuda.empty_cache()
            args = make()
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                torch.cuda._sleep(ops.SLEEP)
            got = call(s, *args)
            del args
            spoil = [torch.full((2 ** 18,), 7.0, dtype=torch.bfloat16, device="cuda:0") for _ in range(24)]
            torch.cuda.current_stream().synchronize()
            in_time = not s.query()  # the memory was written before the call ran
            s.synchronize()
            assert (got == want).all()
            del spoil
            return in_time

        ops.beside(attempt)


def test_captured_with_the_stream_named(gg):
    # the capturing stream passed by name, intermediate tensors dropped inside the capture
    rng = np.random.default_rng(17)
    off = ops.to_dev(ops.offsets_of([50, 14]))
    A, dC = ops.to_dev(ops.bits(rng, 64, 136)), ops.to_dev(ops.bits(rng, 64, 264))
    B = ops.to_dev(ops.bits(rng, 2, 136, 264))

    def step(s=None):
        d = gg.grouped_gemm_dgrad(dC, B, off, stream=s, out_dtype=torch.bfloat16)
        return gg.grouped_gemm_wgrad(d, dC, off, stream=s), gg.grouped_gemm_wgrad(A, dC, off, stream=s)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(torch.cuda.current_stream())
    for seed in (1, 2, 3):
        dC.copy_(ops.to_dev(ops.bits(np.random.default_rng(seed), 64, 264)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want)


def test_other_stream(gg):
    rng = np.random.default_rng(13)
    off = ops.to_dev(ops.offsets_of([50, 14]))
    A, dC = ops.to_dev(ops.bits(rng, 64, 136)), ops.to_dev(ops.bits(rng, 64, 264))
    B = ops.to_dev(ops.bits(rng, 2, 136, 264))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    on_s = [gg.grouped_gemm_dgrad(dC, B, off, stream=s), gg.grouped_gemm_wgrad(A, dC, off, stream=s)]
    s.synchronize()
    for got, want in zip(on_s, (gg.grouped_gemm_dgrad(dC, B, off), gg.grouped_gemm_wgrad(A, dC, off))):
        assert torch.equal(got, want)
