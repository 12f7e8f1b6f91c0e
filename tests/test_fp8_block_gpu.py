"""8-bit operands with a scale for each block of 128 on the GPU against binary64 (needs an MI355X)."""

import numpy as np
import pytest

import oracle
import oracle.layer as ref
import workloads as wl
from tests import operators as ops
from tests import parity
from tests import ring_schedule

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BMS = [0, 16, 32, 64, 128, 256]
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _hot(rng, *shape):
    """Rows with a few columns hotter than the rest, blocks of zeros among them."""
    x = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape[-1]))
    x[..., : min(128, shape[-1])] *= rng.integers(0, 2, size=shape[:-1] + (1,))
    return wl.f32_to_bf16_bits(x.astype(np.float32))


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def same(got, want):
    """Equal bit for bit, NaN being NaN."""
    return np.array_equal(got, want, equal_nan=got.dtype.kind == "f")


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("M,K", [(0, 128), (1, 16), (1, 8192), (3, 224), (33, 128), (129, 1040), (64, 144), (5, 6144)])
def test_quantize_rows(gg, M, K):
    x = _hot(np.random.default_rng(M * K), M, K)
    q, s = gg.fp8_quantize(ops.to_dev(x))
    want_q, want_s = ref.fp8_rows(x)
    assert q.dtype == F8 and same(s.cpu().numpy(), want_s)
    assert same(codes(q), want_q)


@pytest.mark.parametrize("for_grad", [False, True])
@pytest.mark.parametrize("E,K,N", [(1, 16, 16), (3, 224, 48), (2, 256, 256), (2, 1040, 272), (5, 144, 784)])
def test_quantize_weights(gg, E, K, N, for_grad):
    b = _hot(np.random.default_rng(E * K + N), E, K, N)
    q, s = gg.fp8_quantize_weights(ops.to_dev(b), for_grad=for_grad)
    want_q, want_s = ref.fp8_weights(b, for_grad)
    assert same(s.cpu().numpy(), want_s)
    assert same(codes(q), want_q)


def test_quantize_weights_of_eight(gg):
    # the dimension that is not summed may be any multiple of 8
    b = _hot(np.random.default_rng(5), 2, 48, 8)
    assert same(codes(gg.fp8_quantize_weights(ops.to_dev(b))[0]), ref.fp8_weights(b)[0])
    b = _hot(np.random.default_rng(6), 2, 24, 144)
    assert same(codes(gg.fp8_quantize_weights(ops.to_dev(b), for_grad=True)[0]), ref.fp8_weights(b, True)[0])


def test_quantize_every_bf16_value(gg):
    # every finite magnitude in a block of its own with a largest value 0 to 9 binades above
    # it (so that the steps fall everywhere), the signs in turn
    mags = np.arange(0x7F80, dtype=np.uint32)
    x = np.zeros((10, len(mags), 128), np.uint16)
    for up in range(10):
        x[up, :, 0] = np.minimum(mags + 128 * up, 0x7F7F)
        x[up, :, 1] = mags
        x[up, :, 2] = mags | 0x8000
    x = x.reshape(10 * len(mags), 128)
    want_q, want_s = ref.fp8_rows(x)
    q, s = gg.fp8_quantize(ops.to_dev(x))
    assert same(s.cpu().numpy(), want_s) and same(codes(q), want_q)


def test_blocks_with_infinities_and_nan(gg):
    x = _hot(np.random.default_rng(7), 4, 400)
    x[1, 130], x[2, 5], x[3, 399] = 0x7F80, 0x7FC1, 0xFF80
    q, s = gg.fp8_quantize(ops.to_dev(x))
    want_q, want_s = ref.fp8_rows(x)
    assert np.isnan(want_s[1, 1]) and np.isnan(want_s[0, 2]) and np.isnan(want_s[3, 3]) and np.isnan(want_s).sum() == 3
    assert same(s.cpu().numpy(), want_s) and same(codes(q), want_q)
    b = _hot(np.random.default_rng(8), 2, 272, 272)
    b[1, 150, 3] = 0x7F80
    for g in (False, True):
        q, s = gg.fp8_quantize_weights(ops.to_dev(b), for_grad=g)
        want_q, want_s = ref.fp8_weights(b, g)
        assert np.isnan(want_s).sum() == 1
        assert same(s.cpu().numpy(), want_s) and same(codes(q), want_q)


def test_rows_past_2_to_the_32_bytes(gg):
    M, K = 2 ** 18 + 3, 16384  # 2^32 values
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    pick = [0, 1, M // 2, M - 2, M - 1]
    bits = _hot(np.random.default_rng(9), len(pick), K)
    x[pick] = ops.to_dev(bits)
    q, s = gg.fp8_quantize(x)
    want_q, want_s = ref.fp8_rows(bits)
    assert same(codes(q[pick]), want_q) and same(s[:, pick].cpu().numpy(), want_s)
    assert int(q.view(torch.uint8).sum(dtype=torch.int64)) == int(want_q.sum(dtype=np.int64))


# --------------------------------------------------------------------- product

def _operands(rng, sizes, K, N, extra=0):
    M = int(sum(sizes)) + extra
    x, b = _hot(rng, M, K), ops.bits(rng, len(sizes), K, N, scale=1 / np.sqrt(K))
    Aq, As = ref.fp8_rows(x)
    Bq, Bs = ref.fp8_weights(b)
    return Aq, As, Bq, Bs, ops.offsets_of(sizes)


def _dev(args):
    return [ops.to_dev(a) for a in args]


def _check(gg, args, bm=0, spare=0, forms=("f32", "bf16", "swiglu")):
    Aq, As, Bq, Bs, off = args
    K = Aq.shape[1]
    M = int(off[-1])
    C, S, G = (t[:M] for t in ref.fp8_product(*args))
    err = ref.fp8_product_error(S, G, K)
    d = _dev(args)
    N = Bq.shape[1]
    if "f32" in forms:
        out = torch.full((Aq.shape[0], N), 7.0, device=DEV)
        gg.grouped_gemm_fp8_block(*d, out=out, bm=bm)
        ops.check_f32(ops.host(out[:M]), C, err, "fp32")
        assert (out[M:] == 7).all()
    if "bf16" in forms:
        out = torch.full((Aq.shape[0], N), 7.0, dtype=torch.bfloat16, device=DEV)
        gg.grouped_gemm_fp8_block(*d, out=out, bm=bm)
        ops.check_bf16(ops.host(out[:M]), C, err, "bf16")
        assert (out[M:] == 7).all()
    if "swiglu" in forms:
        out = torch.full((Aq.shape[0], N // 2), 7.0, dtype=torch.bfloat16, device=DEV)
        gg.grouped_gemm_fp8_block_swiglu(*d, out=out, bm=bm)
        parity.check_swiglu_bf16(ops.host(out[:M]), C, S, "swiglu", err=err)
        assert (out[M:] == 7).all()


@pytest.mark.parametrize("bm", BMS)
@pytest.mark.parametrize("sizes,K,N", [
    ([1], 16, 8), ([3, 0, 17, 9], 256, 256), ([0, 0, 5], 144, 136), ([40, 1, 0, 33], 400, 392),
    ([300, 7], 1040, 520), ([65, 130, 2], 128, 1000),
])
def test_product(gg, sizes, K, N, bm):
    rng = np.random.default_rng(K + N + len(sizes))
    _check(gg, _operands(rng, sizes, K, N, extra=3), bm)


def test_product_of_no_rows(gg):
    rng = np.random.default_rng(1)
    _check(gg, _operands(rng, [0, 0, 0], 144, 72, extra=4))
    empty = _operands(rng, [0, 0], 144, 72)
    assert gg.grouped_gemm_fp8_block(*_dev(empty)).shape == (0, 72)


def _exact_operands(rng, sizes, K, N, extra=0):
    """Codes of small whole numbers and scales that are powers of two: every sum is exact."""
    M, E = int(sum(sizes)) + extra, len(sizes)
    small = ref.to_e4m3(np.arange(-3, 4).astype(np.float64))
    slices, bands = -(-K // 128), -(-N // 128)
    return (small[rng.integers(0, 7, (M, K))], np.exp2(rng.integers(-2, 2, (slices, M))).astype(np.float32),
            small[rng.integers(0, 7, (E, N, K))], np.exp2(rng.integers(-2, 2, (E, bands, slices))).astype(np.float32),
            ops.offsets_of(sizes))


@pytest.mark.parametrize("bm,width", [(b, w) for b in BMS[1:] for w in (64, 128, 256) if b > 16 or w > 64])
def test_every_tile_exactly(gg, bm, width):
    # each height by its argument, each width by the number of tiles, K below, at and past the
    # ring's stages (64 columns need 32 rows)
    rng = np.random.default_rng(bm + width)
    for E, N in ((1, 264), (24, 264), (24, 1288), (28, 2056), (60, 264)):
        sizes = [int(m) for m in rng.integers(bm // 2 + 1, bm + 1, E)]
        if ring_schedule.tiles(sizes, N, bm)[0] == width:
            break
    else:
        raise AssertionError("no launch runs on this tile")
    stages = ring_schedule.stages(bm, width, False)
    for n in (1, stages - 1, stages, stages + 1, 10):
        args = _exact_operands(rng, sizes, 128 * n - (16 if n > 1 else 0), N)
        C = ref.fp8_product(*args, bounds=False)[0]
        got = gg.grouped_gemm_fp8_block(*_dev(args), bm=bm)
        assert (ops.host(got) == C).all(), (bm, width, n)
        got = gg.grouped_gemm_fp8_block(*_dev(args), bm=bm, out_dtype=torch.bfloat16)
        assert (ops.host(got) == oracle.round_to_bf16(C)).all(), (bm, width, n)


def test_many_tiles_a_workgroup(gg):
    rng = np.random.default_rng(11)
    args = _exact_operands(rng, [int(m) for m in rng.integers(0, 700, 30)], 400, 1288)
    assert (ops.host(gg.grouped_gemm_fp8_block(*_dev(args))) == ref.fp8_product(*args, bounds=False)[0]).all()


@pytest.mark.parametrize("sizes", [[256] * 100 + [1], [700] * 24 + [100] * 60 + [30] * 50, [64] * 300])
def test_rounds_of_tiles(gg, sizes):
    # three and more rounds of tiles on every workgroup, in one height and mixed: a tile's first
    # slice comes in behind the stores of the one before. One to eight slices, every output.
    rng = np.random.default_rng(len(sizes))
    N, M = 2056, sum(sizes)
    for K in (112, 256, 384, 1024):
        args = _dev(_exact_operands(rng, sizes, K, N))
        block, band = torch.arange(K, device=DEV) // 128, torch.arange(N, device=DEV) // 128
        a = args[0].view(F8).double() * args[1].t().double()[:, block]
        C, at = torch.empty(M, N, dtype=torch.float64, device=DEV), 0
        for e, m in enumerate(sizes):
            b = args[2][e].view(F8).double() * args[3][e].double()[band][:, block]
            C[at:at + m] = a[at:at + m] @ b.t()
            at += m
        for _ in range(3):
            assert torch.equal(gg.grouped_gemm_fp8_block(*args).double(), C), K
            assert torch.equal(gg.grouped_gemm_fp8_block(*args, out_dtype=torch.bfloat16), C.bfloat16()), K
            # the activation in fp32 is off by at most (|gate| + 3.5) 2^-23, then rounded to bf16
            gate, up = C[:, 0::2], C[:, 1::2]
            want = gate * torch.sigmoid(gate) * up
            off = (gg.grouped_gemm_fp8_block_swiglu(*args).double() - want).abs()
            assert (off <= (2.0 ** -8 + (gate.abs() + 4) * 2.0 ** -22) * want.abs() + 2.0 ** -100 * up.abs()).all(), K


def test_scales_are_any_numbers(gg):
    # 0, negative, subnormal-making and large ones; a NaN stays in its row or its 128 columns
    rng = np.random.default_rng(12)
    Aq, As, Bq, Bs, off = _exact_operands(rng, [20, 30], 256, 264)
    As[0, 3], As[1, 3], As[0, 4], As[1, 5] = 0.0, -1.5, 2.0 ** -90, 2.0 ** 100
    Bs[0, 1, 0], Bs[1, 2, 1] = -3.0, 2.0 ** -60
    As[1, 7], Bs[1, 1, 0] = np.nan, np.nan
    C = ref.fp8_product(Aq, As, Bq, Bs, off, bounds=False)[0]
    got = ops.host(gg.grouped_gemm_fp8_block(*_dev((Aq, As, Bq, Bs, off))))
    nan = np.isnan(C)
    assert nan[7].all() and nan[20:, 128:256].all() and nan.sum() == 264 + 30 * 128
    assert (np.isnan(got) == nan).all()
    # row 4 adds numbers 2^88 apart, one rounding of the larger
    assert (np.abs(got - C)[~nan] <= 2.0 ** -23 * np.abs(C)[~nan]).all()


# pairs of a row's and of the columns' scales: finite each, their product beyond fp32 or below its
# normal numbers, and the results of the codes' sums not
LARGE = [(2.0 ** 70, 2.0 ** 70), (1.37 * 2.0 ** 100, -1.2 * 2.0 ** 39), (1.9 * 2.0 ** 127, 1.1 * 2.0 ** 12), (-2.0 ** 13, 2.0 ** 127)]
SMALL = [(1.37 * 2.0 ** -75, 1.6 * 2.0 ** -74), (-1.1 * 2.0 ** -126, 1.3 * 2.0 ** -22), (1.2 * 2.0 ** -20, 1.7 * 2.0 ** -126),
         (2.0 ** -140, 1.4 * 2.0 ** -5), (1.5 * 2.0 ** -10, 2.0 ** -135), (2.0 ** -108, 2.0 ** -100)]


@pytest.mark.parametrize("bm", BMS)
@pytest.mark.parametrize("N", [264, 1288])
def test_scales_whose_product_is_beyond_fp32(gg, N, bm):
    # a first block of the least codes, zeros in a third of the rows and columns, at such scales, then
    # ordinary ones: the sums of 0 have to add 0, the others what the scales make of them
    rng = np.random.default_rng(N + bm)
    E, m, K = len(LARGE), 150, 400
    a, b = (rng.integers(-3, 4, shape).astype(np.float64) for shape in ((E * m, K), (E, N, K)))
    a[:, :128], b[:, :, :128] = 0, 0
    a[:, 5:9], b[:, :, 3:12] = (2.0 ** -9 * rng.integers(-1, 2, shape) for shape in ((E * m, 4), (E, N, 9)))
    a[::3, :128] = 0
    b[:, ::3, :128] = 0
    As, Bs = np.ones((4, E * m), np.float32), np.ones((E, -(-N // 128), 4), np.float32)
    for e, (row, column) in enumerate(LARGE):
        As[0, e * m:(e + 1) * m], Bs[e, :, 0] = row, column
    As[0, 7], As[3, 7] = 1.0, 2.0 ** 100  # and rows without one, or with one only
    Bs[1, 1, 0], Bs[2, 0, 3] = 0.0, 2.0 ** 40
    args = (ref.to_e4m3(a), As, ref.to_e4m3(b), Bs, ops.offsets_of([m] * E))
    C, S, G = ref.fp8_product(*args)
    assert np.abs(C).max() < 2.0 ** 127.9
    err = ref.fp8_product_error(S, G, K)
    got = gg.grouped_gemm_fp8_block(*_dev(args), bm=bm)
    ops.check_f32(ops.host(got), C, err, "fp32")
    ops.check_bf16(ops.host(gg.grouped_gemm_fp8_block(*_dev(args), bm=bm, out_dtype=torch.bfloat16)), C, err, "bf16")
    # where no block sum but the ordinary ones' counts, the results are theirs to the last bit (whole
    # numbers below 2^24, which fp32 adds exactly; the far scales of the last block give others)
    args[1][0], args[3][:, :, 0] = 1.0, 1.0
    plain = ref.fp8_product(*args, bounds=False)[0]
    zero = (np.arange(E * m) % 3 == 0)[:, None] | (np.arange(N) % 3 == 0)
    zero &= np.abs(plain) < 2 ** 24
    assert zero.sum() > E * m * N / 3 and (ops.host(got)[zero] == plain[zero]).all()


@pytest.mark.parametrize("sizes", [[256] * 100 + [1], [700] * 24 + [100] * 60 + [30] * 50, [64] * 300])
def test_repeated_blocks_in_rounds_of_tiles(gg, sizes):
    # blocks that are computed again in some tiles of several rounds, between a tile's last products and the
    # next one's first slices: a first block of zeros at scales whose product passes fp32, then whole numbers
    rng = np.random.default_rng(len(sizes))
    N, M, E = 2056, sum(sizes), len(sizes)
    for K in (144, 400, 1024):
        Aq, As, Bq, Bs, off = _exact_operands(rng, sizes, K, N)
        Aq[:, :128] = 0
        for far in (False, True):
            As[0], Bs[:, :, 0] = 1.0, 1.0
            if far:
                As[0, rng.integers(0, 40, M) == 0] = 2.0 ** 100
                Bs[rng.integers(0, 3, E) == 0, :, 0] = -2.0 ** 100
            args = _dev((Aq, As, Bq, Bs, off))
            got = [gg.grouped_gemm_fp8_block(*args), gg.grouped_gemm_fp8_block(*args, out_dtype=torch.bfloat16),
                   gg.grouped_gemm_fp8_block_swiglu(*args)]
            if not far:
                want = got
            for a, b in zip(got, want):
                assert torch.equal(a, b), (K, far)


@pytest.mark.parametrize("K", [128, 384])
def test_scales_whose_product_is_below_fp32(gg, K):
    # a product of scales below 2^-126 is off by 2^-150 at most, a block's sum is less than
    # 448 * 448 * 128 < 2^25: that much a block, and the usual besides
    rng = np.random.default_rng(K)
    E, N, m = len(SMALL), 264, 21
    a, b = (rng.integers(14, 29, shape) * 16.0 for shape in ((E * m, K), (E, N, K)))
    slices = -(-K // 128)
    As = np.repeat(np.array([p for p, _ in SMALL], dtype=np.float32), m)[None].repeat(slices, 0)
    Bs = np.array([p for _, p in SMALL], dtype=np.float32)[:, None, None] * np.ones((E, -(-N // 128), slices), np.float32)
    args = (ref.to_e4m3(a), As, ref.to_e4m3(b), Bs, ops.offsets_of([m] * E))
    C, S, G = ref.fp8_product(*args)
    got = gg.grouped_gemm_fp8_block(*_dev(args))
    ops.check_f32(ops.host(got), C, ref.fp8_product_error(S, G, K) + slices * 2.0 ** -125, "fp32")


def test_infinite_scales_are_the_formulas(gg):
    rng = np.random.default_rng(18)
    args = list(_exact_operands(rng, [20, 30], 256, 264))
    args[1][0, 3], args[1][1, 30], args[3][0, 1, 0] = np.inf, -np.inf, np.inf
    with np.errstate(invalid="ignore"):
        C = ref.fp8_product(*args, bounds=False)[0]
    got = ops.host(gg.grouped_gemm_fp8_block(*_dev(args)))
    assert np.isinf(C).any() and np.isnan(C).any() and same(got, C.astype(np.float32))


def test_rows_past_the_last_group_are_never_used(gg):
    rng = np.random.default_rng(13)
    args = list(_exact_operands(rng, [5, 6], 144, 72, extra=20))
    C = ref.fp8_product(*args, bounds=False)[0][:11]
    args[0][11:] = 0x7F  # NaN codes
    args[1][:, 11:] = np.nan
    assert (ops.host(gg.grouped_gemm_fp8_block(*_dev(args)))[:11] == C).all()


@pytest.mark.parametrize("off", [[0, 40, 20, 64], [5, 5, 70, 64], [-3, 10, 2 ** 31 - 1, 0]])
def test_malformed_offsets_stay_inside(gg, off):
    rng = np.random.default_rng(14)
    args = list(_exact_operands(rng, [20, 20, 24], 144, 72))
    args[4] = np.array(off, dtype=np.int64).astype(np.int32)
    guard = torch.full((64 + 32, 72), 7.0, device=DEV)
    d = _dev(args)
    gg.grouped_gemm_fp8_block(*d, out=guard[16:80])
    torch.cuda.synchronize()
    assert (guard[:16] == 7).all() and (guard[80:] == 7).all()


def test_uint8_codes_and_equal_bits(gg):
    rng = np.random.default_rng(15)
    d = _dev(_operands(rng, [70, 3, 50], 528, 264))
    a = gg.grouped_gemm_fp8_block(*d)
    f8 = [d[0].view(F8), d[1], d[2].view(F8), d[3], d[4]]
    for _ in range(3):
        assert torch.equal(a, gg.grouped_gemm_fp8_block(*f8))


def test_data_gradient(gg):
    # dA = dC B^T with the weights as they lie
    rng = np.random.default_rng(16)
    sizes, K, N = [33, 0, 70, 5], 200, 144
    b, dC = ops.bits(rng, 4, K, N, scale=0.1), _hot(rng, sum(sizes), N)
    off = ops.offsets_of(sizes)
    Wq, Ws = gg.fp8_quantize_weights(ops.to_dev(b), for_grad=True)
    dq, ds = gg.fp8_quantize(ops.to_dev(dC))
    got = ops.host(gg.grouped_gemm_fp8_block(dq, ds, Wq, Ws, ops.to_dev(off)))
    args = (*ref.fp8_rows(dC), *ref.fp8_weights(b, True), off)
    C, S, G = ref.fp8_product(*args)
    ops.check_f32(got, C, ref.fp8_product_error(S, G, N), "data gradient")
    # and near the gradient of the unrounded operands: 2 x 2^-4 relative a term, and what the
    # least codes lose (2^-10 of a block's largest value over 448 a factor)
    exact = np.concatenate([oracle._bf16_to_f64(dC[lo:hi]) @ oracle._bf16_to_f64(b[e]).T
                            for e, (lo, hi) in enumerate(zip(off[:-1], off[1:]))])
    assert np.linalg.norm(got - exact) < 2.0 ** -3 * np.linalg.norm(exact)


def test_weights_past_2_to_the_32_bytes(gg):
    E, K, N, sizes = 66, 8192, 8192, [0] * 64 + [3, 2]
    Bq = torch.zeros((E, N, K), dtype=torch.uint8, device=DEV)  # 4.4e9 bytes
    Bs = torch.ones((E, 64, 64), device=DEV)
    rng = np.random.default_rng(17)
    small = torch.from_numpy(ref.to_e4m3(np.arange(-1, 2).astype(np.float64))).to(DEV)
    for e in (0, 64, 65):
        Bq[e] = small[torch.randint(0, 3, (N, K), device=DEV)]
    Aq = small[torch.randint(0, 3, (5, K), device=DEV)]
    As = torch.from_numpy(np.exp2(rng.integers(-1, 2, (64, 5))).astype(np.float32)).to(DEV)
    got = gg.grouped_gemm_fp8_block(Aq, As, Bq, Bs, ops.to_dev(ops.offsets_of(sizes)))
    a = Aq.view(F8).double() * As.t().repeat_interleave(128, 1).double()
    want = torch.cat([a[:3] @ Bq[64].view(F8).double().t(), a[3:] @ Bq[65].view(F8).double().t()])
    assert torch.equal(got.double(), want)


def test_random_shapes(gg):
    for seed in range(40):
        rng = np.random.default_rng(1000 + seed)
        E = int(rng.integers(1, 20))
        sizes = [int(m) for m in rng.integers(0, int(rng.choice([3, 20, 150])), E)]
        K, N = 16 * int(rng.integers(1, 50)), 8 * int(rng.integers(1, 60))
        _check(gg, _operands(rng, sizes, K, N, extra=int(rng.integers(0, 5))), int(rng.choice(BMS)))
