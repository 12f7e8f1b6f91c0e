"""4-bit microscaled operators on the GPU against binary64 (needs an MI355X)."""

import numpy as np
import pytest

import oracle
import oracle.operators as ref
import workloads as wl
from tests import operators as ops
from tests import parity

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BMS = [0, 16, 32, 64, 128, 256]


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
    x[..., : min(32, shape[-1])] *= rng.integers(0, 2, size=shape[:-1] + (1,))
    return wl.f32_to_bf16_bits(x.astype(np.float32))


@pytest.mark.parametrize("M,K", [(1, 32), (1, 8192), (3, 224), (17, 256), (129, 1056), (64, 288), (5, 6144)])
def test_quantize_rows(gg, M, K):
    x = _hot(np.random.default_rng(M * K), M, K)
    q, s = gg.mx4_quantize(ops.to_dev(x))
    want_q, want_s = ref.mx4_encode(x)
    assert (ops.host(s) == want_s).all()
    assert (ops.host(q) == want_q).all()
    assert (ops.host(gg.mx4_dequantize(q, s)) == ref.mx4_values(want_q, want_s)).all()


@pytest.mark.parametrize("E,K,N", [(1, 32, 8), (3, 224, 40), (2, 256, 256), (2, 1056, 264), (5, 288, 776)])
def test_quantize_weights(gg, E, K, N):
    b = _hot(np.random.default_rng(E * K + N), E, K, N)
    q, s = gg.mx4_quantize_weights(ops.to_dev(b))
    want_q, want_s = ref.mx4_encode(np.ascontiguousarray(np.swapaxes(b, 1, 2)))
    assert (ops.host(s) == want_s).all()
    assert (ops.host(q) == want_q).all()
    assert (ops.host(gg.mx4_dequantize(q, s)) == ref.mx4_values(want_q, want_s)).all()


def test_quantize_every_bf16_value(gg):
    # every finite magnitude beside its neighbours, under a block maximum 0 to 4
    # binades above them (so that the steps fall everywhere in a binade), the
    # signs in turn; then alone in its block
    mags = np.arange(0x7F80, dtype=np.uint16)
    mags = np.concatenate([mags, np.zeros(-len(mags) % 31, dtype=np.uint16)]).reshape(-1, 31)
    blocks = []
    for up in range(5):
        top = np.minimum(mags.max(axis=1) + (up << 7), 0x7F7F).astype(np.uint16)
        blocks.append(np.concatenate([mags, top[:, None]], axis=1))
    blocks.append(np.repeat(np.arange(0x7F80, dtype=np.uint16)[:, None], 32, axis=1))
    x = np.concatenate(blocks)
    x[:, 1::2] |= 0x8000
    x[1::2] ^= 0x8000
    q, s = gg.mx4_quantize(ops.to_dev(x))
    want_q, want_s = ref.mx4_encode(x)
    assert (ops.host(s) == want_s).all()
    assert (ops.host(q) == want_q).all()
    assert (ops.host(gg.mx4_dequantize(q, s)) == ref.mx4_values(want_q, want_s)).all()


def test_quantize_ties_go_to_even(gg):
    # scale 1 (block maximum 4): the borders 0.25 .. 5 and their neighbours
    vals = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.96875, 6.0, 0.251953125, 0.2490234375, -0.25, -0.75,
            -0.0, 0.0, -7.0, 1e-30, -1e-30] + [0.0] * 13
    x = wl.f32_to_bf16_bits(np.array([vals], dtype=np.float32))
    q, s = gg.mx4_quantize(ops.to_dev(x))
    got = ops.host(gg.mx4_dequantize(q, s))[0]
    assert ops.host(s)[0, 0, 0] == 127
    assert got[:10].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6, 6]
    assert got[10:14].tolist() == [0.5, 0, 0, -1]


def test_nonfinite_blocks_stand_for_nan(gg):
    rng = np.random.default_rng(2)
    x = ops.bits(rng, 6, 96)
    x[1, 40] = 0x7F80
    x[2, 0] = 0xFF80
    x[3, 95] = 0x7FC0
    q, s = gg.mx4_quantize(ops.to_dev(x))
    want_q, want_s = ref.mx4_encode(x)
    assert (ops.host(q) == want_q).all() and (ops.host(s) == want_s).all()
    v = ops.host(gg.mx4_dequantize(q, s)).reshape(6, 3, 32)
    bad = np.zeros((6, 3), dtype=bool)
    bad[1, 1] = bad[2, 0] = bad[3, 2] = True
    assert np.isnan(v[bad]).all() and np.isfinite(v[~bad]).all()


def test_dequantize_every_code_and_scale(gg):
    # 256 scale bytes x 16 codes, a block each
    q = np.repeat(np.arange(16, dtype=np.uint8)[None, :] * 17, 256, axis=0)  # K = 32: every code twice
    s = np.zeros((1, 256, 8), dtype=np.uint8)
    s[0, :, 0] = np.arange(256)
    got = ops.host(gg.mx4_dequantize(ops.to_dev(q), ops.to_dev(s))).astype(np.float64)
    want = ref.mx4_values(q, s)
    over = np.abs(want) >= 2.0 ** 128
    assert np.isinf(got[over]).all() and (np.sign(got[over]) == np.sign(want[over])).all()
    assert np.isnan(got[255]).all()
    ok = ~over & ~np.isnan(want)
    assert (got[ok] == want[ok]).all()


def _codes(rng, sizes, K, N, lo=120, hi=135, spare=3):
    off = ops.offsets_of(sizes)
    M, E = int(off[-1]) + spare, len(sizes)
    sl = -(-K // 256)
    u8 = np.uint8
    Aq, Bq = rng.integers(0, 256, (M, K // 2)).astype(u8), rng.integers(0, 256, (E, N, K // 2)).astype(u8)
    a_s, b_s = rng.integers(lo, hi, (sl, M, 8)).astype(u8), rng.integers(lo, hi, (E, sl, N, 8)).astype(u8)
    # bytes past the last block are ignored, whatever they are
    used = np.arange(sl * 8).reshape(sl, 1, 8) < K // 32
    a_s = np.where(used, a_s, u8(255))
    b_s = np.where(used[None], b_s, u8(255))
    return off, Aq, a_s, Bq, b_s


# K that ends after 1 .. 7 blocks of a slice and in several slices; N below, at
# and past a tile; empty and one-row experts, odd first rows
SHAPES = [([0, 1, 17, 130, 0, 300], 352, 392), ([5], 32, 8), ([1], 64, 136), ([16, 16, 16], 96, 1032),
          ([300, 0, 45, 517], 800, 264), ([0, 0, 3], 1056, 520), ([33, 64, 65, 2], 512, 128), ([1, 1, 2], 2080, 24)]


@pytest.mark.parametrize("bm", BMS)
@pytest.mark.parametrize("sizes,K,N", SHAPES)
def test_product(gg, sizes, K, N, bm):
    off, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(K + N), sizes, K, N)
    M = int(off[-1])
    want, S = (t[:M] for t in ref.mx4_product(Aq, a_s, Bq, b_s, off))
    err = ops.sum_bound(K // 32, S)
    dev = [ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off)]
    what = "mx4 %s K=%d N=%d bm=%d" % (sizes, K, N, bm)
    nan = float("nan")
    for dt, check in ((torch.float32, ops.check_f32), (torch.bfloat16, ops.check_bf16)):
        out = torch.full((Aq.shape[0], N), nan, dtype=dt, device="cuda:0")
        gg.grouped_gemm_mx4(*dev, out=out, bm=bm)
        got = ops.host(out)
        check(got[:M], want, err, what)
        assert np.isnan(got[M:]).all()
    out = torch.full((Aq.shape[0], N // 2), nan, dtype=torch.bfloat16, device="cuda:0")
    gg.grouped_gemm_mx4_swiglu(*dev, out=out, bm=bm)
    got = ops.host(out)
    parity.check_swiglu_bf16(got[:M], want, S, what + " swiglu", err=err)
    assert np.isnan(got[M:]).all()


@pytest.mark.parametrize("bm", BMS)
def test_product_exact(gg, bm):
    # scales between 1/2 and 2: every partial sum is a multiple of 1/16 below 2^20
    off, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(3), [40, 0, 1, 129], 544, 264, 126, 129)
    M = int(off[-1])
    got = ops.host(gg.grouped_gemm_mx4(*(ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off)), bm=bm))
    want, _ = ref.mx4_product(Aq, a_s, Bq, b_s, off)
    assert (got[:M] == want[:M]).all()


@pytest.mark.parametrize("copies", [1, 3, 6, 12])
def test_heights_of_a_launch(gg, copies):
    # heights of 16 to 256 together, from a few tiles to several rounds of the widest;
    # exact as above
    sizes = [300, 20, 0, 700, 64, 130] * copies
    off, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(copies), sizes, 288, 1032, 126, 129)
    M = int(off[-1])
    got = ops.host(gg.grouped_gemm_mx4(*(ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off))))
    want, _ = ref.mx4_product(Aq, a_s, Bq, b_s, off)
    assert (got[:M] == want[:M]).all()


def test_product_nan_scales_stay_in_their_row_and_column(gg):
    off, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(4), [20, 30], 288, 136)
    a_s[0, 7, 3] = 255   # row 7
    a_s[1, 50:, 0] = 255  # rows behind the last group
    b_s[1, 1, 100, 0] = 255  # expert 1's column 100
    for bm in BMS:
        got = ops.host(gg.grouped_gemm_mx4(*(ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off)), bm=bm))[:50]
        bad = np.zeros((50, 136), dtype=bool)
        bad[7] = True
        bad[20:, 100] = True
        assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_product_extreme_scales(gg):
    # the smallest and the largest scale bytes meet: 2^-127 * 2^127
    off, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(5), [17], 64, 24)
    a_s[:, :, :2] = 0
    b_s[:, :, :, :2] = 254
    got = ops.host(gg.grouped_gemm_mx4(*(ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off))))[:17]
    want, _ = ref.mx4_product(Aq, a_s, Bq, b_s, off)
    assert (got == want[:17]).all()


def test_single_token_widths(gg):
    # few rows and few columns up to many experts: the narrow, the plain and the
    # wide 16-row tiles
    for sizes, N in (([1], 4096), ([1] * 8, 2688), ([4] * 24, 2688), ([16] * 40, 4096)):
        off, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(N), sizes, 288, N, 126, 129, spare=0)
        got = ops.host(gg.grouped_gemm_mx4(*(ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off))))
        want, _ = ref.mx4_product(Aq, a_s, Bq, b_s, off)
        assert (got == want).all()


@pytest.mark.parametrize("offs", [[0, 9, 4, 30], [-5, 10, 20, 30], [0, 10, 99, 30], [30, 20, 10, 0]])
def test_malformed_offsets_stay_inside(gg, offs):
    _, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(6), [30, 0, 0], 96, 136, spare=0)
    dev = [ops.to_dev(t) for t in (Aq, a_s, Bq, b_s)]
    off = torch.tensor(offs, dtype=torch.int32, device="cuda:0")
    for bm in (0, 16, 256):
        buf = torch.full((94, 136), -7.0, device="cuda:0")
        gg.grouped_gemm_mx4(*dev, off, out=buf[32:62], bm=bm)
        assert (buf[:32] == -7).all() and (buf[-32:] == -7).all()


def test_swiglu_last_columns(gg):
    # 8 columns past a block of 16 in every place of a wave's 64
    for N in (8, 24, 40, 56, 72, 264, 280, 296, 312):
        off, Aq, a_s, Bq, b_s = _codes(np.random.default_rng(N), [300, 5], 96, N, spare=1)
        dev = [ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off)]
        want, S = (t[:305] for t in ref.mx4_product(Aq, a_s, Bq, b_s, off))
        for bm in (0, 256):
            buf = torch.full((306 * (N // 2) + 16,), -7.0, dtype=torch.bfloat16, device="cuda:0")
            gg.grouped_gemm_mx4_swiglu(*dev, out=buf[:306 * (N // 2)].view(306, N // 2), bm=bm)
            got = ops.host(buf)
            parity.check_swiglu_bf16(got[:305 * (N // 2)].reshape(305, -1), want, S, "N=%d" % N,
                                     err=ops.sum_bound(3, S))
            assert (got[305 * (N // 2):] == -7).all()


def test_rows_beyond_4_gigabytes(gg):
    # the last group's codes lie past 2^32 bytes, a slice's scales 2^24 apart
    M, K, N, last = 2_150_000, 4096, 24, 40
    rng = np.random.default_rng(9)
    off, tq, ts, Bq, b_s = _codes(rng, [last, 0], K, N, 126, 129, spare=0)
    Aq = torch.zeros((M, K // 2), dtype=torch.uint8, device="cuda:0")
    a_s = torch.full((K // 256, M, 8), 127, dtype=torch.uint8, device="cuda:0")
    Aq[M - last:] = ops.to_dev(tq)
    a_s[:, M - last:] = ops.to_dev(ts)
    offs = torch.tensor([0, M - last, M], dtype=torch.int32, device="cuda:0")
    got = gg.grouped_gemm_mx4(Aq, a_s, ops.to_dev(Bq[::-1].copy()), ops.to_dev(b_s[::-1].copy()), offs)
    want, _ = ref.mx4_product(tq, ts, Bq, b_s, off)
    assert (ops.host(got[M - last:]) == want).all() and not got[:M - last].any()
    # and there and back through the quantiser
    back = gg.mx4_quantize(gg.mx4_dequantize(Aq, a_s))
    tail = gg.mx4_quantize(gg.mx4_dequantize(ops.to_dev(tq), ops.to_dev(ts)))
    assert torch.equal(back[0][M - last:], tail[0]) and torch.equal(back[1][:, M - last:], tail[1])
    del Aq, a_s, got, back
    torch.cuda.empty_cache()


def test_longest_rows(gg):
    # K at its limit: values -1, 0 and 1 (codes 0 and +-4, scale 1/4), whose sums are exact
    rows, K, N = 3, 2 ** 22, 264
    g = torch.Generator(device="cuda:0").manual_seed(3)
    x = torch.randint(-1, 2, (rows, K), generator=g, device="cuda:0", dtype=torch.int8).to(torch.bfloat16)
    w = torch.randint(-1, 2, (1, K, N), generator=g, device="cuda:0", dtype=torch.int8).to(torch.bfloat16)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda:0")
    a, b = gg.mx4_quantize(x), gg.mx4_quantize_weights(w)
    assert torch.equal(gg.mx4_dequantize(*a), x)
    assert torch.equal(gg.mx4_dequantize(*b)[0], w[0].t())
    want = x.float() @ w[0].float()
    for bm in (0, 256):
        assert torch.equal(gg.grouped_gemm_mx4(*a, *b, off, bm=bm), want)
    del x, w, a, b
    torch.cuda.empty_cache()


def test_serving_a_layer(gg):
    # a layer's weights laid out once, then rows through quantise -> gate/up with
    # SwiGLU -> quantise -> down, against the same steps in binary64
    rng = np.random.default_rng(7)
    sizes, D, I = [3, 0, 40, 1], 288, 160
    off = ops.offsets_of(sizes)
    M, E = int(off[-1]), len(sizes)
    X = _hot(rng, M, D)
    B1, B2 = ops.bits(rng, E, D, 2 * I, scale=D ** -0.5), ops.bits(rng, E, I, D, scale=I ** -0.5)
    w1, w2 = (gg.mx4_quantize_weights(ops.to_dev(b)) for b in (B1, B2))
    toff = ops.to_dev(off)
    xq, xs = gg.mx4_quantize(ops.to_dev(X))
    H = gg.grouped_gemm_mx4_swiglu(xq, xs, *w1, toff)
    hq, hs = gg.mx4_quantize(H)
    Y = ops.host(gg.grouped_gemm_mx4(hq, hs, *w2, toff))

    enc = lambda b: ref.mx4_encode(np.ascontiguousarray(np.swapaxes(b, 1, 2)))  # noqa: E731
    c, S = ref.mx4_product(*ref.mx4_encode(X), *enc(B1), off)
    parity.check_swiglu_bf16(ops.host(H), c, S, "H", err=ops.sum_bound(D // 32, S))
    # H is taken as the kernel rounded it: a value next to a border may go to either side
    y, S = ref.mx4_product(*ref.mx4_encode(ops.bits_of(H)), *enc(B2), off)
    ops.check_f32(Y, y, ops.sum_bound(I // 32, S), "Y")


def test_graph_replays_follow_the_offsets(gg):
    K, N, M = 288, 264, 96
    sets = [([90, 0, 6], 1), ([0, 96, 0], 2), ([30, 31, 35], 3)]
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda:0")
    B = torch.zeros((3, K, N), dtype=torch.bfloat16, device="cuda:0")
    off = torch.zeros(4, dtype=torch.int32, device="cuda:0")

    def step():
        xq, xs = gg.mx4_quantize(X)
        bq, bs = gg.mx4_quantize_weights(B)
        return (xq, xs, bq, bs, gg.grouped_gemm_mx4(xq, xs, bq, bs, off),
                gg.grouped_gemm_mx4_swiglu(xq, xs, bq, bs, off), gg.mx4_dequantize(bq, bs))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for sizes, seed in sets * 2:
        r = np.random.default_rng(seed)
        X.copy_(ops.to_dev(ops.bits(r, M, K)))
        B.copy_(ops.to_dev(ops.bits(r, 3, K, N)))
        off.copy_(ops.to_dev(ops.offsets_of(sizes)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want)


def test_other_stream(gg):
    r = np.random.default_rng(8)
    off, Aq, a_s, Bq, b_s = _codes(r, [50, 14], 288, 264, spare=0)
    dev = [ops.to_dev(t) for t in (Aq, a_s, Bq, b_s, off)]
    X = ops.to_dev(ops.bits(r, 64, 288))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    on_s = [gg.grouped_gemm_mx4(*dev, stream=st), *gg.mx4_quantize(X, stream=st)]
    st.synchronize()
    for got, want in zip(on_s, (gg.grouped_gemm_mx4(*dev), *gg.mx4_quantize(X))):
        assert torch.equal(got, want)
