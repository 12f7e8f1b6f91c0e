"""Every tile of the data gradient and the 4-bit product, with sums long enough that its
ring of LDS stages runs over (needs an MI355X).

``tests/ring_schedule.py`` says which launch runs on which tile; its tests hold that all
are reached. Inputs are small whole numbers (or 4-bit codes at scales of 1/2 to 2), so
that every partial sum is exact in fp32 and results are compared for equality with
binary64 products; the plain form decodes and multiplies expert by expert.
"""

import numpy as np
import pytest

import oracle
import oracle.operators as ref
from tests import operators as ops
from tests import parity
from tests import ring_schedule as rs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SPARE = 3  # rows past the last group


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(gen, *shape):
    return torch.randint(-3, 4, shape, generator=gen, device=DEV, dtype=torch.int8).bfloat16()


def _offsets(sizes):
    return torch.tensor(ops.offsets_of(sizes), dtype=torch.int32, device=DEV)


def _per_expert(rows, weights, sizes):
    """Binary64 products of each expert's rows with the transpose of its weights."""
    parts = rows[:sum(sizes)].double().split([int(m) for m in sizes])
    return torch.cat([a @ w.double().t().contiguous() for a, w in zip(parts, weights)])


def _check_exact(out, want, what):
    m = want.shape[0]
    assert torch.equal(out[:m], want.to(out.dtype)), what
    assert torch.isnan(out[m:]).all(), "%s: rows past the last group were written" % what


def _nan(rows, cols, dtype):
    return torch.full((rows, cols), float("nan"), device=DEV, dtype=dtype)


def _dgrad(gg, sizes, K, N, bm, seed):
    gen = _gen(seed)
    M = sum(sizes) + SPARE
    dC, B = _ints(gen, M, N), _ints(gen, len(sizes), K, N)
    want = _per_expert(dC, B, sizes)
    for dtype in (torch.float32, torch.bfloat16):
        out = _nan(M, K, dtype)
        gg.grouped_gemm_dgrad(dC, B, _offsets(sizes), out=out, bm=bm)
        _check_exact(out, want, "dgrad K=%d N=%d bm=%d %s" % (K, N, bm, dtype))


@pytest.mark.parametrize("height,width", rs.CONFIGS)
def test_dgrad_tiles(gg, height, width):
    sizes, K = rs.launch_for(height, width)
    for i, N in enumerate(rs.lengths_for(height, width, False)):
        _dgrad(gg, sizes, K, N, height, 10 * height + width + i)


def _codes(gen, sizes, K, N, a_lo=126):
    E, M, sl = len(sizes), sum(sizes) + SPARE, -(-K // 256)
    byte = lambda *shape: torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.uint8)  # noqa: E731
    scale = lambda lo, *shape: torch.randint(lo, lo + 3, shape, generator=gen, device=DEV, dtype=torch.uint8)  # noqa: E731
    Aq, a_s, Bq, b_s = byte(M, K // 2), scale(a_lo, sl, M, 8), byte(E, N, K // 2), scale(126, E, sl, N, 8)
    past = (torch.arange(sl * 8, device=DEV).view(sl, 1, 8) >= K // 32)
    return Aq, a_s.masked_fill(past, 255), Bq, b_s.masked_fill(past, 255)  # (ignored by every reader)


def _values(q, scale):
    grid = torch.tensor(np.concatenate([ref.E2M1, -ref.E2M1]), device=DEV)
    v = torch.stack([grid[(q & 15).int()], grid[(q >> 4).int()]], dim=-1).flatten(-2).unflatten(-1, (-1, 32))
    blocks = scale.transpose(-3, -2).flatten(-2)[..., :v.shape[-2]]
    return (v * torch.exp2(blocks.double() - 127)[..., None]).flatten(-2)


def _mx4_want(codes, sizes):
    Aq, a_s, Bq, b_s = codes
    return _per_expert(_values(Aq, a_s), [_values(q, s) for q, s in zip(Bq, b_s)], sizes)


def _mx4(gg, sizes, K, N, bm, seed):
    codes = _codes(_gen(seed), sizes, K, N)
    want = _mx4_want(codes, sizes)
    for dtype in (torch.float32, torch.bfloat16):
        out = _nan(codes[0].shape[0], N, dtype)
        gg.grouped_gemm_mx4(*codes, _offsets(sizes), out=out, bm=bm)
        _check_exact(out, want, "mx4 K=%d N=%d bm=%d %s" % (K, N, bm, dtype))
    return codes, want


@pytest.mark.parametrize("height,width", rs.CONFIGS)
def test_mx4_tiles(gg, height, width):
    sizes, N = rs.launch_for(height, width)
    for i, K in enumerate(rs.lengths_for(height, width, True)):
        _mx4(gg, sizes, K, N, height, 10 * height + width + i)


HEIGHTS = [300, 20, 0, 700, 64, 130]


@pytest.mark.parametrize("copies", [1, 3, 4, 6, 12])
def test_long_sums_at_mixed_heights(gg, copies):
    sizes = HEIGHTS * copies
    width, heights, _ = rs.tiles(sizes, 1032)
    assert width == {1: 64, 3: 128, 4: 256, 6: 128, 12: 256}[copies] and len(heights) == 4
    _dgrad(gg, sizes, 1032, 680, 0, copies)
    _mx4(gg, sizes, 2016, 1032, 0, copies)


SMALL = 119  # row scales for gates of a few units, where the activation bends


def _mx4_swiglu(gg, codes, want, sizes, K, N, bm, what):
    # the product is exact; the reference's error allowance covers the activation alone
    M = codes[0].shape[0]
    guard = torch.full((M * (N // 2) + 64,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = guard[:M * (N // 2)].view(M, N // 2)
    gg.grouped_gemm_mx4_swiglu(*codes, _offsets(sizes), out=out, bm=bm)
    got, c = ops.host(out), want.cpu().numpy()
    parity.check_swiglu_bf16(got[:len(c)], c, np.abs(c), what, err=np.zeros_like(c))
    assert (got[len(c):] == -7).all() and (guard[M * (N // 2):] == -7).all()


@pytest.mark.parametrize("height,width", rs.CONFIGS)
def test_mx4_swiglu_tiles(gg, height, width):
    sizes, N = rs.launch_for(height, width)
    K = rs.lengths_for(height, width, True)[-2]
    codes = _codes(_gen(height + width), sizes, K, N, SMALL)
    _mx4_swiglu(gg, codes, _mx4_want(codes, sizes), sizes, K, N, height, "swiglu %d x %d" % (height, width))


@pytest.mark.parametrize("N", range(1032, 1081, 8))
def test_mx4_swiglu_last_columns_of_wide_tiles(gg, N):
    # 8 columns past a block of 16 (and none) at every place of a wave's 64, on tiles whose
    # waves hold four blocks side by side and store 16 bytes a lane
    sizes = [300, 5] * 40
    for bm in (0, 256):
        width, heights, _ = rs.tiles(sizes, N, bm)
        assert width == 256 and (128 if bm == 0 else 256) in heights
        codes = _codes(_gen(N), sizes, 288, N, SMALL)
        want = _mx4_want(codes, sizes)
        _mx4_swiglu(gg, codes, want, sizes, 288, N, bm, "swiglu N=%d bm=%d" % (N, bm))
        out = _nan(codes[0].shape[0], N, torch.bfloat16)
        gg.grouped_gemm_mx4(*codes, _offsets(sizes), out=out, bm=bm)
        _check_exact(out, want, "bf16 N=%d bm=%d" % (N, bm))


@pytest.mark.parametrize("copies", [1, 3, 4, 6, 12])
def test_mx4_swiglu_at_mixed_heights(gg, copies):
    sizes = HEIGHTS * copies
    codes = _codes(_gen(copies), sizes, 544, 1032, SMALL)
    _mx4_swiglu(gg, codes, _mx4_want(codes, sizes), sizes, 544, 1032, 0, "copies %d" % copies)


def _dgrad_swiglu(gg, sizes, K, N, bm, seed):
    gen = _gen(seed)
    m, M = sum(sizes), sum(sizes) + SPARE
    dY, B, off = _ints(gen, M, N), _ints(gen, len(sizes), K, N), _offsets(sizes)
    C = (2 * torch.randn((M, 2 * K), generator=gen, device=DEV)).bfloat16()
    dh = _per_expert(dY, B, sizes).cpu().numpy()  # exact in the kernel too
    c64 = C[:m].double().cpu().numpy()
    want, want_h = ref.swiglu_grad(dh, c64)
    err, err_h = ref.swiglu_grad_error(dh, 0.0, c64)
    what = "dgrad_swiglu K=%d N=%d bm=%d" % (K, N, bm)
    d, H = _nan(M, 2 * K, torch.bfloat16), _nan(M, K, torch.bfloat16)
    gg.grouped_gemm_dgrad_swiglu(dY, B, off, C, out=d, out_h=H, bm=bm)
    ops.check_bf16(ops.host(d[:m]), want, err, what)
    ops.check_bf16(ops.host(H[:m]), want_h, err_h, what + " H")
    assert torch.isnan(d[m:]).all() and torch.isnan(H[m:]).all(), what
    # without H, and in place: the same bits
    alone = _nan(M, 2 * K, torch.bfloat16)
    gg.grouped_gemm_dgrad_swiglu(dY, B, off, C, out=alone, bm=bm)
    assert torch.equal(alone[:m], d[:m]) and torch.isnan(alone[m:]).all(), what
    spare = C[m:].clone()
    H.fill_(float("nan"))
    gg.grouped_gemm_dgrad_swiglu(dY, B, off, C, out=C, out_h=H, bm=bm)
    assert torch.equal(C[:m], d[:m]) and torch.equal(C[m:], spare), what
    ops.check_bf16(ops.host(H[:m]), want_h, err_h, what + " H in place")


@pytest.mark.parametrize("height,width", rs.CONFIGS)
def test_dgrad_swiglu_tiles(gg, height, width):
    sizes, K = rs.launch_for(height, width)
    _dgrad_swiglu(gg, sizes, K, rs.lengths_for(height, width, False)[-2], height, height + width)


@pytest.mark.parametrize("copies", [1, 3, 4, 6, 12])
def test_dgrad_swiglu_at_mixed_heights(gg, copies):
    _dgrad_swiglu(gg, HEIGHTS * copies, 1032, 328, 0, copies)


def _many(E, seed, tall_at):
    # small groups with empty ones among them; tall ones where tall_at says
    sizes = np.random.default_rng(seed).integers(0, 24, size=E) * np.random.default_rng(seed + 1).integers(0, 2, size=E)
    for e, m in tall_at.items():
        sizes[e] = m
    return sizes.tolist()


# the schedule gives two experts to a thread: 128 to a wave
MANY = {
    # two waves and a bit, several rounds, tall experts in the last waves
    "129": (_many(129, 1, {128: 700, 3: 300}), 1032),
    "300": (_many(300, 2, {131: 300, 140: 700, 298: 130, 299: 517}), 1032),
    "1024": (_many(1024, 3, {0: 130, 511: 300, 640: 700, 1022: 20, 1023: 517}), 520),
    # one round, its only rows behind the first wave: heights cut for idle CUs
    "sparse": ([0] * 200 + [700] + [0] * 300 + [20] + [0] * 521 + [5], 72),
    "last": ([0] * 1023 + [1], 136),
    "equal": ([16] * 1024, 136),
}


@pytest.mark.parametrize("bm", [0, 16, 128])
@pytest.mark.parametrize("case", MANY)
def test_more_experts_than_one_wave_holds(gg, case, bm):
    sizes, cols = MANY[case]
    if bm == 0:
        width, heights, G = rs.tiles(sizes, cols)
        rounds = sum(heights.values()) * -(-cols // width) / G
        assert (rounds > 1 and len(heights) > 2) == (case in ("129", "300", "1024"))
    _dgrad(gg, sizes, cols, 200, bm, 1)
    codes, want = _mx4(gg, sizes, 544, cols, bm, 2)
    out = _nan(codes[0].shape[0], cols // 2, torch.bfloat16)
    gg.grouped_gemm_mx4_swiglu(*codes, _offsets(sizes), out=out, bm=bm)
    m = sum(sizes)
    gate, up = want[:, 0::2], want[:, 1::2]
    # (fp32 activation of exact columns: |gate| + 4 units of 2^-22, then one rounding to bf16)
    h = gate * torch.sigmoid(gate) * up
    bound = (2.0 ** -8 + (gate.abs() + 4) * 2.0 ** -22) * h.abs() + 2.0 ** -100 * up.abs()
    assert ((out[:m].double() - h).abs() <= bound).all() and torch.isnan(out[m:]).all()
    _dgrad_swiglu(gg, sizes, cols, 136, bm, 3)


def test_weights_beyond_4_gigabytes(gg):
    # the last expert's weights, its gradient and its codes lie past 2^32 bytes
    E, K, N, rows = 34, 8192, 8448, 37
    sizes = [0] * (E - 2) + [5, rows]
    gen, off, m = _gen(1), _offsets(sizes), 5 + rows
    B = torch.randint(-3, 4, (E, K, N), generator=gen, device=DEV, dtype=torch.int8).bfloat16()
    assert B[-1].data_ptr() - B.data_ptr() > 2 ** 32
    dC, A = _ints(gen, m, N), _ints(gen, m, K)
    want = torch.cat([dC[:5].double() @ B[-2].double().t().contiguous(), dC[5:].double() @ B[-1].double().t().contiguous()])
    assert torch.equal(gg.grouped_gemm_dgrad(dC, B, off).double(), want)
    # the quantisers: each expert as it is alone
    q, s = gg.mx4_quantize_weights(B)
    for e in (0, E - 1):
        q1, s1 = gg.mx4_quantize_weights(B[e:e + 1])
        assert torch.equal(q[e], q1[0]) and torch.equal(s[e], s1[0])
    del B
    back = gg.mx4_dequantize(q, s)
    assert torch.equal(back[-1], _values(q[-1], s[-1]).bfloat16()) and torch.equal(back[1], _values(q[1], s[1]).bfloat16())
    del back, q, s
    dB = gg.grouped_gemm_wgrad(A, dC, off)
    assert dB[-1].data_ptr() - dB.data_ptr() > 2 ** 32
    for e, lo, hi in ((E - 2, 0, 5), (E - 1, 5, m)):
        assert torch.equal(dB[e].double(), A[lo:hi].double().t().contiguous() @ dC[lo:hi].double())
    assert not dB[:E - 2].any()
    del dB
    torch.cuda.empty_cache()
    # 4-bit codes: four times as many weights
    E, K, N = 33, 16384, 16896
    sizes = [0] * (E - 1) + [rows]
    Aq, a_s, _, _ = _codes(gen, sizes, K, 8)
    Bq = torch.randint(0, 256, (E, N, K // 2), generator=gen, device=DEV, dtype=torch.uint8)
    b_s = torch.full((E, K // 256, N, 8), 126, dtype=torch.uint8, device=DEV)
    assert Bq[-1].data_ptr() - Bq.data_ptr() > 2 ** 32
    a_s.fill_(127)  # products of up to 18 in steps of 1/8: sums of fewer than 2^22 steps
    got = gg.grouped_gemm_mx4(Aq, a_s, Bq, b_s, _offsets(sizes))[:rows]
    want = _values(Aq[:rows], a_s[:, :rows]) @ _values(Bq[-1], b_s[-1]).t().contiguous()
    assert torch.equal(got.double(), want)
    del Bq, b_s, want
    torch.cuda.empty_cache()
