"""What surrounds the experts' products, without a GPU: the references against the formulas
by hand and by differences, the library's host checks, and the build."""

import os
import re
import subprocess

import numpy as np
import pytest

import moe_ragged_grouped_amd as gg
import moe_ragged_grouped_amd.build as hb
import oracle
import oracle.layer as ref
import workloads as wl
from tests import operators as ops
from tests.test_operators import BIG, _fake, _inner_loops

torch = pytest.importorskip("torch")
INVALID, MISALIGNED, UNSUPPORTED, NO_DEVICE = 1, 2, 3, 4


# ------------------------------------------------------------- the references

def test_e4m3_reference_by_hand():
    # the format's own values, and ties: 448 = 1.75 * 2^8, steps of 32 there; 2^-9 the least
    y = np.array([448, 449, 1e9, 432, 400, 416, 1.0, 1.0625, 1.1875, -2 ** -9, 2 ** -10, 3 * 2 ** -10, 0, -0.0])
    want = np.array([448, 448, 448, 448, 384, 416, 1, 1, 1.25, -2 ** -9, 0, 2 ** -8, 0, 0])
    got = oracle.decode_e4m3(ref.to_e4m3(y)).astype(np.float64)
    assert (got == want).all(), got


def test_e4m3_reference_is_torchs():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.standard_normal(4000) * np.exp(3 * rng.standard_normal(4000)),
                        (ref.GRID[1:] + ref.GRID[:-1]) / 2, ref.GRID]).astype(np.float32)
    y = np.clip(np.concatenate([y, -y]), -448, 448)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ref.to_e4m3(y.astype(np.float64)) == want).all()


def test_fp8_blocks_by_hand():
    x = np.zeros((2, 144), np.float32)
    x[0, 0], x[0, 1], x[0, 128], x[1, 5] = 448, -7, 2.0 ** -120, 1
    q, s = ref.fp8_rows(wl.f32_to_bf16_bits(x))
    assert s.shape == (2, 2) and s[0, 0] == 1 and s[0, 1] == np.float32(1 / 448)
    assert s[1, 0] == s[1, 1] == np.float32(2.0 ** -100 / 448)
    v = ref.fp8_row_values(q, s)
    assert v[0, 0] == 448 and v[0, 1] == -7 and v[1, 5] == float(np.float32(1 / 448)) * 448.0
    assert v[0, 128] == 0  # 448 * 2^-20: below half the least code at the least scale
    x[1, 6] = np.inf
    q, s = ref.fp8_rows(wl.f32_to_bf16_bits(x))
    assert np.isnan(s[0, 1]) and not np.isnan(s[1, 1]) and (q[1] == 0).all() and s[0, 0] == 1


def test_fp8_values_are_near():
    rng = np.random.default_rng(1)
    x = ops.bits(rng, 7, 400, scale=3.0)
    v = ref.fp8_row_values(*ref.fp8_rows(x))
    exact = oracle._bf16_to_f64(x)
    tops = np.repeat(ref._tops(exact, 1), 128, axis=1)[:, :400]
    # half a step of 2^-3 relative, of the least step (2^-9 at 448 for the largest), and
    # the scale's rounding
    assert (np.abs(v - exact) <= np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * tops / 447) * 1.001).all()


def test_weights_both_ways_hold_the_same_values():
    b = ops.bits(np.random.default_rng(2), 2, 160, 272)
    q, s = ref.fp8_weights(b)
    qg, sg = ref.fp8_weights(b, for_grad=True)
    assert (np.swapaxes(q, 1, 2) == qg).all() and (np.swapaxes(s, 1, 2) == sg).all()


def test_sort_reference_by_hand():
    e = np.array([[2, 0], [0, 5], [-1, 2], [2, 1]])
    w = np.arange(8, dtype=np.float32).reshape(4, 2)
    off, rows, pos, rw = ref.sort(e, 3, w)
    assert off.tolist() == [0, 2, 3, 6] and rows.tolist() == [0, 1, 3, 0, 2, 3, -1, -1]
    assert pos.tolist() == [[3, 0], [1, -1], [-1, 4], [5, 2]] and rw.tolist() == [1, 2, 7, 0, 5, 6, 0, 0]


def test_combine_gradient_by_differences():
    rng = np.random.default_rng(3)
    T, k, M, N = 4, 3, 9, 5
    pos = rng.permutation(T * k).reshape(T, k)  # some are past the rows
    y, w, dO = rng.standard_normal((M, N)), rng.standard_normal((T, k)), rng.standard_normal((T, N))
    dY, dw, _ = ref.combine_grad(dO, y, pos, w)
    f = lambda y_, w_: (ref.combine(y_, pos, w_)[0] * dO).sum()  # noqa: E731
    h = 1e-5
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((f(y, w + d) - f(y, w - d)) / (2 * h) - dw[i]) < 1e-8
    for i in np.ndindex(y.shape):
        d = np.zeros_like(y)
        d[i] = h
        assert abs((f(y + d, w) - f(y - d, w)) / (2 * h) - (dY[i] if np.isfinite(dY[i]) else 0.0)) < 1e-8
    # the gradient of spreading is the combine without weights
    x = rng.standard_normal((T, N))
    dS = rng.standard_normal((M, N))
    g = ref.combine(dS, pos, np.ones((T, k)))[0]
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        up, dn = (np.nansum(ref.spread(x + s * d, pos, np.zeros((M, N))) * dS) for s in (1, -1))
        assert abs((up - dn) / (2 * h) - g[i]) < 1e-8


def test_norm_gradient_by_differences_and_autograd():
    rng = np.random.default_rng(4)
    T, K, eps = 3, 32, 1e-3
    z, g, dy, res = rng.standard_normal((T, K)), rng.standard_normal(K), rng.standard_normal((T, K)), None
    dz, dg, _, _ = ref.norm_grad(dy, z, g, res, eps)
    f = lambda z_, g_: (ref.norm(z_, None, g_, eps)[1] * dy).sum()  # noqa: E731
    h = 1e-5
    for i in np.ndindex(z.shape):
        d = np.zeros_like(z)
        d[i] = h
        assert abs((f(z + d, g) - f(z - d, g)) / (2 * h) - dz[i]) < 1e-7
    for i in range(K):
        d = np.zeros_like(g)
        d[i] = h
        assert abs((f(z, g + d) - f(z, g - d)) / (2 * h) - dg[i]) < 1e-7
    tz, tg = (torch.tensor(a, requires_grad=True) for a in (z, g))
    y = tz / torch.sqrt((tz * tz).mean(1, keepdim=True) + eps) * tg
    (y * torch.tensor(dy)).sum().backward()
    assert np.allclose(tz.grad.numpy(), dz, rtol=1e-10) and np.allclose(tg.grad.numpy(), dg, rtol=1e-10)


# ------------------------------------------------------------ the host checks

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gg.library_path()):
        hb.build()
    return gg.load_library()


PRODUCT = dict(Aq=16, a_scale=32, Bq=48, b_scale=64, off=80, C=128, E=4, K=256, N=256, M_cap=29, bm=0)


@pytest.mark.parametrize("entry", ["gg_grouped_gemm_fp8_block", "gg_grouped_gemm_fp8_block_bf16out",
                                   "gg_grouped_gemm_fp8_block_swiglu"])
def test_product_host_checks(lib, entry):
    def st(**kw):
        return getattr(lib, entry)(*dict(PRODUCT, **kw).values(), None)
    for name in ("Aq", "a_scale", "Bq", "b_scale", "off", "C"):
        assert st(**{name: 0}) == INVALID and st(**{name: PRODUCT[name] + 2}) == MISALIGNED, name
        if name != "off":
            assert st(**{name: PRODUCT[name] + 8}) == MISALIGNED, name
    for kw in (dict(E=0), dict(K=0), dict(K=-16), dict(N=0), dict(M_cap=-1), dict(bm=8), dict(bm=512)):
        assert st(**kw) == INVALID, kw
    for kw in (dict(E=1025), dict(M_cap=2 ** 31 - 100), dict(K=2 ** 22 + 16), dict(N=2 ** 24 + 256)):
        assert st(**kw) == UNSUPPORTED, kw
    assert st(N=100) == st(K=264) == MISALIGNED
    assert st(M_cap=0) == st(M_cap=0, Aq=0, a_scale=0, C=0) == 0


def test_quantiser_host_checks(lib):
    q = lambda X=16, c=32, s=48, rows=3, K=64: lib.gg_fp8_quantize(X, c, s, rows, K, None)  # noqa: E731
    assert q(X=0) == q(c=0) == q(s=0) == q(rows=-1) == q(K=0) == INVALID
    assert q(X=24) == q(c=40) == q(s=52) == q(K=40) == MISALIGNED
    assert q(rows=2 ** 31) == q(K=2 ** 22 + 16) == q(rows=2 ** 31 - 1, K=2 ** 22) == UNSUPPORTED
    assert q(rows=0) == q(rows=0, X=0, c=0, s=0) == 0
    # 2^23 - 1 workgroups of 32 rows x 512 values pass, and meet the next check
    assert q(rows=32 * (2 ** 23 - 1), K=512, X=0) == INVALID
    assert q(rows=32 * (2 ** 23 - 1) + 1, K=512, X=0) == UNSUPPORTED

    def w(B=16, c=32, s=48, g=0, E=2, K=64, N=16):
        return lib.gg_fp8_quantize_weights(B, c, s, g, E, K, N, None)
    assert w(B=0) == w(c=0) == w(s=0) == w(E=0) == w(K=0) == w(N=-8) == INVALID
    assert w(B=24) == w(c=40) == w(s=52) == w(K=40) == w(N=12) == w(g=1, N=24) == w(g=1, K=12) == MISALIGNED
    assert w(E=1025) == w(K=2 ** 22 + 16) == w(N=2 ** 24 + 16) == UNSUPPORTED
    assert w(g=1, N=2 ** 22 + 16) == w(g=1, K=2 ** 24 + 16) == w(E=1024, K=2 ** 22, N=2 ** 20) == UNSUPPORTED


def test_row_host_checks(lib):
    names = dict(experts=16, wide=0, w=32, off=48, rows=64, pos=80, rw=96, ws=112, T=5, k=2, E=4)

    def sort(**kw):
        return lib.gg_expert_sort(*dict(names, **kw).values(), None)
    for n in ("experts", "w", "off", "rows", "pos", "rw"):
        assert sort(**{n: 0}) == INVALID, n
        assert sort(**{n: names[n] + 2}) == MISALIGNED, n
    assert sort(wide=1, experts=20) == MISALIGNED and sort(ws=120) == MISALIGNED
    assert sort(T=-1) == sort(k=0) == sort(E=0) == INVALID
    assert sort(T=20000, ws=0) == INVALID, "the split sort counts in its workspace"
    assert sort(E=1025) == sort(T=2 ** 31) == sort(T=2 ** 30, k=2) == UNSUPPORTED
    need = lib.gg_expert_sort_workspace
    assert need(0, 4) == need(8192, 1024) == need(2 ** 31, 4) == 0
    assert need(8193, 5) == 9 * 8 * 4 and need(10 ** 6, 1024) == 245 * 1024 * 4 and need(2 ** 31 - 1, 7) == 256 * 8 * 4

    good = dict(X=16, pos=32, out=48, s=64, os=80, sb=4, T=5, k=2, rb=64, slices=2, M=10)

    def spread(**kw):
        return lib.gg_expert_spread(*dict(good, **kw).values(), None)
    for n in ("X", "pos", "out", "s", "os"):
        assert spread(**{n: 0}) == INVALID and spread(**{n: good[n] + 2}) == MISALIGNED, n
    assert spread(sb=3) == spread(slices=-1) == spread(sb=0) == spread(slices=0) == INVALID
    assert spread(T=-1) == spread(k=0) == spread(M=-1) == spread(rb=0) == INVALID
    assert spread(rb=40) == MISALIGNED
    assert spread(T=2 ** 31) == spread(M=2 ** 31) == spread(T=2 ** 30, k=2) == spread(rb=2 ** 31 + 16) == UNSUPPORTED
    bare = dict(sb=0, slices=0, k=1)
    assert spread(T=2 ** 26, **bare) == UNSUPPORTED and spread(T=2 ** 26 - 4, X=0, **bare) == INVALID
    # a quarter of the tokens, and eight workgroups for each 256 of them
    assert spread(T=2 ** 26 - 4, k=1, X=0) == UNSUPPORTED and spread(T=2 ** 25, k=1, X=0) == INVALID
    assert spread(T=0, M=0) == spread(M=0) == spread(T=0, M=0, X=0, pos=0, out=0, s=0, os=0) == 0

    good_c = dict(Y=16, y32=0, pos=32, w=48, out=64, o32=0, T=5, k=2, N=64, M=10)

    def comb(**kw):
        return lib.gg_expert_combine(*dict(good_c, **kw).values(), None)
    for n in ("Y", "pos", "out"):
        assert comb(**{n: 0}) == INVALID and comb(**{n: good_c[n] + 2}) == MISALIGNED, n
    assert comb(w=50) == comb(N=60) == comb(Y=24) == MISALIGNED
    assert comb(N=0) == comb(k=0) == comb(T=-1) == comb(M=-1) == INVALID
    assert comb(N=2 ** 24 + 8) == comb(T=2 ** 30, k=2) == comb(T=2 ** 26, k=1, N=512) == UNSUPPORTED
    assert comb(T=0) == 0

    good_g = dict(dO=16, Y=32, f32=0, pos=48, w=64, dY=80, dw=96, T=5, k=2, N=64, M=10)

    def grad(**kw):
        return lib.gg_expert_combine_grad(*dict(good_g, **kw).values(), None)
    for n in ("dO", "Y", "pos", "w", "dY", "dw"):
        assert grad(**{n: 0}) == INVALID and grad(**{n: good_g[n] + 2}) == MISALIGNED, n
    assert grad(N=60) == MISALIGNED and grad(N=0) == grad(k=0) == grad(T=-1) == INVALID
    assert grad(N=2 ** 24 + 8) == grad(T=2 ** 30, k=2) == grad(T=2 ** 24, k=1) == UNSUPPORTED
    assert grad(T=0, M=0) == 0


def test_norm_host_checks(lib):
    good = dict(X=16, res=32, g=48, q=64, s=80, sum=96, norm=112, T=5, K=64, eps=1e-6)

    def norm(**kw):
        return lib.gg_rms_norm_fp8(*dict(good, **kw).values(), None)
    for n in ("X", "g", "q", "s"):
        assert norm(**{n: 0}) == INVALID
    for n in ("X", "res", "g", "q", "s", "sum", "norm"):
        assert norm(**{n: good[n] + 8}) == MISALIGNED
    assert norm(res=0) == INVALID, "a sum of nothing"
    assert norm(T=-1) == norm(K=0) == norm(eps=-1.0) == norm(eps=float("nan")) == INVALID
    assert norm(K=40) == MISALIGNED
    assert norm(K=16400) == norm(T=2 ** 31) == norm(T=2 ** 24 - 1) == UNSUPPORTED
    assert norm(T=2 ** 24 - 2, X=0) == INVALID
    assert norm(T=0) == norm(T=0, X=0, res=0, q=0, s=0, sum=0, norm=0) == 0
    good_g = dict(dy=16, z=32, g=48, res=64, dz=80, dg=96, ws=112, T=5, K=64, eps=1e-6)

    def grad(**kw):
        return lib.gg_rms_norm_grad(*dict(good_g, **kw).values(), None)
    for n in ("dy", "z", "g", "dz", "dg", "ws"):
        assert grad(**{n: 0}) == INVALID, n
    for n in good_g:
        if n not in ("T", "K", "eps"):
            assert grad(**{n: good_g[n] + 8}) == MISALIGNED, n
    assert grad(T=-1) == grad(K=0) == grad(eps=-1.0) == INVALID
    assert grad(K=40) == MISALIGNED and grad(K=16400) == grad(T=2 ** 31) == grad(T=2 ** 24 - 1) == UNSUPPORTED
    need = lib.gg_rms_norm_grad_workspace
    assert need(0, 64) == need(5, 16400) == 0 and need(3, 64) > 0 and need(10 ** 6, 64) % 16 == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: for hosts without a GPU")
def test_overlapping_arrays_are_refused(lib):
    # each output over the first and the last 16 bytes of every other array, all others
    # 2^40 apart; every call is refused (an accepted one would end in a missing device here)
    E, K, N, M, T, k = 4, 288, 144, 30, 10000, 2
    n = T * k
    calls = {
        "gg_fp8_quantize": ("X *q *s", dict(X=M * K * 2, q=M * K, s=3 * M * 4), lambda a: (*a, M, K)),
        "gg_fp8_quantize_weights": ("B *q *s", dict(B=E * K * N * 2, q=E * K * N, s=E * 6 * 4),
                                    lambda a: (*a, 0, E, K, N)),
        "gg_grouped_gemm_fp8_block": ("A As B Bs off *C", dict(A=M * K, As=3 * M * 4, B=E * K * N, Bs=E * 6 * 4,
                                                               off=20, C=M * N * 4), lambda a: (*a, E, K, N, M, 0)),
        "gg_grouped_gemm_fp8_block_bf16out": ("A As B Bs off *C", dict(A=M * K, As=3 * M * 4, B=E * K * N, Bs=E * 6 * 4,
                                                                       off=20, C=M * N * 2),
                                              lambda a: (*a, E, K, N, M, 0)),
        "gg_grouped_gemm_fp8_block_swiglu": ("A As B Bs off *C", dict(A=M * K, As=3 * M * 4, B=E * K * N, Bs=E * 6 * 4,
                                                                      off=20, C=M * N), lambda a: (*a, E, K, N, M, 0)),
        "gg_expert_sort": ("e w *off *rows *pos *rw *ws", dict(e=n * 4, w=n * 4, off=20, rows=n * 4, pos=n * 4, rw=n * 4,
                                                               ws=20 * 16), lambda a: (a[0], 0, *a[1:], T, k, E)),
        "gg_expert_spread": ("X pos *out s *os", dict(X=T * 64, pos=n * 4, out=M * 64, s=3 * T * 4, os=3 * M * 4),
                             lambda a: (*a, 4, T, k, 64, 3, M)),
        "gg_expert_combine": ("Y pos w *out", dict(Y=M * N * 2, pos=n * 4, w=n * 4, out=T * N * 4),
                              lambda a: (a[0], 0, a[1], a[2], a[3], 1, T, k, N, M)),
        "gg_expert_combine_grad": ("dO Y pos w *dY *dw", dict(dO=T * N * 2, Y=M * N * 2, pos=n * 4, w=n * 4,
                                                              dY=M * N * 2, dw=n * 4),
                                   lambda a: (a[0], a[1], 0, *a[2:], T, k, N, M)),
        "gg_rms_norm_fp8": ("X res g *q *s *sum *norm", dict(X=M * K * 2, res=M * K * 2, g=K * 2, q=M * K, s=3 * M * 4,
                                                             sum=M * K * 2, norm=M * K * 2),
                            lambda a: (*a, M, K, 1e-6)),
        "gg_rms_norm_grad": ("dy z g res *dz *dg *ws", dict(dy=M * K * 2, z=M * K * 2, g=K * 2, res=M * K * 2,
                                                            dz=M * K * 2, dg=K * 4, ws=M * K * 4),
                             lambda a: (*a, M, K, 1e-6)),
    }
    for entry, (names, size, args) in calls.items():
        names = names.split()
        outs = [x[1:] for x in names if x[0] == "*"]
        names = [x.lstrip("*") for x in names]
        home = {x: (i + 1) << 40 for i, x in enumerate(names)}
        call = lambda at: getattr(lib, entry)(*args([at[x] for x in names]), None)  # noqa: E731
        assert call(home) == NO_DEVICE, entry
        in_place = {("sum", "X"), ("sum", "res")} if entry == "gg_rms_norm_fp8" else set()
        for moved in outs:
            for onto in names:
                if moved == onto:
                    continue
                for at in (home[onto] + (16 if (moved, onto) in in_place else 0),
                           home[onto] + (size[onto] - 1) // 16 * 16, home[onto] - (size[moved] - 1) // 16 * 16):
                    assert call(dict(home, **{moved: at})) == INVALID, (entry, moved, onto, at - home[onto])
        for moved, onto in in_place:
            assert call(dict(home, **{moved: home[onto]})) == NO_DEVICE


# ------------------------------------------------------------------ the binding

def _dev(kind, *shape):
    dt = {"f8": torch.float8_e4m3fn, "l": torch.int64, "h": torch.float16}.get(kind)
    return _fake(kind, *shape) if dt is None else torch.empty(shape, dtype=dt, device="cuda")


@pytest.mark.parametrize("call", [
    lambda t: gg.fp8_quantize(t("f", 4, 32)),
    lambda t: gg.fp8_quantize(t("bf", 4, 32), out=t("bf", 4, 32)),
    lambda t: gg.fp8_quantize(t("bf", 4, 32), out_scale=t("f", 4, 1)),
    lambda t: gg.fp8_quantize_weights(t("bf", 4, 32)),
    lambda t: gg.grouped_gemm_fp8_block(t("bf", 4, 32), t("f", 1, 4), t("f8", 2, 8, 32), t("f", 2, 1, 1), t("i", 3)),
    lambda t: gg.grouped_gemm_fp8_block(t("f8", 4, 32), t("f", 4, 1), t("f8", 2, 8, 32), t("f", 2, 1, 1), t("i", 3)),
    lambda t: gg.grouped_gemm_fp8_block(t("f8", 4, 32), t("f", 1, 4), t("f8", 2, 8, 32), t("f", 2, 1, 2), t("i", 3)),
    lambda t: gg.grouped_gemm_fp8_block(t("f8", 4, 32), t("f", 1, 4), t("f8", 2, 8, 32), t("f", 2, 1, 1), t("i", 4)),
    lambda t: gg.grouped_gemm_fp8_block(t("f8", 4, 32), t("f", 1, 4), t("f8", 2, 8, 32), t("f", 2, 1, 1), t("i", 3),
                                        out_dtype=torch.float16),
    lambda t: gg.grouped_gemm_fp8_block_swiglu(t("f8", 4, 32), t("f", 1, 4), t("f8", 2, 8, 32), t("f", 2, 1, 1),
                                               t("i", 3), out=t("bf", 4, 8)),
    lambda t: gg.expert_sort(t("f", 4, 2), 3),
    lambda t: gg.expert_sort(t("i", 8), 3),
    lambda t: gg.expert_sort(t("i", 4, 2), 3, weights=t("bf", 4, 2)),
    lambda t: gg.expert_sort(t("i", 4, 2), 3, weights=t("f", 4, 3)),
    lambda t: gg.expert_sort(t("i", 4, 2), 3, out=(t("i", 4), t("i", 8))),
    lambda t: gg.expert_sort(t("i", 4, 2), 3, out=(t("i", 4), t("i", 7), t("i", 4, 2))),
    lambda t: gg.expert_spread(t("bf", 4, 32), t("l", 4, 2)),
    lambda t: gg.expert_spread(t("bf", 5, 32), t("i", 4, 2)),
    lambda t: gg.expert_spread(t("f8", 4, 32), t("i", 4, 2), scale=t("f", 1, 5)),
    lambda t: gg.expert_spread(t("f8", 4, 32), t("i", 4, 2), scale=t("u8", 1, 4)),
    lambda t: gg.expert_spread(t("f8", 4, 144), t("i", 4, 2), scale=t("f", 1, 4)),
    lambda t: gg.expert_spread(t("f8", 4, 128), t("i", 4, 2), scale=t("f", 2, 4)),
    lambda t: gg.expert_spread(t("bf", 4, 32), t("i", 4, 2), out=t("f", 8, 32)),
    lambda t: gg.expert_combine(t("h", 8, 32), t("i", 4, 2)),
    lambda t: gg.expert_combine(t("bf", 8, 32), t("i", 4, 2), weights=t("f", 8)),
    lambda t: gg.expert_combine(t("bf", 8, 32), t("i", 4, 2), out=t("bf", 5, 32)),
    lambda t: gg.expert_combine_grad(t("f", 4, 32), t("bf", 8, 32), t("i", 4, 2), t("f", 4, 2)),
    lambda t: gg.expert_combine_grad(t("bf", 4, 40), t("bf", 8, 32), t("i", 4, 2), t("f", 4, 2)),
    lambda t: gg.rms_norm_fp8(t("bf", 4, 32), t("f", 32)),
    lambda t: gg.rms_norm_fp8(t("bf", 4, 32), t("bf", 16)),
    lambda t: gg.rms_norm_fp8(t("bf", 4, 32), t("bf", 32), residual=t("bf", 3, 32)),
    lambda t: gg.rms_norm_fp8(t("bf", 4, 32), t("bf", 32), out_sum=t("bf", 4, 32)),
    lambda t: gg.rms_norm_grad(t("f", 4, 32), t("bf", 4, 32), t("bf", 32)),
    lambda t: gg.rms_norm_grad(t("bf", 4, 32), t("bf", 4, 32), t("bf", 32), d_residual=t("bf", 4, 16)),
])
def test_wrong_types_and_shapes_are_refused(lib, call):
    # shapes only: neither memory nor a GPU stands behind these tensors
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(), pytest.raises((TypeError, ValueError)):
        call(_dev)


def test_host_tensors_and_strides_are_refused(lib):
    bf = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        gg.fp8_quantize(bf)
    with pytest.raises(ValueError, match="device tensor"):
        gg.expert_sort(torch.zeros(4, 2, dtype=torch.int32), 3)
    with pytest.raises(ValueError, match="device tensor"):
        gg.rms_norm_fp8(bf, bf[0].clone())
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(), pytest.raises(ValueError, match="contiguous"):
        gg.fp8_quantize(_fake("bf", 32, 4).t())


@pytest.mark.parametrize("call", [
    lambda t: gg.fp8_quantize(t("bf", 1, BIG)),
    lambda t: gg.fp8_quantize_weights(t("bf", 1, 16, BIG)),
    lambda t: gg.fp8_quantize_weights(t("bf", BIG, 16, 16)),
    lambda t: gg.grouped_gemm_fp8_block(t("u8", BIG, 16), t("f", 1, BIG), t("u8", 2, 8, 16), t("f", 2, 1, 1), t("i", 3)),
    lambda t: gg.grouped_gemm_fp8_block_swiglu(t("u8", 4, 16), t("f", 1, 4), t("u8", 2, BIG, 16),
                                               t("f", 2, -(-BIG // 128), 1), t("i", 3)),
    lambda t: gg.expert_sort(t("i", BIG // 2, 2), 3),
    lambda t: gg.expert_sort(t("i", 4, 2), 2 ** 32 + 4),
    lambda t: gg.expert_sort(t("i", 4, 2), 2 ** 30),
    lambda t: gg.expert_spread(t("bf", BIG, 8), t("i", BIG, 1)),
    lambda t: gg.expert_spread(t("bf", 4, 8), t("i", 4, 1), M_cap=BIG),
    lambda t: gg.expert_combine(t("bf", BIG, 8), t("i", 4, 1)),
    lambda t: gg.expert_combine(t("bf", 4, BIG), t("i", 4, 1)),
    lambda t: gg.expert_combine_grad(t("bf", 4, BIG), t("bf", 4, BIG), t("i", 4, 1), t("f", 4, 1)),
    lambda t: gg.rms_norm_fp8(t("bf", 1, BIG), t("bf", BIG)),
    lambda t: gg.rms_norm_grad(t("bf", 1, BIG), t("bf", 1, BIG), t("bf", BIG)),
])
def test_sizes_beyond_int32_are_refused(lib, call):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(), pytest.raises(gg.GroupedGemmError, match="status 3"):
        call(_fake)


# -------------------------------------------------------------------- the build

@pytest.mark.skipif(not os.path.exists(hb.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", hb.LAYER_SOURCES, ids=os.path.basename)
def test_kernels_neither_spill_nor_use_scratch(source):
    cmd = [hb.HIPCC, *[f for f in hb.FLAGS if f != "-shared"], "--offload-device-only", "-c",
           "-Rpass-analysis=kernel-resource-usage", "-o", os.devnull, source]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels, cur = {}, None
    for line in r.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            cur = kernels.setdefault(m.group(1), {})
        m = re.search(r"remark:\s+([A-Za-z /\[\]]+?):\s+(\d+)", line)
        if m and cur is not None:
            cur[m.group(1).strip()] = int(m.group(2))
    assert kernels
    for name, u in kernels.items():
        assert u["VGPRs Spill"] == 0 and u["ScratchSize [bytes/lane]"] == 0, (name, u)
        assert u["Occupancy [waves/SIMD]"] >= 2, (name, u)


@pytest.mark.skipif(not os.path.exists(hb.HIPCC), reason="hipcc not available")
def test_product_loops_hold_what_they_need(tmp_path):
    # as for the other products of packed operands: scalars that do not fit are kept in
    # lanes of a vector register, but not in the loops over slices, and the compiler waits
    # there on no load into LDS, which the ring's own waits (inline asm) count
    out = str(tmp_path / "k.s")
    cmd = [hb.HIPCC, *[f for f in hb.FLAGS if f not in ("-shared", "-fPIC")], "--offload-device-only", "-S",
           "-o", out, hb.LAYER_SOURCES[-1]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    loops = [b for k in re.findall(r"\n(_ZN2gg\w*product_kernel\w*):", text)
             for b in _inner_loops(text[text.index("\n%s:" % k):text.index(".Lfunc_end", text.index("\n%s:" % k))])]
    products = [b for b in loops if any("v_mfma" in ln for ln in b)]
    assert products
    for body in products:
        assert not any("v_readlane" in ln or "v_writelane" in ln or "scratch_" in ln for ln in body)
        for before, ln in zip(body, body[1:]):
            assert "vmcnt" not in ln or "#ASMSTART" in before, ln
    # a 256-row tile's second barrier frees the weights: all 2 x 4 column fragments are read by then
    tallest = [b for b in products if sum("s_barrier" in ln for ln in b) == 2]
    assert len(tallest) == 3
    for body in tallest:
        first, second = (i for i, ln in enumerate(body) if "s_barrier" in ln)
        reads = [i for i, ln in enumerate(body) if "ds_read_b128" in ln]
        assert len(reads) == 24 and sum(first < i < second for i in reads) >= 8
