"""The gradients and the 4-bit operators without a GPU: their references, the
host checks of the C entry points, the binding's refusals and the build.

No call below reaches the HIP runtime: each is rejected by the host checks, or
has nothing to do.
"""

import os
import re
import subprocess

import numpy as np
import pytest
import torch

import moe_ragged_grouped_amd as gg
import moe_ragged_grouped_amd.build as hb
import oracle
import oracle.operators as ref
import workloads as wl
from tests import operators as ops

INVALID, MISALIGNED, UNSUPPORTED, NO_DEVICE = 1, 2, 3, 4


# ---------------------------------------------------------------- references

def _layer(rng, sizes, K, N):
    off = ops.offsets_of(sizes)
    M = int(off[-1])
    return off, ops.bits(rng, M, K), ops.bits(rng, len(sizes), K, N), ops.bits(rng, M, N)


def test_gradient_references_against_autograd():
    rng = np.random.default_rng(0)
    off, A, B, dC = _layer(rng, [3, 0, 5], 16, 24)
    a = torch.from_numpy(oracle._bf16_to_f64(A)).requires_grad_()
    b = torch.from_numpy(oracle._bf16_to_f64(B)).requires_grad_()
    c = torch.cat([a[off[e]:off[e + 1]] @ b[e] for e in range(3)])
    c.backward(torch.from_numpy(oracle._bf16_to_f64(dC)))
    np.testing.assert_allclose(ref.dgrad(dC, B, off)[0], a.grad.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(ref.wgrad(A, dC, off)[0], b.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert (ref.wgrad(A, dC, off)[0][1] == 0).all()


def test_swiglu_reference_against_autograd():
    rng = np.random.default_rng(1)
    C = rng.standard_normal((7, 24)) * 3
    dH = rng.standard_normal((7, 12))
    c = torch.from_numpy(C).requires_grad_()
    h = torch.nn.functional.silu(c[:, 0::2]) * c[:, 1::2]
    h.backward(torch.from_numpy(dH))
    d, H = ref.swiglu_grad(dH, C)
    np.testing.assert_allclose(d, c.grad.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(H, h.detach().numpy(), rtol=1e-12)


def test_swiglu_error_bound_covers_a_float32_evaluation():
    rng = np.random.default_rng(2)
    C = (rng.standard_normal((400, 64)) * 20).astype(np.float32)
    dH = rng.standard_normal((400, 32)).astype(np.float32)
    f = np.float32
    g, u = C[:, 0::2], C[:, 1::2]
    with np.errstate(over="ignore"):
        s = f(1) / (f(1) + np.exp2(-g * f(1.4426950408889634)))
    got = np.stack([dH * u * (s * (f(1) + g * (f(1) - s))), dH * (g * s)], axis=-1).reshape(C.shape)
    want, H = ref.swiglu_grad(dH.astype(np.float64), C.astype(np.float64))
    err, err_h = ref.swiglu_grad_error(dH.astype(np.float64), 0.0, C.astype(np.float64))
    assert (np.abs(got - want) <= err).all()
    assert (np.abs(g * s * u - H) <= err_h).all()


def test_mx4_reference_by_hand():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :6] = [4.0, 2.5, -0.75, 7.0, 0.25, -0.0]  # scale 1
    x[0, 32:35] = [0.75, 0.09375, 0.046875]        # maximum in [1/2, 1): scale 1/8
    q, s = ref.mx4_encode(wl.f32_to_bf16_bits(x))
    assert q.shape == (1, 32) and s.shape == (1, 1, 8)
    assert s[0, 0].tolist() == [127, 124, 0, 0, 0, 0, 0, 0]
    assert q[0, :3].tolist() == [6 | 4 << 4, 10 | 7 << 4, 0 | 8 << 4]
    assert q[0, 16:18].tolist() == [7 | 2 << 4, 1]  # 6, .75 -> 1 (tie to even), .375 -> .5
    v = ref.mx4_values(q, s)
    assert v[0, :6].tolist() == [4, 2, -1, 6, 0, 0] and v[0, 32:35].tolist() == [0.75, 0.125, 0.0625]


def test_mx4_reference_is_the_nearest_value():
    rng = np.random.default_rng(3)
    x = ops.bits(rng, 40, 96)
    q, s = ref.mx4_encode(x)
    v, t = oracle._bf16_to_f64(x).reshape(40, 3, 32), ref.mx4_values(q, s).reshape(40, 3, 32)
    scale = np.ldexp(1.0, s[0, :, :3].astype(int) - 127)[..., None]
    top = np.abs(v).max(-1, keepdims=True)
    assert ((4 * scale <= top) & (top < 8 * scale)).all()
    grid = np.concatenate([ref.E2M1, -ref.E2M1]) * scale[..., None]
    nearest = np.abs(v[..., None] - grid).min(-1)
    assert (np.abs(v - t) == nearest).all()


# ------------------------------------------------------------- host checks

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gg.library_path()):
        hb.build()
    return gg.load_library()


ROW = dict(E=4, K=256, N=256, M_cap=29)
ENTRIES = {
    "gg_grouped_gemm_bf16_dgrad": dict(dC=16, B=32, off=64, dA=128, **ROW, bm=0),
    "gg_grouped_gemm_bf16_dgrad_bf16out": dict(dC=16, B=32, off=64, dA=128, **ROW, bm=0),
    "gg_grouped_gemm_bf16_dgrad_swiglu": dict(dC=16, B=32, off=64, C=80, dA=128, H=144, **ROW, bm=0),
    "gg_grouped_gemm_bf16_wgrad": dict(A=16, dC=32, off=64, dB=128, acc=0, **ROW),
    "gg_grouped_gemm_bf16_wgrad_bf16out": dict(A=16, dC=32, off=64, dB=128, **ROW),
    "gg_grouped_gemm_mx4": dict(Aq=16, a_scale=32, Bq=48, b_scale=64, off=80, C=128, **ROW, bm=0),
    "gg_grouped_gemm_mx4_bf16out": dict(Aq=16, a_scale=32, Bq=48, b_scale=64, off=80, C=128, **ROW, bm=0),
    "gg_grouped_gemm_mx4_swiglu": dict(Aq=16, a_scale=32, Bq=48, b_scale=64, off=80, C=128, **ROW, bm=0),
}


def _status(lib, entry, **kw):
    # fake, aligned addresses: every call is rejected on the host
    args = dict(ENTRIES[entry])
    args.update(kw)
    return getattr(lib, entry)(*args.values(), None)


@pytest.mark.parametrize("entry", ENTRIES)
def test_host_checks(lib, entry):
    good = ENTRIES[entry]
    for name in good:
        if name in ("E", "K", "N", "M_cap", "bm", "acc", "H"):
            continue
        assert _status(lib, entry, **{name: 0}) == INVALID, name
        assert _status(lib, entry, **{name: good[name] + 2}) == MISALIGNED, name
        if name != "off":
            assert _status(lib, entry, **{name: good[name] + 8}) == MISALIGNED, name
    for kw in (dict(E=0), dict(E=-1), dict(K=0), dict(K=-8), dict(N=0), dict(M_cap=-1)):
        assert _status(lib, entry, **kw) == INVALID, kw
    for kw in (dict(E=1025), dict(M_cap=2 ** 31 - 100), dict(K=2 ** 24 + 256), dict(N=2 ** 24 + 256)):
        assert _status(lib, entry, **kw) == UNSUPPORTED, kw
    assert _status(lib, entry, N=100) == MISALIGNED
    assert _status(lib, entry, K=100) == MISALIGNED
    if "mx4" in entry:
        assert _status(lib, entry, K=264) == MISALIGNED
        assert _status(lib, entry, K=2 ** 22 + 32) == UNSUPPORTED
    if "H" in good:
        assert _status(lib, entry, H=136) == MISALIGNED
    if "dgrad" in entry:
        assert _status(lib, entry, N=2 ** 21 + 8) == UNSUPPORTED
    if "wgrad" in entry:
        assert _status(lib, entry, K=2 ** 22 + 8) == UNSUPPORTED
        assert _status(lib, entry, N=2 ** 22 + 8) == UNSUPPORTED
        assert _status(lib, entry, E=1024, K=2 ** 22, N=2 ** 22) == UNSUPPORTED  # tiles beyond the grid
    else:
        for bm in (8, 48, 512, -16):
            assert _status(lib, entry, bm=bm) == INVALID
        rows = {n: 0 for n in ("dC", "dA", "C", "H", "Aq", "a_scale") if n in good}
        assert _status(lib, entry, M_cap=0) == 0
        assert _status(lib, entry, M_cap=0, **rows) == 0, "arrays of no rows may be null"


@pytest.mark.parametrize("entry", [e for e in ENTRIES if "wgrad" not in e])
def test_the_forward_products_tile_bound_holds(lib, entry):
    # (M_cap / 16 + E) * ceil(columns / 256) up to 2^28 passes (and meets the check of the
    # other size, which comes after it), one more 256 columns does not
    cols, other = ("K", "N") if "dgrad" in entry else ("N", "K")
    size = dict(E=4, M_cap=2 ** 28)
    # the forward product draws the same line
    fwd = lambda n: lib.gg_grouped_gemm_bf16(0, 32, 64, 128, 4, 256, n, 2 ** 28, 0, None)  # noqa: E731
    assert fwd(15 * 256) == INVALID and fwd(15 * 256 + 8) == UNSUPPORTED
    assert _status(lib, entry, **size, **{cols: 15 * 256, other: 100}) == MISALIGNED
    assert _status(lib, entry, **size, **{cols: 15 * 256 + 8, other: 100}) == UNSUPPORTED


def test_mx4_row_host_checks(lib):
    q = lambda X=16, c=32, s=48, rows=3, K=64: lib.gg_mx4_quantize(X, c, s, rows, K, None)  # noqa: E731
    assert q(X=0) == q(c=0) == q(s=0) == q(rows=-1) == q(K=0) == INVALID
    assert q(X=24) == q(c=40) == q(s=52) == q(K=40) == MISALIGNED
    assert q(rows=2 ** 31) == q(K=2 ** 22 + 32) == q(rows=2 ** 31 - 1, K=2 ** 22) == UNSUPPORTED
    assert q(rows=0) == q(rows=0, X=0, c=0, s=0) == 0
    w = lambda B=16, c=32, s=48, E=2, K=64, N=8: lib.gg_mx4_quantize_weights(B, c, s, E, K, N, None)  # noqa: E731
    assert w(B=0) == w(c=0) == w(s=0) == w(E=0) == w(K=0) == w(N=-8) == INVALID
    assert w(B=24) == w(c=40) == w(s=52) == w(K=40) == w(N=12) == MISALIGNED
    assert w(E=1025) == w(K=2 ** 22 + 32) == w(N=2 ** 24 + 8) == w(E=1024, K=2 ** 22, N=2 ** 24) == UNSUPPORTED
    d = lambda c=16, s=32, Y=48, b=2, rows=3, K=64: lib.gg_mx4_dequantize(c, s, Y, b, rows, K, None)  # noqa: E731
    assert d(c=0) == d(s=0) == d(Y=0) == d(b=-1) == d(rows=-1) == d(K=0) == INVALID
    assert d(c=24) == d(s=40) == d(Y=56) == d(K=40) == MISALIGNED
    assert d(b=65536) == d(rows=2 ** 31) == UNSUPPORTED
    assert d(b=0) == d(rows=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: for hosts without a GPU")
def test_overlapping_arrays_are_refused(lib):
    # each output over the first and the last 16 bytes of every other array, all others
    # 2^40 apart; every call is refused (an accepted one would end in a missing device here)
    E, K, N, M = 4, 288, 136, 30
    rows = 16 * 2
    D = {"dC": M * N * 2, "B": E * K * N * 2, "off": rows, "A": M * K * 2, "C": M * K * 4, "H": M * K * 2,
         "Aq": M * K // 2, "a_scale": 2 * M * 8, "Bq": E * N * K // 2, "b_scale": E * 2 * N * 8}
    calls = {
        "gg_grouped_gemm_bf16_dgrad": ("dC B off *", M * K * 4, (E, K, N, M, 0)),
        "gg_grouped_gemm_bf16_dgrad_bf16out": ("dC B off *", M * K * 2, (E, K, N, M, 0)),
        "gg_grouped_gemm_bf16_dgrad_swiglu": ("dC B off C * H", M * K * 4, (E, K, N, M, 0)),
        "gg_grouped_gemm_bf16_wgrad": ("A dC off *", E * K * N * 4, (0, E, K, N, M)),
        "gg_grouped_gemm_bf16_wgrad_bf16out": ("A dC off *", E * K * N * 2, (E, K, N, M)),
        "gg_grouped_gemm_mx4": ("Aq a_scale Bq b_scale off *", M * N * 4, (E, K, N, M, 0)),
        "gg_grouped_gemm_mx4_bf16out": ("Aq a_scale Bq b_scale off *", M * N * 2, (E, K, N, M, 0)),
        "gg_grouped_gemm_mx4_swiglu": ("Aq a_scale Bq b_scale off *", M * N, (E, K, N, M, 0)),
        "gg_mx4_quantize": ("A * a_scale", M * K // 2, (M, K)),
        "gg_mx4_quantize_weights": ("B * b_scale", E * N * K // 2, (E, K, N)),
        "gg_mx4_dequantize": ("Bq b_scale *", E * N * K * 2, (E, N, K)),
    }
    for entry, (names, out_bytes, sizes) in calls.items():
        names = names.split()
        size = dict(D, **{"*": out_bytes})
        home = {n: (i + 1) << 40 for i, n in enumerate(names)}
        args = [home[n] for n in names]
        assert getattr(lib, entry)(*args, *sizes, None) == NO_DEVICE, entry
        if "C" in names:  # in place
            args[names.index("*")] = home["C"]
            assert getattr(lib, entry)(*args, *sizes, None) == NO_DEVICE, entry
        pairs = [("*", n) for n in names if n != "*"]
        pairs += [("H", n) for n in names if n != "H"] if "H" in names else []
        pairs += [(n, "*") for n in names if n.endswith("scale") and "quantize" in entry]
        for moved, onto in pairs:
            for at in (home[onto] + (16 if (moved, onto) == ("*", "C") else 0),
                       home[onto] + (size[onto] - 1) // 16 * 16, home[onto] - (size[moved] - 1) // 16 * 16):
                args = [at if n == moved else home[n] for n in names]
                assert getattr(lib, entry)(*args, *sizes, None) == INVALID, (entry, moved, onto, at - home[onto])


def test_launches_of_2_to_the_32_threads_are_refused(lib):
    # 2^24 tiles of 128 x 256 (256 threads each); 2^24 pieces of 8192 values; 2^23 of 256 x 256
    for entry in ("gg_grouped_gemm_bf16_wgrad", "gg_grouped_gemm_bf16_wgrad_bf16out"):
        assert _status(lib, entry, E=1024, K=8, N=2 ** 22) == UNSUPPORTED
    assert lib.gg_mx4_quantize(16, 32, 48, 2 ** 15, 2 ** 22, None) == UNSUPPORTED
    assert lib.gg_mx4_dequantize(16, 32, 48, 1, 2 ** 15, 2 ** 22, None) == UNSUPPORTED
    assert lib.gg_mx4_quantize_weights(16, 32, 48, 512, 2 ** 22, 8, None) == UNSUPPORTED


def test_documented_ends_of_the_launch_limits(lib):
    # the last size that passes meets the check behind the limit (null or overlapping arrays)
    q = lambda rows, K: lib.gg_mx4_quantize(0, 32, 48, rows, K, None)  # noqa: E731
    d = lambda rows, K: lib.gg_mx4_dequantize(0, 32, 48, 1, rows, K, None)  # noqa: E731
    for f in (q, d):
        assert f(2 ** 31 - 128, 64) == INVALID and f(2 ** 31 - 127, 64) == UNSUPPORTED
        assert f(2 ** 24 - 1, 8192) == INVALID and f(2 ** 24, 8192) == UNSUPPORTED
    w = lambda E, K, N: lib.gg_mx4_quantize_weights(16, 32, 48, E, K, N, None)  # noqa: E731
    assert w(1023, 2 ** 21, 256) == INVALID and w(1024, 2 ** 21, 256) == UNSUPPORTED
    for entry in ("gg_grouped_gemm_bf16_wgrad", "gg_grouped_gemm_bf16_wgrad_bf16out"):
        g = lambda E, K, N: _status(lib, entry, E=E, K=K, N=N, dB=32)  # noqa: E731
        # 1 x 16383 tiles go out as 16384: 1023 experts pass, 1024 do not
        assert g(1023, 128, 16383 * 256) == INVALID and g(1024, 128, 16383 * 256) == UNSUPPORTED
        assert g(1024, 128, 16376 * 256) == INVALID


# ------------------------------------------------------------ the binding

def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


OFF = torch.zeros(3, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: gg.grouped_gemm_dgrad(torch.zeros(4, 8), _bf(2, 16, 8), OFF),
    lambda: gg.grouped_gemm_dgrad(_bf(4, 8), _bf(2, 16, 8), OFF.long()),
    lambda: gg.grouped_gemm_dgrad_swiglu(_bf(4, 8), _bf(2, 16, 8), OFF, torch.zeros(4, 32)),
    lambda: gg.grouped_gemm_wgrad(_bf(4, 8), torch.zeros(4, 8), OFF),
    lambda: gg.mx4_quantize(torch.zeros(4, 32)),
    lambda: gg.mx4_quantize_weights(torch.zeros(1, 32, 8)),
    lambda: gg.mx4_dequantize(torch.zeros(4, 16), _u8(1, 4, 8)),
    lambda: gg.grouped_gemm_mx4(_u8(4, 16), _u8(1, 4, 8), _u8(2, 8, 16), _u8(2, 1, 8, 8).float(), OFF),
])
def test_wrong_types_are_refused(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("call", [
    lambda: gg.grouped_gemm_dgrad(_bf(4, 8), _bf(2, 16, 8), OFF),
    lambda: gg.grouped_gemm_dgrad(_bf(4), _bf(2, 16, 8), OFF),
    lambda: gg.grouped_gemm_wgrad(_bf(4, 8), _bf(4, 8), OFF),
    lambda: gg.mx4_quantize(_bf(4, 32)),
    lambda: gg.mx4_dequantize(_u8(16), _u8(1, 8)),
    lambda: gg.grouped_gemm_mx4_swiglu(_u8(4, 16), _u8(1, 4, 8), _u8(2, 8, 16), _u8(2, 1, 8, 8), OFF),
])
def test_host_tensors_and_wrong_ranks_are_refused(call):
    with pytest.raises(ValueError):
        call()


BIG = 2 ** 32 + 32  # what is left of it in 32 bits is a size like any other


def _fake(kind, *shape):
    dt = {"bf": torch.bfloat16, "u8": torch.uint8, "i": torch.int32, "f": torch.float32}[kind]
    return torch.empty(shape, dtype=dt, device="cuda")


@pytest.mark.parametrize("call", [
    lambda t: gg.grouped_gemm_dgrad(t("bf", BIG, 8), t("bf", 2, 8, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_dgrad(t("bf", 4, BIG), t("bf", 2, 8, BIG), t("i", 3)),
    lambda t: gg.grouped_gemm_dgrad(t("bf", 4, 8), t("bf", 2, BIG, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_dgrad(t("bf", 4, 8), t("bf", 2, 8, 8), t("i", 3), bm=2 ** 32 + 16),
    lambda t: gg.grouped_gemm_dgrad(t("bf", 4, 8), t("bf", 2, 8, 8), t("i", 3), bm=16 - 2 ** 32),
    lambda t: gg.grouped_gemm_dgrad_swiglu(t("bf", BIG, 8), t("bf", 2, 8, 8), t("i", 3), t("bf", BIG, 16)),
    lambda t: gg.grouped_gemm_wgrad(t("bf", BIG, 8), t("bf", BIG, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_wgrad(t("bf", 4, BIG), t("bf", 4, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_wgrad(t("bf", 4, 8), t("bf", 4, 8), t("i", BIG + 1)),
    lambda t: gg.mx4_quantize(t("bf", 1, BIG)),
    lambda t: gg.mx4_quantize_weights(t("bf", 1, 32, BIG)),
    lambda t: gg.mx4_quantize_weights(t("bf", BIG, 32, 8)),
    lambda t: gg.mx4_dequantize(t("u8", 1, BIG // 2), t("u8", BIG // 256 + 1, 1, 8)),
    lambda t: gg.grouped_gemm_mx4(t("u8", BIG, 16), t("u8", 1, BIG, 8), t("u8", 2, 8, 16), t("u8", 2, 1, 8, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_mx4_swiglu(t("u8", 4, 16), t("u8", 1, 4, 8), t("u8", 2, BIG, 16), t("u8", 2, 1, BIG, 8),
                                         t("i", 3)),
    lambda t: gg.grouped_gemm(t("bf", BIG, 8), t("bf", 2, 8, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_swiglu(t("bf", 4, 8), t("bf", 2, 8, BIG), t("i", 3)),
    lambda t: gg.grouped_gemm_gather(t("bf", BIG, 8), t("i", 4), t("bf", 2, 8, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_gather_combine(t("bf", 4, 8), t("i", 4), t("bf", 2, 8, 8), t("i", 3), t("i", 4), t("f", 4),
                                             n_dst=BIG),
    lambda t: gg.grouped_gemm_gather_combine(t("bf", 4, 8), t("i", 4), t("bf", 2, 8, 8), t("i", 3), t("i", 4), t("f", 4),
                                             out=t("f", BIG, 8)),
    lambda t: gg.grouped_gemm_fp8w(t("bf", 4, BIG), t("u8", 2, BIG, 8), t("f", 2, 8), t("i", 3)),
    lambda t: gg.grouped_gemm_fp8(t("u8", BIG, 16), t("f", BIG), t("u8", 2, 16, 16), t("f", 2, 16), t("i", 3)),
    lambda t: gg.grouped_gemm_fp8_swiglu(t("u8", 4, 16), t("f", 4), t("u8", 2, 16, BIG), t("f", 2, BIG), t("i", 3)),
    lambda t: gg.tile_schedule(t("i", 3), 8, BIG),
])
def test_sizes_beyond_int32_are_refused(lib, call):
    # shapes only: neither memory nor a GPU stands behind these tensors
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(), pytest.raises(gg.GroupedGemmError, match="status 3"):
        call(_fake)


# --------------------------------------------------------------- the build

@pytest.mark.skipif(not os.path.exists(hb.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", hb.OPERATOR_SOURCES, ids=os.path.basename)
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


def _inner_loops(asm):
    """The bodies of the innermost loops of one kernel's assembly."""
    lines = asm.split("\n")
    label = {m.group(1): i for i, ln in enumerate(lines) if (m := re.match(r"(\.LBB\d+_\d+):", ln))}
    loops = set()
    for i, ln in enumerate(lines):
        m = re.search(r"s_c?branch\w*\s+(\.LBB\d+_\d+)", ln)
        if m and label.get(m.group(1), i) < i:
            loops.add((label[m.group(1)], i))
    return [lines[a:b + 1] for a, b in loops
            if not any(c >= a and d <= b and (c, d) != (a, b) for c, d in loops)]


@pytest.mark.skipif(not os.path.exists(hb.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", hb.OPERATOR_SOURCES, ids=os.path.basename)
def test_product_loops_hold_what_they_need(source, tmp_path):
    # Scalars that do not fit are kept in lanes of a vector register: fine per
    # tile, but not in the loops over slices. Nor may the compiler wait there on
    # the loads into LDS, which the ring's own waits (inline asm) count.
    out = str(tmp_path / "k.s")
    cmd = [hb.HIPCC, *[f for f in hb.FLAGS if f not in ("-shared", "-fPIC")], "--offload-device-only", "-S",
           "-o", out, source]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    loops = [b for k in re.findall(r"\n(_ZN2gg\w*kernel\w*):", text)
             for b in _inner_loops(text[text.index("\n%s:" % k):text.index(".Lfunc_end", text.index("\n%s:" % k))])]
    products = [b for b in loops if any("v_mfma" in ln for ln in b)]
    assert products
    for body in products:
        assert not any("v_readlane" in ln or "v_writelane" in ln or "scratch_" in ln for ln in body)
        for before, ln in zip(body, body[1:]):
            assert "vmcnt" not in ln or "#ASMSTART" in before, ln
    # A 256-row tile's step has a second barrier, after which the weights and
    # scales it multiplies are overwritten: every wave has read its own by then
    # (2 x 4 column fragments; 8 + 4 scale reads) with 7 of its 16 row fragments.
    tallest = [b for b in products if sum("s_barrier" in ln for ln in b) == 2]
    assert len(tallest) == (0 if "wgrad" in source else 3)
    for body in tallest:
        first, second = (i for i, ln in enumerate(body) if "s_barrier" in ln)
        reads = [i for i, ln in enumerate(body) if "ds_read_b128" in ln]
        assert len(reads) == 24 and sum(first < i < second for i in reads) == 8 + 7
        scales = [i for i, ln in enumerate(body) if "ds_read_u16" in ln]
        assert len(scales) == (12 if "mx4" in source else 0) and all(first < i < second for i in scales)
