"""Rows to their experts and back on the GPU against binary64 (needs an MI355X)."""

import numpy as np
import pytest

import oracle
import oracle.layer as ref
from tests import operators as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _choices(rng, T, k, E, outside=0.0):
    """Choices of a router, skewed; some outside [0, E)."""
    p = (rng.permutation(E) + 1.0) ** -1.2
    e = rng.choice(E, size=(T, k), p=p / p.sum())
    far = rng.random((T, k)) < outside
    return np.where(far, rng.choice([-1, -7, E, E + 3, 2 ** 31 - 1, -2 ** 31], size=(T, k)), e).astype(np.int32)


def _fast_sort(e, E, w):
    """oracle.layer.sort for many choices (test_fast_sort_is_the_reference)."""
    flat = e.ravel()
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    off = np.searchsorted(key[order], np.arange(E + 1)).astype(np.int32)
    n = off[-1]
    rows, pos, rw = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32), np.zeros(flat.size, np.float32)
    rows[:n], rw[:n], pos[order[:n]] = order[:n] // e.shape[1], w.ravel()[order[:n]], np.arange(n)
    return off, rows, pos.reshape(e.shape), rw


def test_fast_sort_is_the_reference():
    rng = np.random.default_rng(0)
    e, w = _choices(rng, 300, 3, 11, 0.2), rng.random((300, 3)).astype(np.float32)
    for a, b in zip(_fast_sort(e, 11, w), ref.sort(e, 11, w)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,k,E", [
    (0, 2, 4), (1, 1, 1), (1, 8, 8), (7, 3, 5), (64, 8, 32), (129, 2, 1024), (1000, 8, 64), (1024, 8, 1023),
    (1025, 8, 64), (8193, 1, 3), (2048, 8, 64), (5000, 7, 1000), (16384, 8, 256), (40000, 8, 1), (262145, 1, 6)])
def test_sort(gg, T, k, E, wide):
    rng = np.random.default_rng(T + k + E)
    e, w = _choices(rng, T, k, E, 0.3 if E % 2 else 0.0), rng.random((T, k)).astype(np.float32)
    want = _fast_sort(e, E, w)
    d = ops.to_dev(e.astype(np.int64) if wide else e)
    got = gg.expert_sort(d, E, weights=ops.to_dev(w))
    for a, b in zip(got, want):
        assert np.array_equal(ops.host(a), b)
    for a, b in zip(gg.expert_sort(d, E), want):
        assert np.array_equal(ops.host(a), b)


def test_sort_far_numbers(gg):
    # an int64 choice whose low half is a valid expert is none
    e = torch.tensor([[2 ** 32 + 1, 1], [-2 ** 32, 0]], device=DEV)
    off, rows, pos = gg.expert_sort(e, 2)
    assert off.tolist() == [0, 1, 2] and rows.tolist() == [1, 0, -1, -1] and pos.tolist() == [[-1, 1], [-1, 0]]


@pytest.mark.parametrize("T", [3, 700, 3000, 100000])
def test_sort_all_or_none_here(gg, T):
    for e, n in ((5, T * 4), (-1, 0), (9, 0)):
        x = torch.full((T, 4), e, dtype=torch.int32, device=DEV)
        off, rows, pos, rw = gg.expert_sort(x, 9, weights=torch.ones(T, 4, device=DEV))
        assert off.tolist() == [0] * 6 + [n] * 4
        at = torch.arange(T * 4, dtype=torch.int32, device=DEV)
        assert torch.equal(rows, at // 4 if n else torch.full_like(at, -1))
        assert torch.equal(pos.flatten(), at if n else torch.full_like(at, -1))
        assert (rw == (1 if n else 0)).all()


def test_sort_feeds_the_gathered_products(gg):
    # offsets, rows and row_weights are what the gathered product with combine takes
    rng = np.random.default_rng(3)
    T, k, E, K, N = 50, 3, 6, 64, 72
    e, w = _choices(rng, T, k, E, 0.2), rng.random((T, k)).astype(np.float32)
    X, B = ops.int_bits(rng, T, K), ops.int_bits(rng, E, K, N)
    off, rows, pos, rw = gg.expert_sort(ops.to_dev(e), E, weights=ops.to_dev(w))
    Y = gg.grouped_gemm_gather_combine(ops.to_dev(X), rows, ops.to_dev(B), off, rows, rw)
    C = gg.grouped_gemm_gather(ops.to_dev(X), rows, ops.to_dev(B), off)
    mine = gg.expert_combine(C, pos, ops.to_dev(w))
    want, S = np.zeros((T, N)), np.zeros((T, N))
    x, b = oracle._bf16_to_f64(X), oracle._bf16_to_f64(B)
    for t in range(T):
        for j in range(k):
            if 0 <= e[t, j] < E:
                want[t] += w[t, j] * (x[t] @ b[e[t, j]])
                S[t] += np.abs(w[t, j] * (x[t] @ b[e[t, j]]))
    ops.check_f32(ops.host(Y), want, ops.sum_bound(k, S), "gather_combine")
    ops.check_f32(ops.host(mine), want, ops.sum_bound(k, S), "combine")
    rows_of = gg.expert_spread(ops.to_dev(X), pos)
    assert torch.equal(gg.grouped_gemm(rows_of, ops.to_dev(B), off)[:int(off[-1])], C[:int(off[-1])])


def _pos(rng, T, k, M, holes=0.2):
    """Places of T * k choices among M rows, each row at most once."""
    at = np.full(T * k, -1, np.int32)
    n = min(M, int(T * k * (1 - holes)))
    at[rng.choice(T * k, n, replace=False)] = rng.choice(M, n, replace=False)
    return at.reshape(T, k)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8", "u8"])
@pytest.mark.parametrize("T,k,M,K", [(1, 1, 1, 16), (5, 2, 10, 144), (3, 8, 24, 2064), (64, 8, 512, 6144),
                                     (130, 3, 200, 528), (7, 40, 280, 16)])
def test_spread(gg, T, k, M, K, kind):
    rng = np.random.default_rng(T + K)
    pos = _pos(rng, T, k, M)
    pos.ravel()[: min(3, T * k - 1)] = [-5, M, 2 ** 31 - 1][: min(3, T * k - 1)]
    x = rng.integers(0, 256, (T, K * {"bf16": 2, "fp32": 4}.get(kind, 1)), dtype=np.uint8)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": F8, "u8": torch.uint8}[kind]
    out = torch.full((M, x.shape[1]), 7, dtype=torch.uint8, device=DEV)
    X = ops.to_dev(x).view(dt)
    want = ref.spread(x, pos, np.full((M, x.shape[1]), 7, np.uint8))
    got = gg.expert_spread(X, ops.to_dev(pos), out=out.view(dt))
    assert got.dtype == dt and np.array_equal(got.view(torch.uint8).cpu().numpy(), want)
    if kind == "fp8":
        s = rng.random((-(-K // 128), T)).astype(np.float32)
        out_s = torch.full((s.shape[0], M), 7.0, device=DEV)
        q, got_s = gg.expert_spread(X, ops.to_dev(pos), scale=ops.to_dev(s), out=out.view(dt), out_scale=out_s)
        assert np.array_equal(ops.host(got_s), ref.spread(s.T, pos, np.full((M, s.shape[0]), 7, np.float32)).T)
    if kind == "u8":
        s = rng.integers(0, 256, (-(-2 * K // 256), T, 8), dtype=np.uint8)
        out_s = torch.full((s.shape[0], M, 8), 7, dtype=torch.uint8, device=DEV)
        gg.expert_spread(X, ops.to_dev(pos), scale=ops.to_dev(s), out=out, out_scale=out_s)
        flat = ref.spread(np.swapaxes(s, 0, 1), pos, np.full((M, s.shape[0], 8), 7, np.uint8))
        assert np.array_equal(ops.host(out_s), np.swapaxes(flat, 0, 1))


def test_spread_scales_of_many_slices(gg):
    rng = np.random.default_rng(5)
    T, k, M, K = 9, 2, 18, 128 * 150
    pos, q = _pos(rng, T, k, M, 0.0), rng.integers(0, 256, (T, K), dtype=np.uint8)
    s = rng.random((150, T)).astype(np.float32)
    gq, gs = gg.expert_spread(ops.to_dev(q), ops.to_dev(pos), scale=ops.to_dev(s))
    assert np.array_equal(ops.host(gq), ref.spread(q, pos, np.zeros((M, K), np.uint8)))
    assert np.array_equal(ops.host(gs), ref.spread(s.T, pos, np.zeros((M, 150), np.float32)).T)


def _rows(rng, kind, M, N):
    """(device rows, their binary64 values)"""
    if kind == "bf16":
        b = ops.bits(rng, M, N)
        return ops.to_dev(b), oracle._bf16_to_f64(b)
    x = rng.standard_normal((M, N)).astype(np.float32)
    return ops.to_dev(x), x.astype(np.float64)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T,k,M,N", [(0, 2, 4, 8), (1, 1, 1, 8), (5, 2, 10, 72), (3, 8, 24, 1032), (70, 8, 560, 520),
                                     (130, 3, 200, 264), (9, 21, 100, 6144), (4, 5, 0, 16)])
def test_combine(gg, T, k, M, N, kind):
    rng = np.random.default_rng(T + N + k)
    pos = _pos(rng, T, k, M)
    w = rng.standard_normal((T, k)).astype(np.float32)
    Y, y = _rows(rng, kind, M, N)
    for weights in (None, w):
        want, S = ref.combine(y, pos, np.ones((T, k)) if weights is None else w.astype(np.float64))
        dw = None if weights is None else ops.to_dev(w)
        for dt, check in ((torch.float32, ops.check_f32), (torch.bfloat16, ops.check_bf16)):
            got = gg.expert_combine(Y, ops.to_dev(pos), dw, out_dtype=dt)
            check(ops.host(got), want, ops.sum_bound(k, S), "combine")
        assert gg.expert_combine(Y, ops.to_dev(pos), dw).dtype == Y.dtype


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T,k,M,N", [(0, 2, 4, 8), (1, 1, 1, 8), (5, 2, 10, 72), (3, 8, 24, 1032), (70, 8, 560, 520),
                                     (130, 3, 200, 264), (9, 21, 100, 6144), (2, 9, 18, 20000)])
def test_combine_gradient(gg, T, k, M, N, kind):
    rng = np.random.default_rng(T + N + k)
    pos = _pos(rng, T, k, M)
    w = rng.standard_normal((T, k)).astype(np.float32)
    Y, y = _rows(rng, kind, M, N)
    dO, d = _rows(rng, kind, T, N)
    want, want_w, Sw = ref.combine_grad(d, y, pos, w.astype(np.float64))
    out = torch.full_like(Y, 7)
    dY, dw = gg.expert_combine_grad(dO, Y, ops.to_dev(pos), ops.to_dev(w), out=out)
    named = np.zeros(M, bool)
    named[pos[pos >= 0]] = True
    got = ops.host(dY)
    assert (got[~named] == 7).all()
    check = ops.check_f32 if kind == "fp32" else ops.check_bf16
    check(got[named], want[named], 2.0 ** -24 * np.abs(want[named]), "rows")
    # at most N / 64 + 16 additions follow one another
    ops.check_f32(ops.host(dw), want_w, ops.sum_bound(N // 64 + 16, Sw), "weights")
    assert (ops.host(dw)[pos < 0] == 0).all()


def test_masked_places_hold_anything(gg):
    # rows that no choice names, and weights of choices without a row, may be infinite or NaN
    rng = np.random.default_rng(8)
    T, k, M, N = 6, 3, 18, 40
    pos = _pos(rng, T, k, M, 0.5)
    pos[2] = -1
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[pos < 0] = np.nan
    Y, y = _rows(rng, "bf16", M, N)
    free = np.ones(M, bool)
    free[pos[pos >= 0]] = False
    Y[ops.to_dev(free)] = float("nan")
    want, S = ref.combine(np.where(free[:, None], 0.0, y), pos, w.astype(np.float64))
    got = ops.host(gg.expert_combine(Y, ops.to_dev(pos), ops.to_dev(w)))
    ops.check_bf16(got, want, ops.sum_bound(k, S), "combine")
    assert (got[2] == 0).all()
    dO, _ = _rows(rng, "bf16", T, N)
    dY, dw = gg.expert_combine_grad(dO, Y, ops.to_dev(pos), ops.to_dev(w), out=torch.zeros_like(Y))
    assert torch.isfinite(dY).all() and torch.isfinite(dw).all() and (ops.host(dw)[pos < 0] == 0).all()


def test_the_gradient_of_spreading_is_the_combine(gg):
    rng = np.random.default_rng(9)
    T, k, M, N = 33, 4, 140, 264
    pos = _pos(rng, T, k, M)
    dS, d = _rows(rng, "fp32", M, N)
    got = ops.host(gg.expert_combine(dS, ops.to_dev(pos)))
    ops.check_f32(got, *(lambda c, S: (c, ops.sum_bound(k, S)))(*ref.combine(d, pos, np.ones((T, k)))), "gradient")
    # by differences: one element of X up by h moves <dS, spread(X)> by h times it
    X = torch.zeros(T, N, device=DEV)
    for t, n in ((0, 0), (T - 1, N - 1), (17, 100)):
        X.zero_()
        X[t, n] = 1
        moved = (gg.expert_spread(X, ops.to_dev(pos), out=torch.zeros(M, N, device=DEV)).double() * dS.double()).sum()
        assert abs(moved.item() - got[t, n]) <= 2.0 ** -22 * k * np.abs(d).max()


def test_rows_past_2_to_the_32_bytes(gg):
    T, k, M, K = 3, 2, 2 ** 18 + 5, 8192  # 4.3e9 bytes of bf16 rows
    rng = np.random.default_rng(10)
    pos = np.array([[0, M - 1], [M // 2, -1], [M - 2, 2 ** 17 + 1]], np.int32)
    x = ops.bits(rng, T, K)
    out = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    gg.expert_spread(ops.to_dev(x), ops.to_dev(pos), out=out)
    for t in range(T):
        for at in pos[t][pos[t] >= 0]:
            assert torch.equal(out[at], ops.to_dev(x)[t])
    assert int((out != 0).any(1).sum()) == 5
    w = np.array([[1, 2], [-1, 5], [0.5, 0.25]], np.float32)
    v = oracle._bf16_to_f64(x)
    got = ops.host(gg.expert_combine(out, ops.to_dev(pos), ops.to_dev(w)))
    assert np.array_equal(got, oracle.round_to_bf16(v * np.array([[3.0], [-1.0], [0.75]])))
    dY, dw = gg.expert_combine_grad(ops.to_dev(x), out, ops.to_dev(pos), ops.to_dev(w), out=torch.zeros_like(out))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                assert np.array_equal(ops.host(dY[pos[t, j]]), oracle.round_to_bf16(v[t] * w[t, j]))
    assert np.allclose(ops.host(dw), np.where(pos >= 0, (v * v).sum(1, keepdims=True), 0.0), rtol=1e-5)


def test_many_tokens(gg):
    # more tokens than a launch has workgroups beside each other, one column piece each
    T, k, E, K = 300000, 2, 16, 32
    e = torch.randint(0, E + 2, (T, k), dtype=torch.int32, device=DEV)
    off, rows, pos = gg.expert_sort(e, E)
    X = torch.randint(-8, 9, (T, K), device=DEV).bfloat16()
    Xs = gg.expert_spread(X, pos)
    n = int(off[-1])
    assert torch.equal(Xs[:n], X[rows[:n].long()])
    here = (pos >= 0).sum(1, keepdim=True)
    assert torch.equal(gg.expert_combine(Xs, pos, out_dtype=torch.float32), X.float() * here)
