"""Random shapes through every entry point of the gradients and the 4-bit operators.

Each seed draws one ragged problem: up to 400 experts, some empty, most small, a few of
several hundred rows, K and N any multiple of 8 (of 32 for K in 4 bits), spare rows, a
random tile height. Sums are exact in fp32 and compared for equality with binary64; the
SwiGLU forms and the quantisers are checked as their own tests check them.

The default is a short run of 8 seeds. GG_SWEEP="lo:hi" runs seeds lo..hi-1 instead
(seeds 100..549 have been run through this module in full).
"""

import os

import numpy as np
import pytest

import oracle.operators as ref
from tests import operators as ops
from tests.test_ring_tiles_gpu import (DEV, SMALL, SPARE, _codes, _dgrad, _dgrad_swiglu, _gen, _ints, _mx4,
                                       _mx4_swiglu, _mx4_want, _offsets)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _seeds():
    lo, hi = (int(x) for x in os.environ.get("GG_SWEEP", "100:108").split(":"))
    return range(lo, hi)


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _problem(seed):
    rng = np.random.default_rng(9000 + seed)
    E = int(np.exp(rng.uniform(0, np.log(401))))
    K, N = (8 * int(np.exp(rng.uniform(0, np.log(161)))) for _ in range(2))
    kind = rng.random(E)
    sizes = np.where(kind < 0.25, 0, np.where(kind < 0.85, rng.integers(1, 40, E), rng.integers(40, 900, E)))
    cap = 6e8 / (K * N)
    if sizes.sum() > cap:
        sizes = np.floor(sizes * (cap / sizes.sum())).astype(np.int64)
    bm = [0, 0, 0, 16, 32, 64, 128, 256][int(rng.integers(8))]
    return [int(m) for m in sizes], K, N, bm


def _wgrad(gg, sizes, K, N, seed):
    gen = _gen(seed)
    M = sum(sizes)
    A, dC, off = _ints(gen, M + SPARE, K), _ints(gen, M + SPARE, N), _offsets(sizes)
    parts = zip(A[:M].double().split(sizes), dC[:M].double().split(sizes))
    want = torch.stack([a.t().contiguous() @ d for a, d in parts])
    for dtype in (torch.float32, torch.bfloat16):
        got = torch.full(want.shape, float("nan"), dtype=dtype, device=DEV)
        gg.grouped_gemm_wgrad(A, dC, off, out=got)
        assert torch.equal(got, want.to(dtype)), dtype
    got = _ints(gen, *want.shape).float()
    want += got.double()
    gg.grouped_gemm_wgrad(A, dC, off, out=got, accumulate=True)
    assert torch.equal(got.double(), want)


def _quantize(gg, E, M, K, N, seed):
    rng = np.random.default_rng(seed)
    x = ops.bits(rng, min(M, 300), K, scale=float(np.exp(rng.uniform(-20, 20))))
    b = ops.bits(rng, min(E, 3), K, N)
    for got, bits in ((gg.mx4_quantize(ops.to_dev(x)), x),
                      (gg.mx4_quantize_weights(ops.to_dev(b)), np.ascontiguousarray(np.swapaxes(b, 1, 2)))):
        want = ref.mx4_encode(bits)
        assert all((ops.host(g) == w).all() for g, w in zip(got, want))
        assert (ops.host(gg.mx4_dequantize(*got)) == ref.mx4_values(*want)).all()


@pytest.mark.parametrize("seed", _seeds())
def test_every_operator(gg, seed):
    sizes, K, N, bm = _problem(seed)
    K4 = max(32, K // 32 * 32)
    print("sweep seed %d: E=%d rows=%d K=%d N=%d bm=%d" % (seed, len(sizes), sum(sizes), K, N, bm), flush=True)
    _dgrad(gg, sizes, K, N, bm, seed)
    _dgrad_swiglu(gg, sizes, K, N, bm, seed)
    _wgrad(gg, sizes, K, N, seed)
    _quantize(gg, len(sizes), sum(sizes) + 1, K4, N, seed)
    _mx4(gg, sizes, K4, N, bm, seed)
    codes = _codes(_gen(seed), sizes, K4, N, SMALL)
    _mx4_swiglu(gg, codes, _mx4_want(codes, sizes), sizes, K4, N, bm, "seed %d" % seed)
