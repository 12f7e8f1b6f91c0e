"""The stream argument of the forward entry points (needs an MI355X).

A call on a named stream is ordered on that stream alone: what it makes and
clears is made there, and its tensors may be dropped as soon as it returns.
"""

import numpy as np
import pytest

from tests import operators as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E, M, K, N = 2, 512, 512, 512
E4M3_ONE = 0x38


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _ones(*shape, dtype=torch.bfloat16):
    return torch.ones(shape, dtype=dtype, device="cuda:0")


def _codes(*shape):
    return torch.full(shape, E4M3_ONE, dtype=torch.uint8, device="cuda:0")


def _rows():
    return torch.arange(M, dtype=torch.int32, device="cuda:0")


def _off():
    return torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda:0")


F32 = torch.float32
CALLS = {
    "grouped_gemm": (lambda: (_ones(M, K), _ones(E, K, N), _off()), K),
    "grouped_gemm_swiglu": (lambda: (_ones(M, K), _ones(E, K, N), _off()), K * K),
    "grouped_gemm_gather": (lambda: (_ones(M, K), _rows(), _ones(E, K, N), _off(), _rows()), K),
    "grouped_gemm_gather_combine": (lambda: (_ones(M, K), _rows(), _ones(E, K, N), _off(), _rows(), _ones(M, dtype=F32)), K),
    "grouped_gemm_fp8w": (lambda: (_ones(M, K), _codes(E, K, N), _ones(E, N, dtype=F32), _off()), K),
    "grouped_gemm_fp8": (lambda: (_codes(M, K), _ones(M, dtype=F32), _codes(E, K, N), _ones(E, N, dtype=F32), _off()), K),
    "grouped_gemm_fp8_swiglu": (lambda: (_codes(M, K), _ones(M, dtype=F32), _codes(E, K, N), _ones(E, N, dtype=F32), _off()),
                                K * K),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_dropped_after_the_call(gg, name):
    make, want = CALLS[name]
    getattr(gg, name)(*make())  # a kernel's first launch loads it, which takes its time

    def attempt(s):
        torch.cuda.empty_cache()
        args = make()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(ops.SLEEP)
        got = getattr(gg, name)(*args, stream=s)
        del args
        spoil = [torch.full((n,), 7.0, device="cuda:0") for n in (128, 1024, 2 ** 17, 2 ** 18) for _ in range(12)]
        torch.cuda.current_stream().synchronize()
        in_time = not s.query()  # the memory was written before the call ran
        s.synchronize()
        assert (got == want).all()
        del spoil
        return in_time

    ops.beside(attempt)


@pytest.mark.parametrize("name", CALLS)
def test_results_are_made_in_the_named_streams_order(gg, name):
    # memory that the present stream gave back but still writes to is no place for them
    make, want = CALLS[name]
    args = make()
    getattr(gg, name)(*args)

    def attempt(s):
        torch.cuda.empty_cache()
        old = [torch.empty((M, n), dtype=dt, device="cuda:0") for n in (N, N // 2) for dt in (F32, torch.bfloat16)]
        torch.cuda._sleep(ops.SLEEP)
        for t in old:
            t.fill_(7.0)
        del old, t
        got = getattr(gg, name)(*args, stream=s)
        s.synchronize()
        in_time = not torch.cuda.current_stream().query()  # the call was through before the writing
        torch.cuda.synchronize()
        assert (got == want).all()
        return in_time

    ops.beside(attempt)


def test_an_earlier_error_of_the_runtime_is_not_the_calls(gg):
    # another caller's refused call leaves its error in the runtime: these launches went through
    X, off = _ones(M, K), _off()
    W, C = _ones(E, K, N), torch.zeros((M, 2 * K), dtype=torch.bfloat16, device="cuda:0")
    q, w = gg.mx4_quantize(X), gg.mx4_quantize_weights(W)
    u8 = lambda t: torch.zeros_like(t)  # noqa: E731
    calls = [
        (lambda out: gg.grouped_gemm_dgrad(X, W, off, out=out), _ones(M, K, dtype=F32), float(N)),
        (lambda out: gg.grouped_gemm_dgrad_swiglu(X, W, off, C, out=out), _ones(M, 2 * K), 0.0),
        (lambda out: gg.grouped_gemm_wgrad(X, X, off, out=out), _ones(E, K, K, dtype=F32), M / 2.0),
        (lambda out: gg.mx4_quantize(X, out=out, out_scale=u8_scale[0]), u8(q[0]), 0x66),
        (lambda out: gg.mx4_quantize_weights(W, out=out, out_scale=u8_scale[1]), u8(w[0]), 0x66),
        (lambda out: gg.mx4_dequantize(*q, out=out), _ones(M, K).mul_(3), 1.0),
        (lambda out: gg.grouped_gemm_mx4(*q, *w, off, out=out), _ones(M, N, dtype=F32), float(K))]
    u8_scale = (u8(q[1]), u8(w[1]))
    lib = gg.load_library()
    for call, out, want in calls:
        call(out)
        out.zero_().add_(5)
        torch.cuda.synchronize()
        assert lib.hipSetDevice(12345) != 0  # refused: there is no such device
        call(out)
        lib.hipGetLastError()
        torch.cuda.synchronize()
        assert (out == want).all()


def test_tile_schedule_on_a_busy_stream(gg):
    off = _off()
    want, n = gg.tile_schedule(off, N, M)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(ops.SLEEP)
    got, count = gg.tile_schedule(off, N, M, stream=s)
    assert count == n > 0 and torch.equal(got, want)
    assert np.array_equal(got.cpu().numpy(), want.cpu().numpy())
