"""An expert layer out of the operators, forward and backward, and how its calls behave on
streams, in graphs and at the host's errors (needs an MI355X)."""

import numpy as np
import pytest

import oracle
import oracle.layer as ref
from tests import operators as ops
from tests import parity

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
T, K_TOP, E, D, I = 96, 2, 5, 256, 144  # tokens, choices, experts, the tokens' width, the experts' width


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_ragged_grouped_amd as m
    m.load_library()
    return m


def _layer(seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(s, generator=gen, device=DEV) * scale).to(BF)  # noqa: E731
    return dict(x=r(T, D), res=r(T, D), g=(1 + 0.1 * r(D).float()).to(BF), router=r(D, E, scale=0.2),
                w1=r(E, D, 2 * I, scale=D ** -0.5), w2=r(E, I, D, scale=I ** -0.5))


def _served(gg, p, W1, W2):
    """One layer, served in 8 bits; everything it computes on its way."""
    q, s, z, y = gg.rms_norm_fp8(p["x"], p["g"], residual=p["res"], with_norm=True)
    top, experts = torch.softmax(y.float() @ p["router"].float(), 1).topk(K_TOP, 1)
    weights = top / top.sum(1, keepdim=True)
    off, rows, pos = gg.expert_sort(experts, E)
    xq, xs = gg.expert_spread(q, pos, scale=s)
    h = gg.grouped_gemm_fp8_block_swiglu(xq, xs, *W1, off)
    hq, hs = gg.fp8_quantize(h)
    c = gg.grouped_gemm_fp8_block(hq, hs, *W2, off, out_dtype=BF)
    out = gg.expert_combine(c, pos, weights)
    return dict(q=q, s=s, z=z, y=y, experts=experts, weights=weights, off=off, rows=rows, pos=pos, xq=xq, xs=xs, h=h,
                hq=hq, hs=hs, c=c, out=out)


def _np(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == F8 else ops.host(t)


def _f64(t):
    return ops.host(t).astype(np.float64)


def test_served_layer(gg):
    # each step against binary64 on what the steps before it gave
    p = _layer(0)
    W1, W2 = gg.fp8_quantize_weights(p["w1"]), gg.fp8_quantize_weights(p["w2"])
    r = _served(gg, p, W1, W2)
    z, y = ref.norm(_f64(p["x"]), _f64(p["res"]), _f64(p["g"]), 1e-6)
    assert np.array_equal(_np(r["z"]), z)
    ops.check_bf16(_np(r["y"]), y, ref.NORM_REL * np.abs(y), "norm")
    off, rows, pos, _ = ref.sort(_np(r["experts"]), E)
    for a, b in ((r["off"], off), (r["rows"], rows), (r["pos"], pos)):
        assert np.array_equal(_np(a), b)
    assert np.array_equal(_np(r["xq"]), _np(r["q"])[rows]) and np.array_equal(_np(r["xs"]), _np(r["s"])[:, rows])
    C, S, G = ref.fp8_product(_np(r["xq"]), _np(r["xs"]), _np(W1[0]), _np(W1[1]), off)
    parity.check_swiglu_bf16(_np(r["h"]), C, S, "hidden", err=ref.fp8_product_error(S, G, D))
    hq, hs = ref.fp8_rows(ops.bits_of(r["h"]))
    assert np.array_equal(_np(r["hq"]), hq) and np.array_equal(_np(r["hs"]), hs)
    C, S, G = ref.fp8_product(hq, hs, _np(W2[0]), _np(W2[1]), off)
    ops.check_bf16(_np(r["c"]), C, ref.fp8_product_error(S, G, I), "rows")
    want, S = ref.combine(_f64(r["c"]), pos, _f64(r["weights"]))
    ops.check_bf16(_np(r["out"]), want, ops.sum_bound(K_TOP, S), "out")
    # and the whole of it is near the layer in binary64: five roundings of 2^-4 relative at most
    # (rows, weights, hidden rows, weights, and the activation's slope), far from all of one sign
    x1, exact = _f64(r["y"])[rows], np.zeros((T * K_TOP, D))
    for e in range(E):
        c1 = x1[off[e]:off[e + 1]] @ _f64(p["w1"][e])
        exact[off[e]:off[e + 1]] = (oracle.silu(c1[:, 0::2]) * c1[:, 1::2]) @ _f64(p["w2"][e])
    exact, _ = ref.combine(exact, pos, _f64(r["weights"]))
    assert np.linalg.norm(_f64(r["out"]) - exact) < 5 * 2.0 ** -4 * np.linalg.norm(exact)


def test_trained_layer(gg):
    # forward in bf16 between the new steps, backward through all of them, against autograd in
    # binary64 on the same choices
    p = _layer(1)
    q, s, z, y = gg.rms_norm_fp8(p["x"], p["g"], residual=p["res"], with_norm=True)
    top, experts = torch.softmax(y.float() @ p["router"].float(), 1).topk(K_TOP, 1)
    off, rows, pos = gg.expert_sort(experts, E)
    X = gg.expert_spread(y, pos)
    C = gg.grouped_gemm(X, p["w1"], off, out_dtype=BF)
    H = gg.grouped_gemm_swiglu(X, p["w1"], off)
    Y = gg.grouped_gemm(H, p["w2"], off, out_dtype=BF)
    out = gg.expert_combine(Y, pos, top.contiguous())
    dO = (torch.randn(T, D, device=DEV) * 0.1).to(BF)
    dz_past = (torch.randn(T, D, device=DEV) * 0.1).to(BF)
    dY, dw = gg.expert_combine_grad(dO, Y, pos, top.contiguous())
    dC, H2 = gg.grouped_gemm_dgrad_swiglu(dY, p["w2"], off, C, with_h=True)
    dW2 = gg.grouped_gemm_wgrad(H2, dY, off)
    dX = gg.grouped_gemm_dgrad(dC, p["w1"], off, out_dtype=BF)
    dW1 = gg.grouped_gemm_wgrad(X, dC, off)
    dy = gg.expert_combine(dX, pos)
    dz, dg = gg.rms_norm_grad(dy, z, p["g"], d_residual=dz_past)

    leaf = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    tz, tg, tw, w1, w2 = leaf(z), leaf(p["g"]), leaf(top), leaf(p["w1"]), leaf(p["w2"])
    ty = tz / torch.sqrt((tz * tz).mean(1, keepdim=True) + 1e-6) * tg
    ex = experts.cpu()
    total = torch.zeros(T, D, dtype=torch.float64)
    for e in range(E):
        c1 = ty @ w1[e]
        h = torch.nn.functional.silu(c1[:, 0::2]) * c1[:, 1::2]
        total = total + (tw * (ex == e)).sum(1, keepdim=True) * (h @ w2[e])
    ((total * dO.double().cpu()).sum() + (tz * dz_past.double().cpu()).sum()).backward()
    # each tensor passes at most six bf16 roundings (2^-8 relative each) of what it is made of,
    # with as many of its factors rounded: twelve of them bound the norm of the error
    for name, got, want in (("out", out, total), ("dw", dw, tw.grad), ("dW2", dW2, w2.grad), ("dW1", dW1, w1.grad),
                            ("dz", dz, tz.grad), ("dg", dg, tg.grad)):
        d = (got.double().cpu() - want.detach()).norm() / want.detach().norm()
        assert d < 12 * 2.0 ** -8, (name, d)


def _calls(gg, seed=0):
    """{name: a call of every entry point, taking a stream}"""
    p = _layer(seed)
    rng = np.random.default_rng(seed)
    e = torch.from_numpy(rng.integers(-1, E + 1, (T, K_TOP)).astype(np.int32)).to(DEV)
    many = torch.from_numpy(rng.integers(0, E, (6000, K_TOP)).astype(np.int32)).to(DEV)
    w = torch.from_numpy(rng.random((T, K_TOP)).astype(np.float32)).to(DEV)
    off, rows, pos, rw = gg.expert_sort(e, E, weights=w)
    q, s = gg.fp8_quantize(p["x"])
    W1 = gg.fp8_quantize_weights(p["w1"])
    Xs = gg.expert_spread(p["x"], pos, out=torch.zeros(T * K_TOP, D, dtype=BF, device=DEV))
    xq, xs = gg.fp8_quantize(Xs)
    n = T * K_TOP
    # rows that nothing names stay as they are here, so that whole outputs compare
    zeros = lambda *shape, dt=BF: torch.zeros(shape, dtype=dt, device=DEV)  # noqa: E731
    c, h, sq, ss, dy = zeros(n, 2 * I, dt=F32), zeros(n, I), zeros(n, D, dt=torch.uint8).view(F8), zeros(2, n, dt=F32), zeros(n, D)
    calls = {
        "fp8_quantize": lambda st: gg.fp8_quantize(p["x"], stream=st),
        "fp8_quantize_weights": lambda st: gg.fp8_quantize_weights(p["w1"], stream=st),
        "grouped_gemm_fp8_block": lambda st: (gg.grouped_gemm_fp8_block(xq, xs, *W1, off, out=c, stream=st),),
        "grouped_gemm_fp8_block_swiglu": lambda st: (gg.grouped_gemm_fp8_block_swiglu(xq, xs, *W1, off, out=h, stream=st),),
        "expert_sort": lambda st: gg.expert_sort(e, E, weights=w, stream=st),
        "expert_sort split": lambda st: gg.expert_sort(many, E, stream=st),
        "expert_spread": lambda st: gg.expert_spread(q, pos, scale=s, stream=st, out=sq, out_scale=ss),
        "expert_combine": lambda st: (gg.expert_combine(Xs, pos, w, stream=st),),
        "expert_combine_grad": lambda st: gg.expert_combine_grad(p["x"], Xs, pos, w, out=dy, stream=st),
        "rms_norm_fp8": lambda st: gg.rms_norm_fp8(p["x"], p["g"], residual=p["res"], with_norm=True, stream=st),
        "rms_norm_grad": lambda st: gg.rms_norm_grad(p["res"], p["x"], p["g"], stream=st),
    }
    return calls


def _equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


NAMES = ["fp8_quantize", "fp8_quantize_weights", "grouped_gemm_fp8_block", "grouped_gemm_fp8_block_swiglu", "expert_sort",
         "expert_sort split", "expert_spread", "expert_combine", "expert_combine_grad", "rms_norm_fp8", "rms_norm_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_a_call_waits_for_its_stream(gg, name):
    # on a busy stream, current or named, the result is that of the idle one
    call = _calls(gg)[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(ops.SLEEP // 10)
        got = call(None)
    st.synchronize()
    assert _equal(got, want)
    with torch.cuda.stream(st):
        torch.cuda._sleep(ops.SLEEP // 10)
    got = call(st)
    st.synchronize()
    assert _equal(got, want)


def test_two_streams_at_once(gg):
    calls = [_calls(gg, seed) for seed in (0, 1)]
    want = [{n: [t.clone() for t in c(None)] for n, c in x.items()} for x in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [{} for _ in calls]
    for n in NAMES:
        for x, st, g in zip(calls, streams, got):
            with torch.cuda.stream(st):
                g[n] = [x[n](None) for _ in range(3)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for n in NAMES:
            for one in g[n]:
                assert _equal(one, w[n]), n


def test_graph_replays(gg):
    # every call captured once, two graphs of them with memory of their own, replayed in turn on
    # other inputs with eager work between
    p = _layer(5)
    rng = np.random.default_rng(5)
    e = torch.zeros((T, K_TOP), dtype=torch.int32, device=DEV)
    many = torch.zeros((6000, K_TOP), dtype=torch.int32, device=DEV)
    w = torch.zeros((T, K_TOP), device=DEV)
    n = T * K_TOP

    def step():
        W1, W2 = gg.fp8_quantize_weights(p["w1"]), gg.fp8_quantize_weights(p["w2"])
        q, s, z, y = gg.rms_norm_fp8(p["x"], p["g"], residual=p["res"], with_norm=True)
        off, rows, pos, rw = gg.expert_sort(e, E, weights=w)
        big = gg.expert_sort(many, E)
        xq, xs = gg.expert_spread(q, pos, scale=s, out=torch.zeros(n, D, dtype=torch.uint8, device=DEV).view(F8),
                                  out_scale=torch.zeros(2, n, device=DEV))
        h = torch.zeros(n, I, dtype=BF, device=DEV)
        gg.grouped_gemm_fp8_block_swiglu(xq, xs, *W1, off, out=h)
        hq, hs = gg.fp8_quantize(h)
        c = gg.grouped_gemm_fp8_block(hq, hs, *W2, off, out=torch.zeros(n, D, device=DEV))
        out = gg.expert_combine(c, pos, w)
        dY, dw = gg.expert_combine_grad(out, c, pos, w, out=torch.zeros_like(c))
        dz, dg = gg.rms_norm_grad(y, z, p["g"])
        return [q, s, z, y, off, rows, pos, rw, *big, xq, xs, h, hq, hs, c, out, dY, dw, dz, dg]

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for turn in range(6):
        new = _layer(10 + turn % 3)
        for k in p:
            p[k].copy_(new[k])
        e.copy_(torch.from_numpy(rng.integers(-1, E + 1, (T, K_TOP)).astype(np.int32)))
        many.copy_(torch.from_numpy(rng.integers(-1, E + 1, (6000, K_TOP)).astype(np.int32)))
        w.copy_(torch.from_numpy(rng.random((T, K_TOP)).astype(np.float32)))
        torch.cuda.synchronize()
        graphs[turn % 2].replay()
        want = step()
        if turn % 2:
            graphs[0].replay()
        torch.cuda.synchronize()
        assert _equal(outs[turn % 2], want)
        assert _equal(outs[0], want) or turn % 2 == 0


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_a_named_stream_may_be_dropped(gg, name):
    # inputs that nothing holds any more are kept until the named stream has passed the call
    want = [t.clone() for t in _calls(gg)[name](None)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    calls = _calls(gg)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(ops.SLEEP // 4)
    got = calls[name](st)
    del calls
    spoil = [torch.full((m,), 7.0, device=DEV) for m in (128, 1024, 2 ** 14, 2 ** 15, 2 ** 17, 2 ** 18) for _ in range(12)]
    torch.cuda.current_stream().synchronize()
    st.synchronize()
    assert _equal(got, want)
    del spoil


def test_an_earlier_error_of_the_runtime_is_not_the_calls(gg):
    lib = gg.load_library()
    for name, call in _calls(gg).items():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        assert lib.hipSetDevice(12345) != 0  # refused: there is no such device
        got = call(None)
        lib.hipGetLastError()
        torch.cuda.synchronize()
        assert _equal(got, want), name


def test_refusals(gg):
    bf = torch.zeros((4, 40), dtype=BF, device=DEV)
    for call, status in ((lambda: gg.fp8_quantize(bf), "status 2"),
                         (lambda: gg.rms_norm_fp8(bf, bf[0].clone()), "status 2"),
                         (lambda: gg.expert_spread(bf[:, :4].contiguous(), torch.zeros((4, 1), dtype=torch.int32, device=DEV)),
                          "status 2"),
                         (lambda: gg.expert_sort(torch.zeros((4, 1), dtype=torch.int32, device=DEV), 1025), "status 3"),
                         (lambda: gg.expert_sort(torch.zeros((4, 1), dtype=torch.int32, device=DEV), 0), "status 1"),
                         (lambda: gg.expert_combine(bf, torch.zeros((4, 1), dtype=torch.int32, device=DEV), out=bf),
                          "status 1")):
        with pytest.raises(gg.GroupedGemmError, match=status):
            call()
