"""The cases on which the expert-gradient and 4-bit operators are measured.

Each case runs one operator on one ragged MoE batch: M routed rows grouped by
expert, group sizes only known on the device. ``run`` computes it either by
the framework's entry points (``own`` true) or in a plain form of elementary
torch operations in 32 bits, one product per expert.

Operators (``op`` of a case):

* ``dgrad``        dA[r] = dC[r] @ B[e].T, the data gradient of the grouped product
* ``dgrad_swiglu`` the data gradient of the down projection with the backward
                   of SwiGLU applied to it: (d gate/up columns, activation)
* ``wgrad``        dB[e] = A_e.T @ dC_e, the weight gradient
* ``quantize``     rows -> 4-bit microscaled blocks -> the values they stand for
* ``quantize_weights`` the same for [E, K, N] weights, blocks along K, [E, N, K] out
* ``mx4``          the grouped product of 4-bit microscaled rows and weights
"""

import math

import numpy as np
import torch

own = False

F32, BF16 = "fp32", "bf16"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the smallest training call: a few rows on a test-sized layer, latency only
        {"name": "dgrad_tiny", "op": "dgrad", "E": 4, "M": 29, "K": 256, "N": 256, "skew": 1.2, "out": F32},
        # data gradient of the headline layer, balanced routing
        {"name": "dgrad_uniform16k", "op": "dgrad", "E": 64, "M": 16384, "K": 1024, "N": 2688, "skew": -1.0, "out": BF16},
        # the down projection's gradient and the SwiGLU backward of the same layer, skewed routing
        {"name": "dgrad_swiglu_skew16k", "op": "dgrad_swiglu", "E": 64, "M": 16384, "K": 1344, "N": 1024, "skew": 1.2, "out": BF16},
        # a small ragged batch on odd sizes
        {"name": "dgrad_swiglu_odd", "op": "dgrad_swiglu", "E": 12, "M": 777, "K": 712, "N": 1000, "skew": 0.8, "out": BF16},
        # weight gradient into fp32 master gradients, balanced routing
        {"name": "wgrad_uniform16k", "op": "wgrad", "E": 64, "M": 16384, "K": 1024, "N": 2688, "skew": -1.0, "out": F32},
        # weight gradient of the headline layer, skewed routing (one expert holds a quarter of the rows)
        {"name": "wgrad_skew16k", "op": "wgrad", "E": 64, "M": 16384, "K": 1024, "N": 2688, "skew": 1.2, "out": BF16},
        # few rows on wide weights: the gradient's own bytes are the work
        {"name": "wgrad_skew2k_wide", "op": "wgrad", "E": 32, "M": 2048, "K": 6144, "N": 4096, "skew": 1.2, "out": BF16},
        # activations of a prompt on their way into the 4-bit product
        {"name": "quantize_rows16k", "op": "quantize", "M": 16384, "K": 6144},
        # the layer's weights, laid out once after training
        {"name": "quantize_weights", "op": "quantize_weights", "E": 64, "K": 1024, "N": 2688},
        # one token's experts: eight rows on eight experts
        {"name": "mx4_single_token", "op": "mx4", "E": 8, "M": 8, "K": 1024, "N": 2688, "skew": -1.0, "out": BF16},
        # the decode shape: 32 experts x 16 rows, weight bytes only
        {"name": "mx4_decode", "op": "mx4", "E": 32, "M": 512, "K": 6144, "N": 4096, "skew": -1.0, "out": F32},
        # a prompt through the gate and up projections, activation fused, skewed routing
        {"name": "mx4_swiglu_skew16k", "op": "mx4", "E": 64, "M": 16384, "K": 1024, "N": 2688, "skew": 1.2, "out": "swiglu"},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(step, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step)

    op = rng.choice(["dgrad", "dgrad", "dgrad_swiglu", "wgrad", "wgrad", "quantize", "quantize_weights", "mx4", "mx4"])
    step = 32 if op in ("quantize", "quantize_weights", "mx4") else 8
    case = {"op": op, "K": log(64, 6144, step)}
    if op == "quantize":
        return dict(case, M=log(1, 16384))
    E = log(1, 128)
    N = log(64, 4096, 8)
    while E * case["K"] * N > 2.5e8:
        E = max(1, E // 2)
    case.update(E=E, N=N)
    if op == "quantize_weights":
        return case
    case.update(M=log(1, 16384), skew=rng.choice([-1.0, 0.0, 0.6, 1.2]))
    while case["M"] * case["K"] * N > 4.5e10:
        case["M"] //= 2
    case["out"] = rng.choice({"dgrad_swiglu": [BF16], "mx4": [F32, BF16, "swiglu"]}.get(op, [F32, BF16]))
    return case


def _shares(case, seed):
    """Each expert's share of the routed rows: rank^-skew, ranks shuffled by the seed."""
    E = case["E"]
    rank = np.random.default_rng([seed, 17]).permutation(E) + 1
    p = rank.astype(np.float64) ** -max(0.0, case["skew"])
    return p / p.sum()


def _group_sizes(case, seed):
    """Rows of each expert: an even split (skew < 0), or every row drawn by the shares."""
    E, M = case["E"], case["M"]
    if case["skew"] < 0:
        return [M // E + (e < M % E) for e in range(E)]
    return np.random.default_rng([seed, 19]).multinomial(M, _shares(case, seed)).tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, K = case["op"], case["K"]
    s = {"op": op, "out": case.get("out")}

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()

    def activations(rows, cols):
        # a few columns run several times hotter than the rest
        heat = torch.exp(0.8 * torch.randn(cols, generator=gen, device="cuda"))
        return (torch.randn(rows, cols, generator=gen, device="cuda") * heat).bfloat16()

    if op == "quantize":
        return dict(s, X=activations(case["M"], K))
    if op == "quantize_weights":
        return dict(s, B=normal(case["E"], K, case["N"], scale=1 / math.sqrt(K)))
    E, M, N = case["E"], case["M"], case["N"]
    s["sizes"] = _group_sizes(case, seed)
    s["offsets"] = torch.tensor(np.cumsum([0] + s["sizes"]), dtype=torch.int32, device="cuda")
    if op == "mx4":
        s["Aq"], s["a_scale"] = _mx4_codes(activations(M, K).float())
        w = [_mx4_codes(normal(N, K, scale=1 / math.sqrt(K)).float()) for _ in range(E)]
        s["Bq"], s["b_scale"] = torch.stack([q for q, _ in w]), torch.stack([c for _, c in w])
        return s
    s["B"] = normal(E, K, N, scale=1 / math.sqrt(K)) if op != "wgrad" else None
    s["dC"] = normal(M, N, scale=0.02)
    if op == "wgrad":
        s["A"] = activations(M, K)
    if op == "dgrad_swiglu":
        s["C"] = normal(M, 2 * K, scale=1.5)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import moe_ragged_grouped_amd as gg

    op = s["op"]
    dt = torch.float32 if s["out"] == F32 else torch.bfloat16
    if op == "dgrad":
        return gg.grouped_gemm_dgrad(s["dC"], s["B"], s["offsets"], out_dtype=dt)
    if op == "dgrad_swiglu":
        return gg.grouped_gemm_dgrad_swiglu(s["dC"], s["B"], s["offsets"], s["C"], with_h=True)
    if op == "wgrad":
        return gg.grouped_gemm_wgrad(s["A"], s["dC"], s["offsets"], out_dtype=dt)
    if op == "quantize":
        return gg.mx4_dequantize(*gg.mx4_quantize(s["X"]))
    if op == "quantize_weights":
        return gg.mx4_dequantize(*gg.mx4_quantize_weights(s["B"]))
    if s["out"] == "swiglu":
        return gg.grouped_gemm_mx4_swiglu(s["Aq"], s["a_scale"], s["Bq"], s["b_scale"], s["offsets"])
    return gg.grouped_gemm_mx4(s["Aq"], s["a_scale"], s["Bq"], s["b_scale"], s["offsets"], out_dtype=dt)


def _run_plain(s):
    op = s["op"]
    dt = torch.float32 if s["out"] == F32 else torch.bfloat16
    if op == "quantize":
        return _mx4_values(*_mx4_codes(s["X"].float())).bfloat16()
    if op == "quantize_weights":
        return _mx4_values(*_mx4_codes(s["B"].float().transpose(1, 2))).bfloat16()
    if op == "wgrad":
        pairs = zip(s["A"].float().split(s["sizes"]), s["dC"].float().split(s["sizes"]))
        return torch.stack([a.t() @ d for a, d in pairs]).to(dt)
    if op == "mx4":
        rows = _mx4_values(s["Aq"], s["a_scale"]).split(s["sizes"])
        weights = zip(s["Bq"], s["b_scale"])
        C = torch.cat([a @ _mx4_values(q, c).t() for a, (q, c) in zip(rows, weights)])
        if s["out"] != "swiglu":
            return C.to(dt)
        gate, up = C[:, 0::2], C[:, 1::2]
        return (gate / (1 + torch.exp(-gate)) * up).to(dt)
    dA = torch.cat([d @ b.float().t() for d, b in zip(s["dC"].float().split(s["sizes"]), s["B"])])
    if op == "dgrad":
        return dA.to(dt)
    gate, up = s["C"].float()[:, 0::2], s["C"].float()[:, 1::2]
    sig = 1 / (1 + torch.exp(-gate))
    d_gate, d_up = dA * up * sig * (1 + gate * (1 - sig)), dA * gate * sig
    return torch.stack([d_gate, d_up], dim=2).flatten(1).to(dt), (gate * sig * up).to(dt)


def _mx4_codes(x):
    """fp32 [..., M, K] -> E2M1 codes [..., M, K/2] (even k in the low half byte) and E8M0
    scale codes, slice by slice of 256 k: [..., K/256, M, 8], zeros behind the last block.

    A block's scale is 2^(floor(log2 max|x|) - 2); x over the scale goes to the
    nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code, at most 6."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127)
    # two factors: one of 2^127 at most each, so that neither overflows
    y = (b * torch.exp2(-(e // 2).float())[..., None] * torch.exp2(-(e - e // 2).float())[..., None])
    a = y.abs()
    a = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    code = (a.clamp(max=7) + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    scale = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[-1] % 8))
    scale = scale.unflatten(-1, (-1, 8)).transpose(-3, -2).contiguous()
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def _by_row(scale, blocks):
    """Scale codes [..., K/256, M, 8] -> [..., M, K/32]."""
    return scale.transpose(-3, -2).flatten(-2)[..., :blocks]


def _mx4_values(q, scale):
    """The fp32 values that codes and scales stand for."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    v = torch.stack([grid[(q & 15).int()], grid[(q >> 4).int()]], dim=-1).flatten(-2).unflatten(-1, (-1, 32))
    return (v * torch.exp2(_by_row(scale, v.shape[-2]).float() - 127)[..., None]).flatten(-2)


def work(case):
    op, K = case["op"], case["K"]
    if op == "quantize":  # rows in; codes, scales and the values they stand for out
        return {"bytes": case["M"] * K * (2 + 0.5 + 1 / 32 + 2), "flops": 0}
    E, N = case["E"], case["N"]
    if op == "quantize_weights":
        return {"bytes": E * K * N * (2 + 0.5 + 1 / 32 + 2), "flops": 0}
    M = case["M"]
    ob = 4 if case["out"] == F32 else 2
    # experts that get a row, whose weights have to be read
    busy = min(E, M) if case["skew"] < 0 else float(np.sum(1 - (1 - _shares(case, 0)) ** M))
    flops = 2 * M * K * N
    if op == "dgrad":
        return {"bytes": M * N * 2 + busy * K * N * 2 + M * K * ob, "flops": flops}
    if op == "dgrad_swiglu":
        return {"bytes": M * N * 2 + busy * K * N * 2 + M * K * (4 + 4 + 2), "flops": flops}
    if op == "wgrad":
        return {"bytes": M * (K + N) * 2 + E * K * N * ob, "flops": flops}
    q = 0.5 + 1 / 32
    return {"bytes": M * K * q + busy * K * N * q + M * N * (1 if case["out"] == "swiglu" else ob), "flops": flops}


def exact(case, seed):
    """What run() returns for these inputs, in 64 bits, straight from the definitions."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_rounding(s["X"].double())
    if op == "quantize_weights":
        return torch.stack([_exact_rounding(b.double().t().contiguous()) for b in s["B"]])
    ends = np.cumsum(s["sizes"])
    spans = [slice(int(b) - m, int(b)) for b, m in zip(ends, s["sizes"])]
    if op == "wgrad":
        A, dC = s["A"].double(), s["dC"].double()
        out = torch.empty(case["E"], case["K"], case["N"], dtype=torch.float64, device="cuda")
        for e, rows in enumerate(spans):
            torch.matmul(A[rows].t(), dC[rows], out=out[e])
        return out
    if op == "mx4":
        A = _exact_values(s["Aq"], s["a_scale"])
        C = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for e, rows in enumerate(spans):
            C[rows] = A[rows] @ _exact_values(s["Bq"][e], s["b_scale"][e]).t()
        return C if case["out"] != "swiglu" else C[:, 0::2] * torch.sigmoid(C[:, 0::2]) * C[:, 1::2]
    dC = s["dC"].double()
    dA = torch.empty(case["M"], case["K"], dtype=torch.float64, device="cuda")
    for e, rows in enumerate(spans):
        dA[rows] = dC[rows] @ s["B"][e].double().t()
    if op == "dgrad":
        return dA
    C = s["C"].double()
    g, u = C[:, 0::2], C[:, 1::2]
    sg = torch.sigmoid(g)
    d = torch.empty_like(C)
    d[:, 0::2] = dA * u * (sg + g * sg * (1 - sg))
    d[:, 1::2] = dA * g * sg
    return d, g * sg * u


def _exact_values(q, scale):
    """E2M1 bits as sign, two exponent bits and one mantissa bit; E8M0 as a power of two."""
    c = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).double()
    sign, low = 1 - 2 * torch.floor(c / 8), torch.remainder(c, 8)
    ex, man = torch.floor(low / 2), torch.remainder(low, 2)
    v = torch.where(ex == 0, man / 2, (1 + man / 2) * torch.exp2(ex - 1))
    blocks = torch.stack([scale[b // 8, :, b % 8] for b in range(c.shape[-1] // 32)], dim=-1)
    return sign * v * torch.exp2(blocks.double() - 127).repeat_interleave(32, dim=-1)


def _exact_rounding(x):
    """x [rows, K] rounded to the nearest 4-bit value of its block, by distance to the grid's midpoints."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    # frexp: top = f * 2^e with f in [.5, 1), so floor(log2 top) = e - 1
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127)
    scale = torch.exp2(e.double())
    y = b.abs() / scale
    # a tie goes to the even code: up out of an odd code, down out of an even one
    borders = zip(E2M1, E2M1[1:], (torch.gt, torch.ge) * 4)
    v = sum((hi - lo) * above(y, (lo + hi) / 2) for lo, hi, above in borders)
    return (torch.sign(b) * v * scale).reshape(x.shape)
