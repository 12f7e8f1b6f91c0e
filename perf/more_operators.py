"""The cases on which routing, the norm before it and the 8-bit block-scaled product are measured.

An expert layer normalises its tokens, sorts them by the experts that their
router chose, multiplies each expert's rows by its weights and brings the rows
back, each times its weight. ``run`` computes one of these steps either by the
framework's entry points (``own`` true) or in a plain form of elementary torch
operations in 32 bits.

Operators (``op`` of a case):

* ``sort``     choices [T, k] -> rows grouped by expert: the groups' offsets, each
               row's token and weight, each choice's place, and the rows themselves
* ``combine``  each token's k rows times their weights, summed; or its gradient:
               that of the rows and that of the weights
* ``norm``     root-mean-square norm of X + residual in 8 bits, a scale for each
               block of 128 values of a row; or the gradient of the norm
* ``product``  the grouped product of 8-bit rows (a scale for 128 values along K)
               and 8-bit weights (a scale for 128 x 128 values)
* ``weights``  bf16 weights [E, K, N] -> 8 bits [E, N, K], the operand of that product

8 bits are E4M3: sign, 4 exponent and 3 mantissa bits, 448 at most. A block is
multiplied by 448 over its largest magnitude (2^-100 at least), cut to 16
significant bits, so that the product with a bf16 value is exact in 32 bits, and
rounded to the nearest code; its scale is the inverse of that multiplier.
"""

import math

import numpy as np
import torch

own = False

F32, BF16, FP8 = "fp32", "bf16", "fp8"
TOP, LEAST, EPS = 448.0, 2.0 ** -100, 1e-6
F8 = torch.float8_e4m3fn


def listed():
    return [
        # a step of serving: 64 sequences, one token each, on 32 experts
        {"name": "sort_decode", "op": "sort", "T": 64, "k": 8, "E": 32, "ranks": 1, "skew": 0.6, "K": 6144, "rows": FP8},
        # the headline batch: 16384 routed rows on 64 experts, in training
        {"name": "sort_16k", "op": "sort", "T": 2048, "k": 8, "E": 64, "ranks": 1, "skew": 1.2, "K": 1024, "rows": BF16},
        # a prompt on one of 8 ranks that share 256 experts: most choices live elsewhere
        {"name": "sort_rank_of_8", "op": "sort", "T": 16384, "k": 8, "E": 32, "ranks": 8, "skew": 0.6, "K": 1024, "rows": BF16},
        # the expert rows of a prompt on their way back to its tokens
        {"name": "combine_16k", "op": "combine", "grad": False, "T": 2048, "k": 8, "E": 64, "ranks": 1, "skew": 1.2, "K": 6144, "rows": BF16},
        # the same in training, backward, with an odd number of tokens
        {"name": "combine_grad_16k", "op": "combine", "grad": True, "T": 2051, "k": 8, "E": 64, "ranks": 1, "skew": 1.2, "K": 6144, "rows": BF16},
        # a step of serving through the norm
        {"name": "norm_decode", "op": "norm", "grad": False, "T": 16, "K": 6144, "residual": True},
        # a prompt through the norm
        {"name": "norm_prompt", "op": "norm", "grad": False, "T": 16384, "K": 6144, "residual": True},
        # the norm's gradient over an odd number of tokens
        {"name": "norm_grad", "op": "norm", "grad": True, "T": 8191, "K": 6144, "residual": True},
        # the layer's weights, laid out once after training
        {"name": "weights", "op": "weights", "E": 64, "K": 1024, "N": 2688},
        # one token's experts: eight rows on eight experts
        {"name": "product_single_token", "op": "product", "E": 8, "M": 8, "K": 1024, "N": 2688, "skew": -1.0, "out": BF16, "rows": FP8},
        # the decode shape: 32 experts x 16 rows, weight bytes only
        {"name": "product_decode", "op": "product", "E": 32, "M": 512, "K": 6144, "N": 4096, "skew": -1.0, "out": BF16, "rows": FP8},
        # a prompt's bf16 rows through the gate and up projections: quantised, multiplied, activated
        {"name": "product_swiglu_skew16k", "op": "product", "E": 64, "M": 16384, "K": 1024, "N": 2688, "skew": 1.2, "out": "swiglu", "rows": BF16},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(step, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step)

    op = rng.choice(["sort", "sort", "combine", "combine", "norm", "norm", "weights", "product", "product", "product"])
    case = {"op": op, "K": log(64, 6144, 16)}
    if op == "norm":
        return dict(case, grad=rng.random() < 0.5, T=log(1, 16384 if case["K"] < 4096 else 8192), residual=rng.random() < 0.7)
    if op in ("sort", "combine"):
        k = rng.choice([1, 2, 4, 6, 8])
        case.update(k=k, E=max(k, log(4, 256)), ranks=rng.choice([1, 1, 4]), skew=rng.choice([0.0, 0.6, 1.2]), T=log(1, 16384))
        while case["T"] * k * case["K"] > 8.0e7:
            case["T"] = (case["T"] + 1) // 2
        if op == "combine":
            return dict(case, grad=rng.random() < 0.5, rows=rng.choice([BF16, BF16, F32]))
        return dict(case, rows=rng.choice([BF16, FP8]))
    case.update(E=log(1, 128), N=log(64, 4096, 8))
    while case["E"] * case["K"] * case["N"] > 1.7e8:
        case["E"] = max(1, case["E"] // 2)
    if op == "weights":
        return case
    case.update(M=log(1, 16384), skew=rng.choice([-1.0, 0.0, 0.6, 1.2]))
    while case["M"] * case["K"] * case["N"] > 4.5e10:
        case["M"] //= 2
    return dict(case, out=rng.choice([BF16, "swiglu"]), rows=rng.choice([FP8, FP8, BF16]))


def _shares(case, seed):
    """Each expert's share of the choices: rank^-skew, ranks shuffled by the seed."""
    E = case["E"] * case.get("ranks", 1)
    rank = np.random.default_rng([seed, 17]).permutation(E) + 1
    p = rank.astype(np.float64) ** -max(0.0, case["skew"])
    return p / p.sum()


def _group_sizes(case, seed):
    """Rows of each expert: an even split (skew < 0), or every row drawn by the shares."""
    E, M = case["E"], case["M"]
    if case["skew"] < 0:
        return [M // E + (e < M % E) for e in range(E)]
    return np.random.default_rng([seed, 19]).multinomial(M, _shares(case, seed)).tolist()


def _choices(case, seed, gen):
    """k different experts a token, and their weights. Experts of other ranks get a
    number outside [0, E)."""
    noise = -torch.log(-torch.log(torch.rand(case["T"], case["E"] * case["ranks"], generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    score = noise + torch.tensor(np.log(_shares(case, seed)), dtype=torch.float32, device="cuda")
    top, experts = score.topk(case["k"], dim=1)
    return experts.int(), torch.softmax(top, dim=1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, K = case["op"], case["K"]
    s = dict(case)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()

    def activations(rows, cols):
        # a few columns run several times hotter than the rest
        heat = torch.exp(0.8 * torch.randn(cols, generator=gen, device="cuda"))
        return (torch.randn(rows, cols, generator=gen, device="cuda") * heat).bfloat16()

    if op == "norm":
        s["X"] = activations(case["T"], K)
        s["g"] = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).bfloat16()
        s["res"] = activations(case["T"], K) if case["residual"] else None  # the residual, or its gradient
        s["dY"] = normal(case["T"], K, scale=0.02) if case["grad"] else None
        return s
    if op in ("sort", "combine"):
        s["experts"], s["w"] = _choices(case, seed, gen)
        rows = case["T"] * case["k"]
        if op == "sort":
            s["X"], s["scale"] = activations(case["T"], K), None
            if case["rows"] == FP8:
                s["X"], s["scale"] = _fp8_rows(s["X"].float())
            # rows of other ranks' experts leave the last rows of these as they are
            s["out"] = torch.zeros(rows, K, dtype=torch.uint8 if case["rows"] == FP8 else torch.bfloat16, device="cuda")
            s["out"] = s["out"].view(F8) if case["rows"] == FP8 else s["out"]
            s["out_scale"] = torch.zeros(-(-K // 128), rows, device="cuda") if case["rows"] == FP8 else None
            return s
        s["pos"] = _order(s["experts"], case["E"])[2]
        s["Y"] = normal(rows, K) if case["rows"] == BF16 else torch.randn(rows, K, generator=gen, device="cuda")
        if case["grad"]:
            s["dO"] = normal(case["T"], K, scale=0.02).to(s["Y"].dtype)
            s["out"] = torch.zeros_like(s["Y"])
        return s
    E, N = case["E"], case["N"]
    if op == "weights":
        return dict(s, B=normal(E, K, N, scale=1 / math.sqrt(K)))
    s["sizes"] = _group_sizes(case, seed)
    s["offsets"] = torch.tensor(np.cumsum([0] + s["sizes"]), dtype=torch.int32, device="cuda")
    s["X"], s["scale"] = activations(case["M"], K), None
    if case["rows"] == FP8:
        s["X"], s["scale"] = _fp8_rows(s["X"].float())
    w = [_fp8_tiles(normal(N, K, scale=1 / math.sqrt(K)).float()) for _ in range(E)]
    s["Bq"], s["b_scale"] = torch.stack([q.view(torch.uint8) for q, _ in w]).view(F8), torch.stack([c for _, c in w])
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import moe_ragged_grouped_amd as gg

    op = s["op"]
    if op == "sort":
        offsets, rows, pos, w = gg.expert_sort(s["experts"], s["E"], weights=s["w"])
        if s["rows"] == FP8:
            return offsets, rows, pos, w, gg.expert_spread(s["X"], pos, scale=s["scale"], out=s["out"], out_scale=s["out_scale"])
        return offsets, rows, pos, w, gg.expert_spread(s["X"], pos, out=s["out"])
    if op == "combine":
        if s["grad"]:
            return gg.expert_combine_grad(s["dO"], s["Y"], s["pos"], s["w"], out=s["out"])
        return gg.expert_combine(s["Y"], s["pos"], s["w"])
    if op == "norm":
        if s["grad"]:
            return gg.rms_norm_grad(s["dY"], s["X"], s["g"], d_residual=s["res"], eps=EPS)
        return gg.rms_norm_fp8(s["X"], s["g"], residual=s["res"], eps=EPS)
    if op == "weights":
        return gg.fp8_quantize_weights(s["B"])
    X, scale = gg.fp8_quantize(s["X"]) if s["rows"] == BF16 else (s["X"], s["scale"])
    if s["out"] == "swiglu":
        return gg.grouped_gemm_fp8_block_swiglu(X, scale, s["Bq"], s["b_scale"], s["offsets"])
    return gg.grouped_gemm_fp8_block(X, scale, s["Bq"], s["b_scale"], s["offsets"], out_dtype=torch.bfloat16)


def _run_plain(s):
    op = s["op"]
    if op == "sort":
        offsets, order, pos = _order(s["experts"], s["E"])
        inside = torch.arange(order.numel(), device="cuda") < offsets[-1]
        rows = torch.where(inside, order // s["k"], -1)
        w = torch.where(inside, s["w"].flatten()[order], 0.0)
        from_row = rows.clamp(min=0)
        if s["rows"] == FP8:  # bytes are moved as bytes
            q = torch.where(inside[:, None], s["X"].view(torch.uint8)[from_row], s["out"].view(torch.uint8)).view(F8)
            return offsets, rows.int(), pos, w, (q, torch.where(inside, s["scale"][:, from_row], s["out_scale"]))
        return offsets, rows.int(), pos, w, torch.where(inside[:, None], s["X"][from_row], s["out"])
    if op == "combine":
        here = (s["pos"] >= 0)[..., None]
        at = s["pos"].clamp(min=0).long()
        if not s["grad"]:
            return torch.where(here, s["w"][..., None] * s["Y"].float()[at], 0.0).sum(1).to(s["Y"].dtype)
        dO = s["dO"].float()
        dw = torch.where(here, dO[:, None] * s["Y"].float()[at], 0.0).sum(2)
        dY = (s["w"][..., None] * dO[:, None]).to(s["Y"].dtype).flatten(0, 1)
        # every row of a present choice has one; the others go to a row that is cut off
        out = torch.cat([s["out"], s["out"][:1]])
        out[torch.where(here, at[..., None], s["out"].shape[0]).flatten()] = dY
        return out[:-1], dw
    if op == "norm":
        x = s["X"].float()
        if s["grad"]:
            dy, g = s["dY"].float(), s["g"].float()
            r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
            dx = r * (g * dy - x * r * r * (g * dy * x).mean(1, keepdim=True))
            if s["res"] is not None:
                dx = dx + s["res"].float()
            return dx.bfloat16(), (dy * x * r).sum(0)
        if s["res"] is not None:
            x = (x + s["res"].float()).bfloat16().float()
        q, scale = _fp8_rows(x * (1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)) * s["g"].float())
        return (q, scale) if s["res"] is None else (q, scale, x.bfloat16())
    if op == "weights":
        q, scale = zip(*[_fp8_tiles(b.t().float()) for b in s["B"]])
        return torch.stack([x.view(torch.uint8) for x in q]).view(F8), torch.stack(scale)
    X, scale = _fp8_rows(s["X"].float()) if s["rows"] == BF16 else (s["X"], s["scale"])
    rows = (X.float() * scale.t().repeat_interleave(128, 1)[:, :X.shape[1]]).split(s["sizes"])
    C = torch.cat([a @ _tile_values(q, c).t() for a, q, c in zip(rows, s["Bq"], s["b_scale"])])
    if s["out"] != "swiglu":
        return C.bfloat16()
    gate, up = C[:, 0::2], C[:, 1::2]
    return (gate / (1 + torch.exp(-gate)) * up).bfloat16()


def _order(experts, E):
    """Choices [T, k] -> the groups' offsets [E + 1], the choice of each row (choices
    outside [0, E) last), and the row of each choice, -1 outside. Rows of a group lie in
    the order of their choices."""
    flat = experts.flatten()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    by_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by_key, torch.arange(E + 1, dtype=by_key.dtype, device="cuda"))
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    return offsets.int(), order, torch.where(key < E, pos, -1).int().view(experts.shape)


def _codes(x, top):
    """fp32 blocks (last dimension) and their largest magnitudes -> E4M3, scales."""
    m = ((TOP / top.clamp(min=LEAST)).view(torch.int32) & -256).view(torch.float32)
    return (x * m[..., None]).clamp(-TOP, TOP).to(F8), 1 / m


def _fp8_rows(x):
    """fp32 [M, K] -> E4M3 [M, K], scales [ceil(K/128), M]."""
    M, K = x.shape
    b = torch.nn.functional.pad(x, (0, -K % 128)).unflatten(1, (-1, 128))
    q, scale = _codes(b, b.abs().amax(2))
    return q.flatten(1).view(torch.uint8)[:, :K].contiguous().view(F8), scale.t().contiguous()


def _fp8_tiles(x):
    """fp32 [N, K] -> E4M3 [N, K], scales [ceil(N/128), ceil(K/128)]."""
    N, K = x.shape
    b = torch.nn.functional.pad(x, (0, -K % 128, 0, -N % 128)).unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
    q, scale = _codes(b, b.abs().amax((1, 3))[:, None].expand(-1, 128, -1))
    return q.flatten(2).flatten(0, 1).view(torch.uint8)[:N, :K].contiguous().view(F8), scale[:, 0].contiguous()


def _tile_values(q, scale):
    return q.float() * scale.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def work(case):
    op, K = case["op"], case["K"]
    q = 1 + 4 / 128  # a value in 8 bits with its share of the scale
    if op == "norm":
        n = case["T"] * K
        if case["grad"]:  # dY, X and the residual's gradient in, dX out
            return {"bytes": n * (6 + 2 * case["residual"]) + K * 6, "flops": 12 * n}
        return {"bytes": n * (2 + q + 4 * case["residual"]) + K * 2, "flops": 8 * n}
    if op in ("sort", "combine"):
        T, k = case["T"], case["k"]
        rows = T * k / case["ranks"]  # about that many have a row here
        index = T * k * 4
        if op == "sort":  # choices and weights in; tokens, places and weights out; each token's row in, k out
            b = {BF16: 2, FP8: q}[case["rows"]]
            return {"bytes": 5 * index + (case["E"] + 1) * 4 + (min(T, rows) + rows) * K * b, "flops": 0}
        b = 2 if case["rows"] == BF16 else 4
        if case["grad"]:  # dO and the rows in, their gradient and the weights' out
            return {"bytes": 3 * index + (T + 2 * rows) * K * b, "flops": 3 * rows * K}
        return {"bytes": 2 * index + (T + rows) * K * b, "flops": 2 * rows * K}
    E, N = case["E"], case["N"]
    if op == "weights":
        return {"bytes": E * K * N * 3, "flops": 0}
    M = case["M"]
    # experts that get a row, whose weights have to be read
    busy = min(E, M) if case["skew"] < 0 else float(np.sum(1 - (1 - _shares(case, 0)) ** M))
    rows = M * K * (2 if case["rows"] == BF16 else q)
    return {"bytes": rows + busy * K * N + M * N * (1 if case["out"] == "swiglu" else 2), "flops": 2 * M * K * N}


def exact(case, seed):
    """What run() returns for these inputs, in 64 bits, straight from the definitions."""
    s = prepare(case, seed)
    op, K = case["op"], case["K"]
    if op == "sort":
        e = s["experts"].cpu().numpy().ravel()
        E, k = case["E"], case["k"]
        picks = [np.flatnonzero(e == i) for i in range(E)]
        offsets = np.concatenate([[0], np.cumsum([len(p) for p in picks])])
        order = np.concatenate(picks).astype(np.int64)
        n = len(order)
        rows, pos = np.full(e.size, -1), np.full(e.size, -1)
        rows[:n], pos[order] = order // k, np.arange(n)
        w = np.zeros(e.size)
        w[:n] = s["w"].double().cpu().numpy().ravel()[order]
        token = torch.from_numpy(order // k).cuda()
        out = torch.zeros(e.size, K, dtype=torch.float64, device="cuda")
        out[:n] = s["X"].double()[token]
        if case["rows"] == FP8:
            scale = torch.zeros(-(-K // 128), e.size, dtype=torch.float64, device="cuda")
            scale[:, :n] = s["scale"].double()[:, token]
            out = (out, scale)
        return offsets.astype(np.int32), rows.astype(np.int32), pos.astype(np.int32).reshape(-1, k), w, out
    if op == "combine":
        w, pos = s["w"].double(), s["pos"].long()
        total = torch.zeros(case["T"], K, dtype=torch.float64, device="cuda")
        dY, dw = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda"), torch.zeros_like(w)
        for j in range(case["k"]):
            t = torch.nonzero(pos[:, j] >= 0).flatten()
            y = s["Y"][pos[t, j]].double()
            if case["grad"]:
                d = s["dO"][t].double()
                dw[t, j] = torch.linalg.vecdot(d, y)
                dY[pos[t, j]] = d * w[t, j, None]
            else:
                total[t] += y * w[t, j, None]
        return (dY, dw) if case["grad"] else total
    if op == "norm":
        parts = [_exact_norm(s, slice(a, a + 2048)) for a in range(0, case["T"], 2048)]
        if case["grad"]:
            return torch.cat([p[0] for p in parts]), sum(p[1] for p in parts)
        whole = [torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]).t()]
        return whole + ([torch.cat([p[2] for p in parts])] if case["residual"] else [])
    if op == "weights":
        q, scale = zip(*[_exact_codes(b.double().t(), 128) for b in s["B"]])
        return torch.stack(q), torch.stack(scale)
    if case["rows"] == BF16:
        X, scale = _exact_codes(s["X"].double(), 1)
    else:
        X, scale = s["X"].double(), s["scale"].double().t()
    block = torch.arange(K, device="cuda") // 128
    column = torch.arange(case["N"], device="cuda") // 128
    X = X * scale[:, block]
    C = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
    ends = np.cumsum(s["sizes"])
    for e, (m, end) in enumerate(zip(s["sizes"], ends)):
        B = s["Bq"][e].double() * s["b_scale"][e].double()[column][:, block]
        C[int(end) - m:int(end)] = X[int(end) - m:int(end)] @ B.t()
    return C if case["out"] != "swiglu" else C[:, 0::2] * torch.sigmoid(C[:, 0::2]) * C[:, 1::2]


def _exact_norm(s, rows):
    x, g = s["X"][rows].double(), s["g"].double()
    n = x.shape[1]
    res = None if s["res"] is None else s["res"][rows].double()
    if s["grad"]:
        dy = s["dY"][rows].double()
        ms = torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / n + EPS
        unit = x * ms ** -0.5
        gy = dy * g
        dx = (gy - unit * (gy * unit).sum(1, keepdim=True) / n) * ms ** -0.5
        return dx if res is None else dx + res, (dy * unit).sum(0)
    if res is not None:  # the sum is what the next layer sees: bf16
        x = (x + res).float().bfloat16().double()
    ms = torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / n + EPS
    q, scale = _exact_codes(x * g * ms ** -0.5, 1)
    return q, scale, x


def _exact_codes(x, height):
    """x [rows, K] -> the E4M3 values nearest to x times its block's multiplier, ties to even,
    and the scales [ceil(rows / height), ceil(K / 128)] of blocks height x 128."""
    rows, K = x.shape
    block = torch.arange(K, device=x.device) // 128
    band = torch.arange(rows, device=x.device) // height
    top = torch.stack([x[:, a:a + 128].abs().amax(1) for a in range(0, K, 128)], 1)
    if height > 1:
        top = torch.stack([top[a:a + height].amax(0) for a in range(0, rows, height)])
    f, e = torch.frexp(TOP / top.clamp(min=LEAST))
    m = torch.ldexp(torch.floor(f * 65536), e - 16)
    y = x * m[band][:, block]
    # a value in [2^e, 2^(e+1)) is a multiple of 2^(e-3); below 2^-6 of 2^-9
    step = torch.exp2(torch.frexp(y)[1].clamp(min=-5).double() - 4)
    return torch.round(y / step).clamp(-TOP / step, TOP / step) * step, 1 / m
