"""Cases for a linear layer's operators: the product with its bias, activation and residual, its gradients, and the
orthogonalised update of its weights.

Each case names one operator (`op`) and its sizes.  `prepare` makes the inputs and the output buffers, `run` makes one
pass: with `own` false in plain torch operations in 32 bits, with `own` true through the library's entry points.
`exact` is the same result from the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7  # the quintic iteration, as Muon runs it


def listed():
    return [
        # serving: one token through a gated or plain up-projection
        {"name": "linear-one-token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "act": "silu", "bias": "f32",
         "residual": False, "preact": False, "out": "bf16"},
        # serving: a batch of 24 decoded tokens, down-projection added to the residual stream
        {"name": "linear-decode-batch", "op": "linear", "M": 24, "N": 2048, "K": 8192, "act": "none", "bias": "none",
         "residual": True, "preact": False, "out": "bf16"},
        # serving: a short ragged prompt, all sizes odd, logits kept in 32 bits
        {"name": "linear-odd-f32", "op": "linear", "M": 257, "N": 1023, "K": 777, "act": "relu", "bias": "bf16",
         "residual": True, "preact": False, "out": "f32"},
        # training: a ragged batch through the up-projection, pre-activations kept for the backward pass
        {"name": "linear-train-up", "op": "linear", "M": 2047, "N": 4096, "K": 6144, "act": "gelu_tanh",
         "bias": "bf16", "residual": False, "preact": True, "out": "bf16"},
        # training: a large batch through the down-projection, added to the residual stream
        {"name": "linear-train-down", "op": "linear", "M": 8192, "N": 4096, "K": 8192, "act": "none", "bias": "bf16",
         "residual": True, "preact": False, "out": "bf16"},
        # training: backward of a small ragged layer, chained to the activation before it
        {"name": "grad-odd-chained", "op": "grad", "M": 1021, "N": 1000, "K": 513, "act": "gelu", "before": "relu",
         "bias": True, "base": False, "grad_w": "bf16"},
        # training: backward of a projection without activation, weight gradients accumulated in 32 bits
        {"name": "grad-accumulate", "op": "grad", "M": 4096, "N": 2048, "K": 2048, "act": "none", "before": "none",
         "bias": True, "base": True, "grad_w": "f32"},
        # training: backward of the large up-projection
        {"name": "grad-train-up", "op": "grad", "M": 8192, "N": 8192, "K": 4096, "act": "silu", "before": "none",
         "bias": True, "base": False, "grad_w": "bf16"},
        # optimiser: the update of one small projection
        {"name": "orth-small", "op": "orth", "count": 1, "R": 512, "C": 768, "g": "bf16"},
        # optimiser: odd sizes, more rows than columns, updates held in 32 bits
        {"name": "orth-tall-odd", "op": "orth", "count": 1, "R": 2300, "C": 1001, "g": "f32"},
        # optimiser: the updates of a mixture-of-experts layer's matrices, one for each expert
        {"name": "orth-experts", "op": "orth", "count": 8, "R": 4096, "C": 2048, "g": "bf16"},
        # optimiser: one large square matrix
        {"name": "orth-large", "op": "orth", "count": 1, "R": 4096, "C": 4096, "g": "bf16"},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi], now and then a multiple of 64."""
    n = round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))
    if rng.random() < 0.4:
        n = n // 64 * 64
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(["linear", "linear", "grad", "orth"])
    while True:
        if op == "linear":
            case = {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 64, 8192), "K": _size(rng, 64, 8192),
                    "act": rng.choice(ACTS), "bias": rng.choice(["none", "bf16", "f32"]),
                    "residual": rng.random() < 0.5, "preact": rng.random() < 0.3, "out": rng.choice(["bf16", "f32"])}
            most = "linear-train-down"
        elif op == "grad":
            act = rng.choice(ACTS)
            case = {"op": op, "M": _size(rng, 16, 8192), "N": _size(rng, 64, 8192), "K": _size(rng, 64, 8192),
                    "act": act, "before": rng.choice(["none", "none", *ACTS[1:]]), "bias": rng.random() < 0.5,
                    "base": rng.random() < 0.5, "grad_w": rng.choice(["bf16", "f32"]) if act == "none" else "bf16"}
            most = "grad-train-up"
        else:
            case = {"op": op, "count": rng.choice([1, 1, 1, 2, 5]), "R": _size(rng, 64, 4096), "C": _size(rng, 64, 4096),
                    "g": rng.choice(["bf16", "f32"])}
            most = "orth-experts"
        if work(case)["flops"] <= work(next(c for c in listed() if c["name"] == most))["flops"]:
            return case


# ---------------------------------------------------------------- inputs
def _rows(r, c, dtype, lead=()):
    """An empty [r, c] matrix whose rows start 16-byte aligned, as the products' operands need."""
    step = max(1, 16 // torch.empty(0, dtype=dtype).element_size())
    return torch.empty((*lead, r, -(-c // step) * step), dtype=dtype, device="cuda")[..., :c]


def _normal(r, c, dtype, g, scale=1.0):
    t = _rows(r, c, dtype)
    t.copy_(scale * torch.randn((r, c), device="cuda", generator=g))
    return t


def _activations(r, c, dtype, g):
    """Normal values with a few strong channels and rows of unequal size, as activations have."""
    x = torch.randn((r, c), device="cuda", generator=g)
    x *= torch.exp(0.7 * torch.randn((1, c), device="cuda", generator=g))
    x *= torch.exp(0.5 * torch.randn((r, 1), device="cuda", generator=g))
    t = _rows(r, c, dtype)
    t.copy_(x)
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        out = TYPES[case["out"]]
        st["x"] = _activations(M, K, torch.bfloat16, g)
        st["w"] = _normal(N, K, torch.bfloat16, g, 1 / math.sqrt(K))
        st["bias"] = None if case["bias"] == "none" else \
            (0.5 * torch.randn(N, device="cuda", generator=g)).to(TYPES[case["bias"]])
        st["residual"] = _normal(M, N, out, g, 2.0) if case["residual"] else None
        st["y"] = _rows(M, N, out)
        st["preact"] = _rows(M, N, out) if case["preact"] else None
    elif op == "grad":
        M, N, K = case["M"], case["N"], case["K"]
        bf16 = torch.bfloat16
        st["grad_y"] = _normal(M, N, bf16, g, 0.01)
        st["preact"] = _normal(M, N, bf16, g, 1.5) if case["act"] != "none" else None
        st["x"] = _activations(M, K, bf16, g)
        st["w"] = _normal(N, K, bf16, g, 1 / math.sqrt(K))
        st["before"] = _normal(M, K, bf16, g, 1.5) if case["before"] != "none" else None
        st["base"] = _normal(N, K, TYPES[case["grad_w"]], g) if case["base"] else None
        st["grad_z"] = _rows(M, N, bf16) if case["act"] != "none" else None
        st["grad_x"] = _rows(M, K, bf16)
        st["grad_w"] = _rows(N, K, TYPES[case["grad_w"]])
        st["grad_bias"] = torch.empty(N, dtype=torch.float32, device="cuda") if case["bias"] else None
    else:
        n, R, C = case["count"], case["R"], case["C"]
        lead = (n,) if n > 1 else ()
        st["g"] = _rows(R, C, TYPES[case["g"]], lead)
        # an averaged gradient: noise and a part of low rank that dominates it, of any magnitude
        u = torch.randn((*lead, R, 8), device="cuda", generator=g)
        v = torch.randn((*lead, 8, C), device="cuda", generator=g)
        size = 10.0 ** (4 * torch.rand((*lead, 1, 1), device="cuda", generator=g) - 5)
        st["g"].copy_(size * (torch.randn((*lead, R, C), device="cuda", generator=g) + 0.3 * torch.matmul(u, v)))
        st["out"] = _rows(R, C, torch.bfloat16, lead)
    return st


# ---------------------------------------------------------------- plain forms, 32 bits
def _sigmoid(z):
    return torch.reciprocal(1.0 + torch.exp(-z))


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z * _sigmoid(z)
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    s = _sigmoid(z)
    return s * (1.0 + z * (1.0 - s))


def _orthogonalise(x):
    a, b, c = COEFFICIENTS
    x = x / (torch.sqrt((x * x).sum((-2, -1), keepdim=True)) + EPS)
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-2, -1) if tall else x
    for _ in range(STEPS):
        A = torch.matmul(x, x.transpose(-2, -1))
        x = a * x + torch.matmul(b * A + c * torch.matmul(A, A), x)
    return x.transpose(-2, -1) if tall else x


def _plain(st):
    case = st["case"]
    if case["op"] == "linear":
        z = torch.matmul(st["x"].float(), st["w"].float().t())
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        out = {"y": y.to(st["y"].dtype)}
        if st["preact"] is not None:
            out["preact"] = z.to(st["y"].dtype)
        return out
    if case["op"] == "grad":
        gz = st["grad_y"].float()
        if case["act"] != "none":
            gz = gz * _act_slope(st["preact"].float(), case["act"])
        gx = torch.matmul(gz, st["w"].float())
        if case["before"] != "none":
            gx = gx * _act_slope(st["before"].float(), case["before"])
        gw = torch.matmul(gz.t(), st["x"].float())
        if st["base"] is not None:
            gw = gw + st["base"].float()
        out = {"grad_x": gx.to(torch.bfloat16), "grad_w": gw.to(st["grad_w"].dtype)}
        if case["bias"]:
            out["grad_bias"] = gz.sum(0)
        return out
    return {"out": _orthogonalise(st["g"].float()).to(torch.bfloat16)}


# ---------------------------------------------------------------- the library's operators
def _library(st):
    import tile_scheduling_gb300 as ts

    case = st["case"]
    if case["op"] == "linear":
        ts.ts_linear(st["x"], st["w"], st["y"], bias=st["bias"], act=case["act"], residual=st["residual"],
                     preact=st["preact"])
        return {n: st[n] for n in ("y", "preact") if st[n] is not None}
    if case["op"] == "grad":
        gz = st["grad_y"]
        if case["act"] != "none":
            ts.ts_act_grad(gz, st["preact"], st["grad_z"], grad_bias=st["grad_bias"], act=case["act"])
            gz = st["grad_z"]
        elif case["bias"]:
            ts.ts_act_grad(gz, None, None, grad_bias=st["grad_bias"])
        ts.ts_linear_grad_input(gz, st["w"], st["grad_x"], act=case["before"], preact=st["before"])
        ts.ts_linear_grad_weight(gz, st["x"], st["grad_w"], base=st["base"])
        return {n: st[n] for n in ("grad_x", "grad_w", "grad_bias") if st[n] is not None}
    ts.ts_orthogonalise(st["g"], st["out"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    return {"out": st["out"]}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- what one pass cannot do without
def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["out"] == "f32" else 2
        n = 2 * (M * K + N * K) + {"none": 0, "bf16": 2, "f32": 4}[case["bias"]] * N
        return {"bytes": n + M * N * size * (1 + case["residual"] + case["preact"]), "flops": 2 * M * N * K}
    if case["op"] == "grad":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["grad_w"] == "f32" else 2
        n = 2 * M * N * (1 + (case["act"] != "none")) + 2 * M * K * (2 + (case["before"] != "none")) + 2 * N * K
        return {"bytes": n + N * K * size * (1 + case["base"]) + (4 * N if case["bias"] else 0), "flops": 4 * M * N * K}
    R, C, n = case["R"], case["C"], case["count"]
    lo, hi = min(R, C), max(R, C)
    # of the two symmetric products of a step only half the entries have to be formed
    flops = n * STEPS * (lo * lo * hi + lo ** 3 + 2 * lo * lo * hi)
    return {"bytes": n * R * C * ((4 if case["g"] == "f32" else 2) + 2), "flops": flops}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    F = torch.nn.functional
    acts = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}
    if case["op"] == "linear":
        z = torch.einsum("mk,nk->mn", st["x"].to(d), st["w"].to(d))
        z += 0 if st["bias"] is None else st["bias"].to(d)
        y = acts[case["act"]](z)
        out = {"y": y if st["residual"] is None else st["residual"].to(d) + y}
        if case["preact"]:
            out["preact"] = z
        return out
    if case["op"] == "grad":
        def back(z, act, grad):
            if act == "none":
                return grad
            z = z.to(d).requires_grad_()
            acts[act](z).backward(grad)
            return z.grad

        gz = back(st["preact"], case["act"], st["grad_y"].to(d))
        gw = torch.einsum("mn,mk->nk", gz, st["x"].to(d))
        out = {"grad_x": back(st["before"], case["before"], torch.einsum("mn,nk->mk", gz, st["w"].to(d))),
               "grad_w": gw if st["base"] is None else st["base"].to(d) + gw}
        if case["bias"]:
            out["grad_bias"] = torch.einsum("mn->n", gz)
        return out
    # p(s) = a s + b s^3 + c s^5 on the singular values, step by step
    x = st["g"].to(d)
    x = x / (torch.linalg.matrix_norm(x)[..., None, None] + EPS)
    wide = x.shape[-1] >= x.shape[-2]
    for _ in range(STEPS):
        s2 = torch.einsum("...ik,...jk->...ij" if wide else "...ki,...kj->...ij", x, x)
        p = COEFFICIENTS[1] * s2 + COEFFICIENTS[2] * torch.einsum("...ij,...jk->...ik", s2, s2)
        p.diagonal(dim1=-2, dim2=-1).add_(COEFFICIENTS[0])
        x = torch.einsum("...ij,...jk->...ik" if wide else "...kj,...ij->...ki", *((p, x) if wide else (x, p)))
    return {"out": x}
