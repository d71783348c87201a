"""Cases for the mixture-of-experts operators: routing, 8-bit quantisation, block-scaled 8-bit products and the combine.

Each case names one operator (`op`) and its sizes.  `prepare` makes the inputs and the output buffers, `run` makes one
pass: with `own` false in plain torch operations in 32 bits, with `own` true through the library's entry points.
`exact` is the same result from the definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128              # elements that share a scale
E4M3_MAX, E5M2_MAX = 448.0, 57344.0
AMAX_MIN = 2.0 ** -100   # a block's largest magnitude is taken as at least this
FORMATS = {"e4m3": (torch.float8_e4m3fn, E4M3_MAX), "e5m2": (torch.float8_e5m2, E5M2_MAX)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # serving: the router of one token, sigmoid scores, a bias for balance, 4 of 8 expert groups kept
        {"name": "route-one-token", "op": "route", "tokens": 1, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "keep": 4, "best": 2, "renorm": True, "logits": "f32", "train": False},
        # training: a ragged batch with padding tokens (whole rows masked), softmax scores, and the gradient
        {"name": "route-batch-train", "op": "route", "tokens": 8191, "experts": 128, "top_k": 6, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "best": 1, "renorm": True, "logits": "bf16", "train": True},
        # serving: 32 tokens, each sent to 8 experts, quantised on the way
        {"name": "quant-gather-decode", "op": "quant", "rows": 256, "cols": 4096, "gather": 8, "transpose": False,
         "x": "bf16", "format": "e4m3"},
        # training: activations quantised down the token axis for the weight gradient
        {"name": "quant-transposed-train", "op": "quant", "rows": 8192, "cols": 8192, "gather": 0, "transpose": True,
         "x": "bf16", "format": "e4m3"},
        # serving: one token through one layer; the weights' bytes are the work
        {"name": "gemm-one-token", "op": "gemm", "M": 1, "N": 4096, "K": 8192, "b_scale": "block", "trans_b": False,
         "a": "e4m3", "out": "bf16"},
        # training: input gradient of a ragged batch, weights read in place, gradients in e5m2
        {"name": "gemm-input-gradient", "op": "gemm", "M": 2047, "N": 4096, "K": 6144, "b_scale": "block",
         "trans_b": True, "a": "e5m2", "out": "bf16"},
        # training: weight gradient, scales along the tokens on both sides, fp32 out
        {"name": "gemm-weight-gradient", "op": "gemm", "M": 4096, "N": 4096, "K": 8191, "b_scale": "row",
         "trans_b": False, "a": "e4m3", "out": "f32"},
        # training or prefill: the largest dense product
        {"name": "gemm-large", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "b_scale": "block", "trans_b": False,
         "a": "e4m3", "out": "bf16"},
        # serving: 32 tokens x 8 experts spread over 64 experts; every expert's weights are read for a few rows
        {"name": "experts-decode", "op": "experts", "rows": 256, "experts": 64, "N": 2048, "K": 2048,
         "trans_b": False, "skew": 0.5, "out": "bf16"},
        # training or prefill: 16384 rows over 32 experts of unequal load
        {"name": "experts-batch", "op": "experts", "rows": 16384, "experts": 32, "N": 4096, "K": 2048,
         "trans_b": False, "skew": 0.5, "out": "bf16"},
        # serving: 32 tokens take their experts' rows back
        {"name": "combine-decode", "op": "combine", "tokens": 32, "top_k": 8, "N": 4096, "drop": 0.0, "train": False},
        # training: combine and its gradient, a few slots dropped
        {"name": "combine-train", "op": "combine", "tokens": 8192, "top_k": 4, "N": 4096, "drop": 0.02, "train": True},
    ]


def _size(rng, low, high):
    """Log-uniform in [low, high]; half of the draws are made odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(low, min(high, v | 1 if rng.random() < 0.5 else v))


def draw(rng):
    op = rng.choice(["route", "quant", "gemm", "gemm", "experts", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _size(rng, 8, 512 // groups)
        keep = rng.randint(max(1, groups // 4), groups)
        top_k = min(rng.randint(1, 8), keep * (experts // groups))
        return {"op": op, "tokens": _size(rng, 1, 8192), "experts": experts, "top_k": top_k,
                "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.5, "groups": groups,
                "keep": keep, "best": rng.choice([1, 2]),
                # a single weight that is renormalised is 1, its gradient 0: nothing to compute
                "renorm": top_k > 1 and rng.random() < 0.7, "logits": rng.choice(["f32", "bf16"]), "train": rng.random() < 0.5}
    if op == "quant":
        transpose = rng.random() < 0.4
        return {"op": op, "rows": _size(rng, 1, 8192), "cols": _size(rng, 64, 8192),
                "gather": 0 if transpose else rng.choice([0, 1, 4, 8]), "transpose": transpose,
                "x": rng.choice(["bf16", "f32"]), "format": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "gemm":
        b_scale = rng.choice(["block", "block", "row"])
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 64, 8192), "K": _size(rng, 64, 8192),
                "b_scale": b_scale, "trans_b": b_scale == "block" and rng.random() < 0.4,
                "a": rng.choice(["e4m3", "e4m3", "e5m2"]), "out": rng.choice(["bf16", "f32"])}
    if op == "experts":
        return {"op": op, "rows": _size(rng, 1, 16384), "experts": _size(rng, 2, 64), "N": _size(rng, 64, 4096),
                "K": _size(rng, 64, 2048), "trans_b": rng.random() < 0.3, "skew": rng.choice([0.0, 0.5, 1.0]),
                "out": rng.choice(["bf16", "f32"])}
    return {"op": op, "tokens": _size(rng, 1, 8192), "top_k": rng.randint(1, 8), "N": _size(rng, 64, 4096),
            "drop": rng.choice([0.0, 0.02, 0.3]), "train": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _blocks(n):
    return -(-n // BLOCK)


def _rows(r, c, dtype):
    """An empty [r, c] matrix whose rows start 16-byte aligned, as the products' operands need."""
    step = max(1, 16 // torch.empty(0, dtype=dtype).element_size())
    return torch.empty((r, -(-c // step) * step), dtype=dtype, device="cuda")[:, :c]


def _scales(r, blocks):
    """Scales [r, blocks], stored with the rows contiguous."""
    return torch.empty((blocks, r), dtype=torch.float32, device="cuda").t()


def _quantised_rows(x, fmt="e4m3"):
    """x [r, c] float32 as 8-bit values and one scale for each row and 128 columns."""
    dtype, top = FORMATS[fmt]
    r, c = x.shape
    nb = _blocks(c)
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - c)).view(r, nb, BLOCK)
    amax = v.abs().amax(2).clamp_min(AMAX_MIN)
    q = _rows(r, c, dtype)
    q.copy_((v * (top / amax)[:, :, None]).clamp_(-top, top).view(r, -1)[:, :c].to(dtype))
    s = _scales(r, nb)
    s.copy_(amax / top)
    return q, s


def _quantised_blocks(x):
    """x [..., r, c] float32 as e4m3 and one scale for each 128 x 128 block."""
    r, c = x.shape[-2:]
    lead = x.shape[:-2]
    rb, cb = _blocks(r), _blocks(c)
    v = torch.nn.functional.pad(x, (0, cb * BLOCK - c, 0, rb * BLOCK - r)).view(*lead, rb, BLOCK, cb, BLOCK)
    amax = v.abs().amax((-3, -1)).clamp_min(AMAX_MIN)
    q = (v * (E4M3_MAX / amax)[..., :, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX)
    q = q.view(*lead, rb * BLOCK, cb * BLOCK)[..., :r, :c].to(torch.float8_e4m3fn)
    keep = torch.empty((*lead, r, -(-c // 16) * 16), dtype=torch.float8_e4m3fn, device="cuda")[..., :c]
    keep.copy_(q)
    return keep, (amax / E4M3_MAX).contiguous()


def _activations(r, c, g):
    """Normal values with a few strong channels and rows of unequal size, as activations and gradients have."""
    x = torch.randn((r, c), device="cuda", generator=g)
    x *= torch.exp(0.7 * torch.randn((1, c), device="cuda", generator=g))
    x *= torch.exp(0.5 * torch.randn((r, 1), device="cuda", generator=g))
    return x


def _loads(rows, experts, skew, g):
    """Offsets [experts + 1] of `rows` rows dealt to experts of unequal popularity."""
    pop = torch.softmax(skew * torch.randn(experts, device="cuda", generator=g), 0)
    pick = torch.multinomial(pop, rows, replacement=True, generator=g)
    off = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    off[1:] = torch.bincount(pick, minlength=experts).cumsum(0)
    return off


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        x = 1.5 * torch.randn((T, E), device="cuda", generator=g)
        if case["train"]:  # padding tokens: every expert masked; and now and then an expert out of service
            pad = torch.rand((T, 1), device="cuda", generator=g) < 0.02
            x = x.masked_fill(pad | (torch.rand((T, E), device="cuda", generator=g) < 0.01), -math.inf)
        st["logits"] = x.to(TYPES[case["logits"]])
        # the balancing bias moves in steps of 0.001
        st["bias"] = 0.001 * torch.round(30 * torch.randn(E, device="cuda", generator=g)) if case["bias"] else None
        st["grad_weights"] = torch.randn((T, k), device="cuda", generator=g)
        st["experts"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        st["offsets"] = torch.empty(E + 1, dtype=torch.int64, device="cuda")
        st["order"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        st["position"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["grad_logits"] = torch.empty_like(st["logits"])
    elif op == "quant":
        R, C, k = case["rows"], case["cols"], case["gather"]
        src = max(1, R // k) if k else R
        st["x"] = _rows(src, C, TYPES[case["x"]])
        st["x"].copy_(_activations(src, C, g))
        # rows of the sorted layout: slots in expert order, slot // k is the token
        st["index"] = torch.randperm(src * k, device="cuda", generator=g)[:R].to(torch.int32) if k else None
        if k and R > src * k:
            st["index"] = torch.randint(0, src * k, (R,), device="cuda", generator=g).to(torch.int32)
        dtype = FORMATS[case["format"]][0]
        qr, qc = (C, R) if case["transpose"] else (R, C)
        st["q"] = _rows(qr, qc, dtype)
        st["scales"] = _scales(qr, _blocks(qc))
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        st["A"], st["SA"] = _quantised_rows(_activations(M, K, g), case["a"])
        if case["b_scale"] == "row":
            st["B"], st["SB"] = _quantised_rows(_activations(N, K, g))
        else:
            shape = (K, N) if case["trans_b"] else (N, K)
            st["B"], st["SB"] = _quantised_blocks(torch.randn(shape, device="cuda", generator=g) / math.sqrt(K))
        st["D"] = torch.empty((M, N), dtype=TYPES[case["out"]], device="cuda")
    elif op == "experts":
        R, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
        st["A"], st["SA"] = _quantised_rows(_activations(R, K, g))
        shape = (E, K, N) if case["trans_b"] else (E, N, K)
        st["B"], st["SB"] = _quantised_blocks(torch.randn(shape, device="cuda", generator=g) / math.sqrt(K))
        st["offsets"] = _loads(R, E, case["skew"], g)
        st["most"] = int(st["offsets"].diff().max())  # rows of the busiest expert
        st["D"] = torch.empty((R, N), dtype=TYPES[case["out"]], device="cuda")
    else:
        T, k, N = case["tokens"], case["top_k"], case["N"]
        slots = T * k
        st["y"] = torch.randn((slots, N), device="cuda", generator=g).bfloat16()
        st["weights"] = torch.rand((T, k), device="cuda", generator=g)
        pos = torch.randperm(slots, device="cuda", generator=g)
        drop = torch.rand(slots, device="cuda", generator=g) < case["drop"]
        st["position"] = pos.masked_fill(drop, -1).to(torch.int32).view(T, k)
        st["grad_out"] = torch.randn((T, N), device="cuda", generator=g).bfloat16()
        st["out"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        # rows that no slot takes keep what they hold
        st["grad_y"] = torch.zeros((slots, N), dtype=torch.bfloat16, device="cuda")
        st["grad_weights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms, 32 bits
def _halving_sum(v):
    """Sum over the last axis by folding its upper half onto the lower one: the order that the router's softmax fixes."""
    n = max(32, 1 << (v.shape[-1] - 1).bit_length())
    v = torch.nn.functional.pad(v, (0, n - v.shape[-1]))
    while n > 1:
        n //= 2
        v = v[..., :n] + v[..., n:]
    return v


def _scores(x, score):
    if score == "sigmoid":
        return torch.reciprocal(1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True).clamp_min(torch.finfo(x.dtype).min)
    e = torch.exp(x - top)
    total = _halving_sum(e) if x.dtype == torch.float32 else e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def _route(x, bias, case):
    """experts [T, k] (-1 where none is left) and weights [T, k] in x's type."""
    T, E = x.shape
    k, G, keep = case["top_k"], case["groups"], case["keep"]
    s = _scores(x, case["score"])
    c = s if bias is None else s + bias
    c = c.masked_fill(x == -math.inf, -math.inf)
    if G > 1:
        best = c.view(T, G, E // G).sort(dim=2, descending=True, stable=True).values
        gs = best[:, :, 0]
        if case["best"] == 2 and E // G > 1:
            gs = torch.where(best[:, :, 1] > -math.inf, gs + best[:, :, 1], gs)
        kept = gs.sort(dim=1, descending=True, stable=True).indices[:, :keep]
        mask = torch.ones((T, G), dtype=torch.bool, device=x.device).scatter_(1, kept, False)
        c = c.masked_fill(mask.repeat_interleave(E // G, 1), -math.inf)
    value, pick = c.sort(dim=1, descending=True, stable=True)
    value, pick = value[:, :k], pick[:, :k]
    there = value > -math.inf
    w = torch.where(there, s.gather(1, pick), torch.zeros_like(value))
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return torch.where(there, pick, torch.full_like(pick, -1)).to(torch.int32), w, s


def _route_grad(s, experts, gw, case):
    """Gradient by the logits of the weights' weighted sum."""
    there = experts >= 0
    at = experts.clamp_min(0).long()
    sj = torch.where(there, s.gather(1, at), torch.zeros_like(gw))
    g = torch.where(there, gw, torch.zeros_like(gw))
    if case["renorm"]:
        total = sj.sum(1, keepdim=True)
        safe = torch.where(total > 0, total, torch.ones_like(total))
        g = torch.where(there & (total > 0), (g - (g * sj).sum(1, keepdim=True) / safe) / safe, torch.zeros_like(g))
    ds = torch.zeros_like(s).scatter_add_(1, at, g)
    if case["score"] == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdim=True))


def _plan(experts, E):
    """offsets [E + 1], order [T k] (sorted row -> slot), position [T, k] (slot -> sorted row)."""
    key = experts.reshape(-1).long()
    key = torch.where(key < 0, torch.full_like(key, E), key)
    n = key.numel()
    order = key.sort(stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=key.device))
    row = torch.arange(n, device=key.device)
    position = torch.empty_like(key).scatter_(0, order, row)
    valid = offsets[E]
    order = torch.where(row < valid, order, torch.full_like(order, -1))
    position = torch.where(position < valid, position, torch.full_like(position, -1))
    return offsets, order.to(torch.int32), position.to(torch.int32).view(experts.shape)


def _by_rows(q, s, dtype=torch.float32):
    return q.to(dtype) * s.to(dtype).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _by_blocks(q, s, dtype=torch.float32):
    s = s.to(dtype).repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]
    return q.to(dtype) * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _quant(x, case):
    dtype, top = FORMATS[case["format"]]
    x = x.t() if case["transpose"] else x
    r, c = x.shape
    v = torch.nn.functional.pad(x, (0, _blocks(c) * BLOCK - c)).view(r, -1, BLOCK)
    amax = v.abs().amax(2).clamp_min(AMAX_MIN)
    q = v * torch.div(torch.full_like(amax, top), amax)[:, :, None]
    return q.clamp(-top, top).view(r, -1)[:, :c].to(dtype), amax / top


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        experts, w, s = _route(st["logits"].float(), st["bias"], case)
        offsets, order, position = _plan(experts, case["experts"])
        out = {"experts": experts, "weights": w, "offsets": offsets, "order": order, "position": position}
        if case["train"]:
            out["grad_logits"] = _route_grad(s, experts, st["grad_weights"], case).to(st["logits"].dtype)
        return out
    if op == "quant":
        x = st["x"] if st["index"] is None else st["x"][st["index"].long() // case["gather"]]
        q, s = _quant(x.float(), case)
        return {"q": q, "scales": s}
    if op == "gemm":
        A = _by_rows(st["A"], st["SA"])
        if case["b_scale"] == "row":
            B = _by_rows(st["B"], st["SB"]).t()
        else:
            B = _by_blocks(st["B"], st["SB"])
            B = B if case["trans_b"] else B.t()
        return (A @ B).to(TYPES[case["out"]])
    if op == "experts":
        return _experts(st, torch.float32).to(TYPES[case["out"]])
    y, pos, w = st["y"], st["position"], st["weights"]
    there = pos >= 0
    at = pos.clamp_min(0).long()
    wj = torch.where(there, w, torch.zeros_like(w))
    rows = y[at].float()
    out = {"out": (rows * wj[:, :, None]).sum(1).to(torch.bfloat16)}
    if case["train"]:
        go = st["grad_out"].float()
        out["grad_weights"] = torch.where(there, (rows * go[:, None, :]).sum(2), torch.zeros_like(w))
        slots, N = y.shape
        gy = y.new_zeros((slots + 1, N))  # the last row takes what the dropped slots give
        row = torch.where(there, at, torch.full_like(at, slots)).view(-1)
        gy.index_copy_(0, row, (wj[:, :, None] * go[:, None, :]).to(gy.dtype).view(slots, N))
        out["grad_y"] = gy[:slots]
    return out


def _experts(st, dtype):
    """Every expert's rows, padded to the busiest one's, times its weights."""
    off, E, R = st["offsets"], st["case"]["experts"], st["case"]["rows"]
    A = _by_rows(st["A"], st["SA"], dtype)
    B = _by_blocks(st["B"], st["SB"], dtype)
    B = B if st["case"]["trans_b"] else B.transpose(1, 2)
    at = off[:-1, None] + torch.arange(st["most"], device=off.device)
    P = torch.bmm(A[at.clamp_max(R - 1)], B)
    row = torch.arange(R, device=off.device)
    e = torch.searchsorted(off[1:], row, right=True)
    return P[e, row - off[e]]


# ---------------------------------------------------------------- the library's operators
def _library(st):
    import tile_scheduling_gb300 as ts

    case = st["case"]
    op = case["op"]
    if op == "route":
        ts.ts_moe_route(st["logits"], st["experts"], st["weights"], bias=st["bias"], score=case["score"],
                        groups=case["groups"], keep_groups=case["keep"], group_best=case["best"],
                        renorm=case["renorm"])
        ts.ts_moe_plan(st["experts"], st["offsets"], st["order"], st["position"])
        out = {n: st[n] for n in ("experts", "weights", "offsets", "order", "position")}
        if case["train"]:
            ts.ts_moe_route_grad(st["logits"], st["experts"], st["grad_weights"], st["grad_logits"],
                                 score=case["score"], renorm=case["renorm"])
            out["grad_logits"] = st["grad_logits"]
        return out
    if op == "quant":
        ts.ts_quant_fp8(st["x"], st["q"], st["scales"], rows=st["index"], rows_div=case["gather"] or 1,
                        transpose=case["transpose"])
        return {"q": st["q"], "scales": st["scales"]}
    if op == "gemm":
        ts.ts_gemm_fp8(st["A"], st["SA"], st["B"], st["SB"], st["D"], trans_b=case["trans_b"])
        return st["D"]
    if op == "experts":
        ts.ts_gemm_fp8_grouped(st["A"], st["SA"], st["B"], st["SB"], st["D"], st["offsets"], trans_b=case["trans_b"])
        return st["D"]
    ts.ts_moe_combine(st["y"], st["position"], st["out"], weights=st["weights"])
    out = {"out": st["out"]}
    if case["train"]:
        ts.ts_moe_combine_grad(st["grad_out"], st["y"], st["position"], st["weights"], st["grad_y"],
                               st["grad_weights"])
        out["grad_weights"], out["grad_y"] = st["grad_weights"], st["grad_y"]
    return out


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- what one pass cannot do without
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        size = 4 if case["logits"] == "f32" else 2
        n = T * E * size + (4 * E if case["bias"] else 0) + T * k * 8 + T * k * 8 + 8 * (E + 1)
        flops = T * E * 6
        if case["train"]:
            n += T * E * size + T * k * 4
            flops += T * E * 4
        return {"bytes": n, "flops": flops}
    if op == "quant":
        R, C, k = case["rows"], case["cols"], case["gather"]
        size = 4 if case["x"] == "f32" else 2
        src = max(1, R // k) if k else R
        n = src * C * size + R * C + (4 * R if k else 0)
        n += 4 * (C * _blocks(R) if case["transpose"] else R * _blocks(C))
        return {"bytes": n, "flops": 3 * R * C}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        sb = N * _blocks(K) if case["b_scale"] == "row" else _blocks(N) * _blocks(K)
        n = M * K + N * K + 4 * (M * _blocks(K) + sb) + M * N * (4 if case["out"] == "f32" else 2)
        return {"bytes": n, "flops": 2 * M * N * K}
    if op == "experts":
        R, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
        hit = E * (1 - (1 - 1 / E) ** R)  # experts that get a row, were the load even
        n = R * K + 4 * R * _blocks(K) + hit * (N * K + 4 * _blocks(N) * _blocks(K)) + 8 * (E + 1)
        return {"bytes": n + R * N * (4 if case["out"] == "f32" else 2), "flops": 2 * R * N * K}
    T, k, N = case["tokens"], case["top_k"], case["N"]
    rows = T * k * (1 - case["drop"])
    n = rows * N * 2 + T * N * 2 + T * k * 8
    flops = 2 * rows * N
    if case["train"]:
        n += T * N * 2 + rows * N * 2 + T * k * 4
        flops += 3 * rows * N
    return {"bytes": n, "flops": flops}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op == "route":
        x = st["logits"].to(d)
        T, E = x.shape
        k, G, keep = case["top_k"], case["groups"], case["keep"]
        out_of = torch.isneginf(x)
        if case["score"] == "sigmoid":
            s = torch.special.expit(x)
        else:
            s = torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
        c = s + (0 if st["bias"] is None else st["bias"].to(d))
        c = torch.where(out_of, torch.full_like(c, -math.inf), c)
        if G > 1:
            n = E // G
            top = c.view(T, G, n).topk(min(case["best"], n), 2).values
            gs = torch.where(torch.isneginf(top), torch.zeros_like(top), top).sum(2)
            gs = torch.where(torch.isneginf(top[:, :, 0]), top[:, :, 0], gs)
            rank = gs.argsort(dim=1, descending=True, stable=True).argsort(1)
            c = torch.where((rank < keep).repeat_interleave(n, 1), c, torch.full_like(c, -math.inf))
        v, e = torch.sort(c, dim=1, descending=True, stable=True)
        v, e = v[:, :k], e[:, :k]
        there = ~torch.isneginf(v)
        chosen = torch.zeros_like(s).scatter_(1, e, there.to(d))  # 1 at the experts taken
        w = s.gather(1, e) * there
        S = w.sum(1, keepdim=True)
        inv = torch.where(S > 0, 1 / S.clamp_min(1e-300), torch.zeros_like(S)) if case["renorm"] else 1.0
        out = {"experts": None, "weights": w * inv, "offsets": None, "order": None, "position": None}
        if case["train"]:
            g = torch.zeros_like(s).scatter_(1, e, st["grad_weights"].to(d) * there)
            ds = chosen * (g - (g * s * chosen).sum(1, keepdim=True) * inv) * inv if case["renorm"] else chosen * g
            if case["score"] == "sigmoid":
                out["grad_logits"] = ds * s * torch.special.expit(-x)
            else:
                out["grad_logits"] = s * ds - s * (s * ds).sum(1, keepdim=True)
        return out
    if op == "quant":
        dtype, top = FORMATS[case["format"]]
        x = st["x"].to(d)
        if st["index"] is not None:
            x = x[torch.div(st["index"].long(), case["gather"], rounding_mode="floor")]
        if case["transpose"]:
            x = x.t().contiguous()
        r, c = x.shape
        block = torch.arange(c, device="cuda") // BLOCK
        amax = torch.zeros((r, _blocks(c)), dtype=d, device="cuda")
        amax.scatter_reduce_(1, block.expand(r, c), x.abs(), "amax")
        amax = amax.clamp_min(AMAX_MIN)
        q = (x * top / amax[:, block]).clamp(-top, top)
        return {"q": q.to(dtype).to(d), "scales": amax / top}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = torch.arange(K, device="cuda") // BLOCK
        nb = torch.arange(N, device="cuda") // BLOCK
        A = st["A"].to(d) * st["SA"].to(d)[:, kb]
        if case["b_scale"] == "row":
            B = st["B"].to(d) * st["SB"].to(d)[:, kb]
        elif case["trans_b"]:
            B = (st["B"].to(d) * st["SB"].to(d)[kb][:, nb]).t()
        else:
            B = st["B"].to(d) * st["SB"].to(d)[nb][:, kb]
        return torch.einsum("mk,nk->mn", A, B)
    if op == "experts":
        R, N, K = case["rows"], case["N"], case["K"]
        kb = torch.arange(K, device="cuda") // BLOCK
        nb = torch.arange(N, device="cuda") // BLOCK
        A = st["A"].to(d) * st["SA"].to(d)[:, kb]
        D = torch.zeros((R, N), dtype=d, device="cuda")
        off = st["offsets"].tolist()
        for e in range(case["experts"]):
            if off[e + 1] > off[e]:
                W, S = st["B"][e].to(d), st["SB"][e].to(d)
                W = W * S[kb][:, nb] if case["trans_b"] else (W * S[nb][:, kb]).t()
                D[off[e]:off[e + 1]] = A[off[e]:off[e + 1]] @ W
        return D
    pos, w = st["position"].long(), st["weights"].to(d)
    T, k = pos.shape
    y = torch.cat([st["y"].to(d), torch.zeros((1, case["N"]), dtype=d, device="cuda")])  # the last row: dropped slots
    at = torch.where(pos >= 0, pos, torch.full_like(pos, len(st["y"])))
    o = torch.zeros((T, case["N"]), dtype=d, device="cuda")
    gw = torch.zeros((T, k), dtype=d, device="cuda")
    gy = torch.zeros_like(y)
    go = st["grad_out"].to(d)
    for j in range(k):
        o += w[:, j:j + 1] * y[at[:, j]]
        if case["train"]:
            gw[:, j] = torch.einsum("tn,tn->t", go, y[at[:, j]])
            gy[at[:, j]] = w[:, j:j + 1] * go
    if case["train"]:
        return {"out": o, "grad_weights": gw, "grad_y": gy[:-1]}
    return {"out": o}
