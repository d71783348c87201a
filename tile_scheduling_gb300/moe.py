"""A mixture-of-experts layer on the library's operators, forward and backward.

The layer is a router and one linear map per expert:

    logits = x @ router.T;  experts, weights = the top_k of each token
    out[t] = sum_j weights[t, j] * W[experts[t, j]] @ x[t]

It shows the operators in the order a user calls them and keeps what the backward
pass needs.  backward gives the gradients of the input and of the router; the experts'
weights stay as they are (no operator forms their gradient from a plan).

Rounded to fewer bits, in this order: the experts' weights (once, e4m3 in 128 x 128
blocks), x (e4m3 for each row and 128 columns, for the experts; bf16 for the router),
y and the output (bf16); backward, grad_y (bf16, then e5m2, whose range gradients need),
the rows' gradients (bf16), grad_logits (bf16 for the input's gradient; e4m3 along the
tokens, with x, for the router's weights, whose sum over the tokens averages the
rounding) and grad_x (bf16).

Usage: python -m tile_scheduling_gb300.run_workload moe
"""
from __future__ import annotations

import torch

import tile_scheduling_gb300 as ts

BLOCK = 128


def quantise_blocks(w: torch.Tensor):
    """Weights [..., R, C] as e4m3 and one fp32 scale for each 128 x 128 block (rows padded to 16 bytes).

    Done once for weights, in plain torch."""
    R, C = w.shape[-2:]
    lead = w.shape[:-2]
    rb, cb = -(-R // BLOCK), -(-C // BLOCK)
    v = torch.nn.functional.pad(w.float(), (0, cb * BLOCK - C, 0, rb * BLOCK - R)).view(*lead, rb, BLOCK, cb, BLOCK)
    amax = v.abs().amax((-3, -1)).clamp_min(2.0 ** -100)
    q = (v * (448.0 / amax)[..., :, None, :, None]).clamp_(-448.0, 448.0).view(*lead, rb * BLOCK, cb * BLOCK)
    out = torch.empty((*lead, R, -(-C // 16) * 16), dtype=torch.float8_e4m3fn, device=w.device)[..., :C]
    out.copy_(q[..., :R, :C])
    return out, (amax / 448.0).contiguous()


def _fp8(rows: int, cols: int, device, dtype=torch.float8_e4m3fn):
    """Room for a quantised matrix: rows on 16-byte boundaries, scales with their rows contiguous."""
    q = torch.empty((rows, -(-cols // 16) * 16), dtype=dtype, device=device)[:, :cols]
    return q, torch.empty((-(-cols // BLOCK), rows), dtype=torch.float32, device=device).t()


def _bf16_rows(x: torch.Tensor) -> torch.Tensor:
    """A matrix as bf16 with its rows on 16-byte boundaries, where the bf16 products take them (x itself if it is)."""
    rows, cols = x.shape
    if x.dtype is torch.bfloat16 and x.stride(1) == 1 and x.data_ptr() % 16 == 0 and \
            (rows <= 1 or (x.stride(0) >= cols and x.stride(0) % 8 == 0)):
        return x
    out = torch.empty((rows, -(-cols // 8) * 8), dtype=torch.bfloat16, device=x.device)[:, :cols]
    return out.copy_(x)


class MoeLayer:
    """router [E, K] and experts [E, N, K] (bf16 or fp32 CUDA tensors); routing options as ts_moe_route."""

    def __init__(self, router: torch.Tensor, experts: torch.Tensor, top_k: int, score="softmax", bias=None, groups=1,
                 keep_groups=0, group_best=1, renorm=True, scale=1.0):
        self.router = _bf16_rows(router)
        self.w, self.sw = quantise_blocks(experts)
        self.top_k, self.bias, self.score, self.renorm, self.scale = top_k, bias, score, renorm, scale
        self.groups = dict(groups=groups, keep_groups=keep_groups, group_best=group_best)

    def forward(self, x: torch.Tensor):
        """x [T, K] bf16 -> (out [T, N] bf16, what backward needs)."""
        if x.dtype is not torch.bfloat16:
            raise TypeError("x must be a torch.bfloat16 tensor")
        T, K = x.shape
        E, N = self.w.shape[0], self.w.shape[1]
        k = self.top_k
        f32, i32, bf16 = (dict(dtype=t, device=x.device) for t in (torch.float32, torch.int32, torch.bfloat16))
        s = {"x": x, "logits": torch.empty((T, E), **f32), "experts": torch.empty((T, k), **i32),
             "weights": torch.empty((T, k), **f32), "offsets": torch.empty(E + 1, dtype=torch.int64, device=x.device),
             "order": torch.empty(T * k, **i32), "position": torch.empty((T, k), **i32),
             "y": torch.empty((T * k, N), **bf16)}
        ts.ts_gemm_bf16_ex(_bf16_rows(x), self.router, s["logits"])
        ts.ts_moe_route(s["logits"], s["experts"], s["weights"], bias=self.bias, score=self.score, renorm=self.renorm,
                        scale=self.scale, **self.groups)
        ts.ts_moe_plan(s["experts"], s["offsets"], s["order"], s["position"])
        # tokens laid out by expert and quantised on the way
        s["q"], s["sq"] = _fp8(T * k, K, x.device)
        ts.ts_quant_fp8(x, s["q"], s["sq"], rows=s["order"], rows_div=k)
        ts.ts_gemm_fp8_grouped(s["q"], s["sq"], self.w, self.sw, s["y"], s["offsets"])
        out = torch.empty((T, N), **bf16)
        ts.ts_moe_combine(s["y"], s["position"], out, weights=s["weights"])
        return out, s

    def backward(self, s: dict, grad_out: torch.Tensor):
        """grad_out [T, N] bf16 -> (grad_x [T, K] bf16, grad_router [E, K] fp32)."""
        T, K = s["x"].shape
        E, N = self.w.shape[0], self.w.shape[1]
        k = self.top_k
        device = grad_out.device
        f32, bf16 = (dict(dtype=t, device=device) for t in (torch.float32, torch.bfloat16))
        grad_out = grad_out.contiguous()  # a sum's gradient is one value expanded to [T, N]
        grad_y = torch.empty((T * k, N), **bf16)
        grad_w = torch.empty((T, k), **f32)
        ts.ts_moe_combine_grad(grad_out, s["y"], s["position"], s["weights"], grad_y, grad_w)
        # the experts' input gradient: gradients in e5m2, the same weights read the other way
        gq, gs = _fp8(T * k, N, device, torch.float8_e5m2)
        ts.ts_quant_fp8(grad_y, gq, gs)
        grad_rows = torch.empty((T * k, K), **bf16)
        ts.ts_gemm_fp8_grouped(gq, gs, self.w, self.sw, grad_rows, s["offsets"], trans_b=True)
        grad_x = torch.empty((T, K), **bf16)
        ts.ts_moe_combine(grad_rows, s["position"], grad_x)  # the gather's gradient: a sum over the token's slots
        # the router: through the weights to the logits, then its weights' gradient along the tokens
        grad_logits = torch.empty_like(s["logits"])
        ts.ts_moe_route_grad(s["logits"], s["experts"], grad_w, grad_logits, score=self.score, renorm=self.renorm,
                             scale=self.scale)
        lq, ls = _fp8(E, T, device)
        xq, xs = _fp8(K, T, device)
        ts.ts_quant_fp8(grad_logits, lq, ls, transpose=True)
        ts.ts_quant_fp8(s["x"], xq, xs, transpose=True)
        grad_router = torch.empty((E, K), **f32)
        ts.ts_gemm_fp8(lq, ls, xq, xs, grad_router)
        from_router = torch.empty((T, K), **bf16)
        ts.ts_gemm_bf16_ex(_bf16_rows(grad_logits), _bf16_rows(self.router.t()), from_router)
        return grad_x.add_(from_router), grad_router
