"""The mixture-of-experts layer's composition at sizes and inputs off its usual grid.

Each operator has its own test against 64 bits; here the layer's gradients are recomputed in 64 bits from
the operands as the operators quantise them, so the bounds are those of fp32 sums and bf16 results alone.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _rows(q, s):
    return q.double() * s.double().repeat_interleave(128, 1)[:, : q.shape[1]]


def _blocks(q, s):
    s = s.double().repeat_interleave(128, -2)[..., : q.shape[-2], :].repeat_interleave(128, -1)[..., : q.shape[-1]]
    return q.double() * s


def _quant(lib, x, dtype=torch.float8_e4m3fn, transpose=False):
    r, c = x.shape[::-1] if transpose else x.shape
    q = torch.empty((r, c), dtype=dtype, device="cuda")
    s = torch.empty((r, -(-c // 128)), dtype=torch.float32, device="cuda")
    lib.ts_quant_fp8(x, q, s, transpose=transpose)
    return _rows(q, s)


def _layer(T, E, N, K, k, **kw):
    from tile_scheduling_gb300.moe import MoeLayer

    g = torch.Generator("cuda").manual_seed(T + E + K)
    randn = lambda *s: torch.randn(s, dtype=torch.float32, device="cuda", generator=g)  # noqa: E731
    layer = MoeLayer(randn(E, K) / K ** 0.5, randn(E, N, K) / K ** 0.5, k, **kw)
    return layer, randn(T, K).bfloat16(), randn(T, N).bfloat16()


def _check_layer(lib, layer, x, grad_out, out, s, grad_x, grad_router):
    (T, K), (E, N), k = x.shape, layer.w.shape[:2], layer.top_k
    slot = s["order"].long()
    e, pos = s["experts"].flatten().long()[slot], s["position"].long()
    w = _blocks(layer.w, layer.sw)
    # forward
    logits = x.double() @ layer.router.double().t()
    mag = x.double().abs() @ layer.router.double().abs().t()
    assert bool(((s["logits"].double() - logits).abs() <= 2.0 ** -20 * mag).all())
    q = _quant(lib, x)[slot // k]
    y = torch.einsum("rk,rnk->rn", q, w[e])
    mag = torch.einsum("rk,rnk->rn", q.abs(), w[e].abs())
    y_err = 2.0 ** -8 * y.abs() + 2.0 ** -16 * mag
    want = (y[pos] * s["weights"].double()[:, :, None]).sum(1)
    err = (y_err[pos] * s["weights"].double()[:, :, None]).sum(1) + 2.0 ** -8 * want.abs() + \
        2.0 ** -20 * (y[pos].abs() * s["weights"].double()[:, :, None]).sum(1)
    assert out.shape == (T, N) and bool(((out.double() - want).abs() <= 2 * err + 1e-30).all())
    # the experts' input gradient: grad_y in bf16, then e5m2, as the layer does
    gy, gw = torch.zeros((T * k, N), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s["weights"])
    lib.ts_moe_combine_grad(grad_out.contiguous(), s["y"], s["position"], s["weights"], gy, gw)
    gq = _quant(lib, gy, torch.float8_e5m2)
    rows, mag = torch.einsum("rn,rnk->rk", gq, w[e]), torch.einsum("rn,rnk->rk", gq.abs(), w[e].abs())
    from_experts = rows[pos].sum(1)
    err = (2.0 ** -8 * rows.abs() + 2.0 ** -16 * mag)[pos].sum(1) + 2.0 ** -8 * from_experts.abs()
    # through the router: bf16 gradients of the logits times its bf16 weights
    gl = torch.zeros_like(s["logits"])
    lib.ts_moe_route_grad(s["logits"], s["experts"], gw, gl, score=layer.score, renorm=layer.renorm, scale=layer.scale)
    glb = gl.bfloat16().double()
    from_router, mag = glb @ layer.router.double(), glb.abs() @ layer.router.double().abs()
    want = from_experts + from_router
    err = err + 2.0 ** -8 * from_router.abs() + 2.0 ** -20 * mag + 2.0 ** -8 * want.abs()
    assert grad_x.shape == (T, K) and bool(((grad_x.double() - want).abs() <= 2 * err + 1e-30).all())
    # the router's weights: both sides quantised along the tokens
    if T:
        a, b = _quant(lib, gl, transpose=True), _quant(lib, x, transpose=True)
        want, mag = a @ b.t(), a.abs() @ b.abs().t()
        assert bool(((grad_router.double() - want).abs() <= 2.0 ** -15 * mag + 1e-30).all())
    assert grad_router.shape == (E, K) and (T or not grad_router.any())


@pytest.mark.parametrize("T,E,N,K,k,score", [(37, 12, 72, 264, 3, "softmax"), (130, 60, 128, 136, 6, "sigmoid"),
                                             (9, 4, 200, 256, 4, "softmax"), (64, 13, 33, 100, 2, "sigmoid"),
                                             (5, 1, 128, 128, 1, "softmax"), (300, 7, 130, 129, 7, "sigmoid"),
                                             (0, 12, 128, 128, 2, "softmax")])
def test_rows_off_the_16_byte_grid(lib, T, E, N, K, k, score):
    layer, x, grad_out = _layer(T, E, N, K, k, score=score)
    out, s = layer.forward(x)
    grads = layer.backward(s, grad_out)
    lib.ts_sync_and_check()
    _check_layer(lib, layer, x, grad_out, out, s, *grads)


def test_default_dtype_does_not_reach_the_layers_buffers(lib):
    layer, x, grad_out = _layer(40, 8, 64, 128, 2)
    try:
        torch.set_default_dtype(torch.float64)
        out, s = layer.forward(x)
        grads = layer.backward(s, grad_out)
        lib.ts_sync_and_check()
    finally:
        torch.set_default_dtype(torch.float32)
    _check_layer(lib, layer, x, grad_out, out, s, *grads)


@pytest.mark.parametrize("how", ["sum", "column", "transposed"])
def test_gradients_that_are_not_dense(lib, how):
    # what out.sum().backward() and friends hand over: one value, or one row, expanded; columns first
    T, N = 40, 64
    layer, x, grad_out = _layer(T, 8, N, 128, 2)
    grad_out = {"sum": torch.ones((), dtype=torch.bfloat16, device="cuda").expand(T, N),
                "column": grad_out[:1].expand(T, N), "transposed": grad_out.t().contiguous().t()}[how]
    out, s = layer.forward(x)
    grads = layer.backward(s, grad_out)
    lib.ts_sync_and_check()
    _check_layer(lib, layer, x, grad_out, out, s, *grads)
