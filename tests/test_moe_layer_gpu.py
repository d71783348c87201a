"""The operators together, as a mixture-of-experts layer runs them, against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _rows(q, s):
    return q.double() * s.double().repeat_interleave(128, 1)[:, : q.shape[1]]


def _blocks(q, s):
    s = s.double().repeat_interleave(128, -2)[..., : q.shape[-2], :].repeat_interleave(128, -1)[..., : q.shape[-1]]
    return q.double() * s


@pytest.mark.parametrize("T,E,N,K,k,score", [(1, 8, 256, 128, 2, "softmax"), (37, 16, 200, 264, 4, "sigmoid"),
                                             (500, 8, 512, 384, 2, "softmax"), (1030, 64, 128, 136, 6, "sigmoid")])
def test_layer_forward_and_backward(lib, T, E, N, K, k, score):
    from tile_scheduling_gb300.moe import MoeLayer

    g = torch.Generator("cuda").manual_seed(T + E)
    x = torch.randn((T, K), device="cuda", generator=g).bfloat16()
    layer = MoeLayer(torch.randn((E, K), device="cuda", generator=g) / K ** 0.5,
                     torch.randn((E, N, K), device="cuda", generator=g) / K ** 0.5, k, score=score)
    out, s = layer.forward(x)
    grad_out = torch.randn((T, N), device="cuda", generator=g).bfloat16()
    grad_x, grad_router = layer.backward(s, grad_out)
    lib.ts_sync_and_check()

    # the layout: each row holds its slot's token, and experts own consecutive rows
    off, order = s["offsets"].tolist(), s["order"].long()
    assert off[0] == 0 and off[-1] == T * k and sorted(order.tolist()) == list(range(T * k))
    e_of_row = s["experts"].flatten().long()[order]
    assert torch.equal(e_of_row, e_of_row.sort().values)

    # forward, from the operands as they were quantised
    q, w = _rows(s["q"], s["sq"]), _blocks(layer.w, layer.sw)
    assert bool(((q - x.double()[order // k]).abs() <= 2.0 ** -4 * q.abs() + 2.0 ** -9 * s["sq"].double().amax()).all())
    y = torch.einsum("rk,rnk->rn", q, w[e_of_row])
    scale = torch.einsum("rk,rnk->rn", q.abs(), w[e_of_row].abs())
    # one bf16 rounding, and the 2^-16 of the magnitudes that the products' own test allows
    assert bool(((s["y"].double() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -16 * scale).all())
    rows = s["y"].double()[s["position"].long()] * s["weights"].double()[:, :, None]
    assert bool(((out.double() - rows.sum(1)).abs() <= 2.0 ** -8 * rows.sum(1).abs() + 2.0 ** -20 * rows.abs().sum(1)).all())

    # backward: against the same operators' definitions on the layer's own values.  grad_y is rounded to bf16
    # (2^-9) and to e5m2 (2^-3, or its grid's step of the block's largest); the rows' gradient to bf16
    go = grad_out.double()
    gy = (s["weights"].double()[:, :, None] * go[:, None, :]).view(T * k, N)[order]
    gr = torch.einsum("rn,rnk->rk", gy, w[e_of_row])
    mag = torch.einsum("rn,rnk->rk", gy.abs(), w[e_of_row].abs())
    dw = (rows_dot(go, s["y"].double()[s["position"].long()]))
    sc = torch.sigmoid(s["logits"].double()) if score == "sigmoid" else torch.softmax(s["logits"].double(), 1)
    se = sc.gather(1, s["experts"].long())
    S = se.sum(1, keepdim=True)
    ds = torch.zeros_like(sc).scatter_add_(1, s["experts"].long(), (dw - (dw * se).sum(1, keepdim=True) / S) / S)
    gl = ds * sc * (1 - sc) if score == "sigmoid" else sc * (ds - (ds * sc).sum(1, keepdim=True))
    want = gr[s["position"].long()].sum(1) + gl @ layer.router.double()
    bound = 0.14 * mag[s["position"].long()].sum(1) + 2.0 ** -6 * gl.abs() @ layer.router.double().abs() + 1e-6
    assert bool(((grad_x.double() - want).abs() <= bound).all())
    # e4m3 on both sides of the router's weight gradient: 2^-4 each of the magnitudes, and its smallest step
    want, mag = gl.t() @ x.double(), gl.abs().t() @ x.double().abs()
    step = 2.0 ** -9 * (gl.abs().amax() * x.double().abs().amax()) * T
    assert bool(((grad_router.double() - want).abs() <= 0.14 * mag + step).all())


def rows_dot(go, rows):
    return (rows * go[:, None, :]).sum(2)


def test_layer_repeats_to_the_bit(lib):
    from tile_scheduling_gb300.moe import MoeLayer

    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((300, 256), device="cuda", generator=g).bfloat16()
    layer = MoeLayer(torch.randn((16, 256), device="cuda", generator=g), torch.randn((16, 384, 256), device="cuda", generator=g), 4)
    go = torch.randn((300, 384), device="cuda", generator=g).bfloat16()
    first = None
    for _ in range(3):
        out, s = layer.forward(x)
        gx, gr = layer.backward(s, go)
        lib.ts_sync_and_check()
        if first is None:
            first = (out, gx, gr)
        assert all(torch.equal(a, b) for a, b in zip(first, (out, gx, gr)))


def test_layer_in_a_cuda_graph(lib):
    from tile_scheduling_gb300.moe import MoeLayer

    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn((64, 256), device="cuda", generator=g).bfloat16()
    layer = MoeLayer(torch.randn((8, 256), device="cuda", generator=g), torch.randn((8, 256, 256), device="cuda", generator=g), 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = layer.forward(x)
    x.copy_(torch.randn((64, 256), device="cuda", generator=g).bfloat16())
    graph.replay()
    lib.ts_sync_and_check()
    again, _ = layer.forward(x)
    lib.ts_sync_and_check()
    assert torch.equal(out, again)
