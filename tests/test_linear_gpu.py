"""A linear layer's products (ts_linear, its two gradient products) and ts_act_grad against a 64-bit reference.

Two kinds of inputs.  Small integers: every product and sum is exact in fp32, so with no activation or
relu the result must be the reference's to the bit (rounded once).  Random values: within a bound derived
from the arithmetic below.
"""
import math
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "gelu_tanh": 1.13, "silu": 1.1}  # the largest of |act'|
BEND = {"none": 0.0, "relu": 0.0, "gelu": 0.8, "gelu_tanh": 0.8, "silu": 0.5}     # the largest of |act''|
HALF = {BF16: 2.0 ** -9, F32: 2.0 ** -25}  # of the bit above the value's leading one: twice this is half a step


def _act(z, act):
    F = torch.nn.functional
    return {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[act](z)


def _slope(z, act):
    z = z.clone().requires_grad_()
    _act(z, act).sum().backward()
    return z.grad


def _pitched(r, c, dtype, step=8, extra=0):
    t = torch.full((max(r, 1), -(-c // step) * step + extra), float("nan"), dtype=dtype, device="cuda")
    return t[:r, :c]


def _fill(r, c, g, dtype=BF16, ints=False, scale=1.0, **kw):
    v = torch.randint(-3, 4, (r, c), device="cuda", generator=g) if ints else \
        scale * torch.randn((r, c), device="cuda", generator=g)
    t = _pitched(r, c, dtype, **kw)
    t.copy_(v)
    return t


def _gen(*key):
    return torch.Generator("cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _sum_bound(S, K):
    # One MMA adds 16 products and the running sum, each aligned to the largest and cut at no less than
    # 23 bits; ceil(K / 16) of them follow each other, and the partial sums stay below S.
    return (17 * -(-K // 16) * 2.0 ** -23 + 2.0 ** -23) * S


def _close(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    worst = float(((got - ref).abs() - bound).max()) if ref.numel() else 0.0
    assert worst <= 0, f"{what}: {worst} past the bound"


SIZES = [(1, 1, 1), (1, 4096, 512), (2, 1000, 1111), (7, 129, 64), (24, 384, 2048), (33, 65, 40), (64, 1024, 1024),
         (127, 65, 300), (128, 128, 128), (129, 257, 1024), (255, 383, 777), (257, 640, 2048), (513, 512, 64),
         (1023, 1025, 255), (2047, 1000, 520)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("extras", ["", "b", "r", "p", "brp", "inplace"])
def test_integers(lib, M, N, K, out, act, extras):
    g = _gen(M, N, K)
    x, w = _fill(M, K, g, ints=True), _fill(N, K, g, ints=True)
    bias = torch.randint(-9, 10, (N,), device="cuda", generator=g).to(BF16 if M % 2 else F32) if "b" in extras else None
    y = _pitched(M, N, out, step=1)
    res = _fill(M, N, g, out, ints=True, step=1) if "r" in extras else None
    if extras == "inplace":
        y = res = _fill(M, N, g, out, ints=True)
    pre = _pitched(M, N, out, step=1, extra=3) if "p" in extras else None
    z = x.double() @ w.double().t() + (bias.double() if bias is not None else 0)
    want = _act(z, act) + (res.double() if res is not None else 0)
    lib.ts_linear(x, w, y, bias=bias, act=act, residual=res, preact=pre)
    lib.ts_sync_and_check()
    assert torch.equal(y, want.to(out))
    if pre is not None:
        assert torch.equal(pre, z.to(out))


@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (300, 700, 192), (129, 515, 2048), (1024, 1024, 320)])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("workers", [0, 1])
def test_tiles(lib, M, N, K, tile, out, pre, workers):
    g = _gen(M, N, K, tile)
    x, w, res = _fill(M, K, g, ints=True), _fill(N, K, g, ints=True), _fill(M, N, g, out, ints=True)
    y, z = _pitched(M, N, out), _pitched(M, N, out) if pre else None
    bias = torch.randint(-9, 10, (N,), device="cuda", generator=g).float()
    lib.ts_linear(x, w, y, bias=bias, residual=res, preact=z, tile=tile, max_workers=workers, act="relu")
    lib.ts_sync_and_check()
    want = x.double() @ w.double().t() + bias.double()
    assert torch.equal(y, (want.relu() + res.double()).to(out))
    if pre:
        assert torch.equal(z, want.to(out))


@pytest.mark.parametrize("M,N,K", [(1, 515, 1024), (19, 384, 512), (257, 515, 300), (700, 1024, 2048)])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
def test_random(lib, M, N, K, out, act):
    g = _gen(M, N, K, act)
    x, w = _fill(M, K, g, scale=1.5), _fill(N, K, g, scale=1 / math.sqrt(K))
    bias, res = torch.randn(N, device="cuda", generator=g), _fill(M, N, g, out)
    y, pre = _pitched(M, N, out), _pitched(M, N, out)
    lib.ts_linear(x, w, y, bias=bias, act=act, residual=res, preact=pre)
    lib.ts_sync_and_check()
    z = x.double() @ w.double().t() + bias.double()
    S = x.double().abs() @ w.double().abs().t() + bias.double().abs()
    err = _sum_bound(S, K)
    _close(pre, z, err + 2 * HALF[out] * z.abs(), f"preact {act}")
    want = _act(z, act) + res.double()
    # the activation's own error: some units in the last place of |z| + 1, and 2^-24 |z| in its exponent
    own = 2.0 ** -20 * (z.abs() + 1) if act not in ("none", "relu") else 0
    _close(y, want, SLOPE[act] * err + own + 2.0 ** -23 * (want.abs() + res.double().abs()) + 2 * HALF[out] * want.abs(), act)


GRAD_SIZES = [(1, 1, 1), (16, 64, 64), (7, 130, 40), (129, 257, 300), (515, 128, 1000), (1021, 520, 513), (2048, 384, 640)]


@pytest.mark.parametrize("M,N,K", GRAD_SIZES)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("tile", ["auto", "128x128", "128x256", "256x256"])
def test_gradient_products_integers(lib, M, N, K, out, tile):
    g = _gen(M, N, K, 5)
    gz, w, x = (_fill(*s, g, ints=True) for s in ((M, N), (N, K), (M, K)))
    gx, gw = _pitched(M, K, out, step=1), _pitched(N, K, out, step=1)
    lib.ts_linear_grad_input(gz, w, gx, tile=tile)
    lib.ts_linear_grad_weight(gz, x, gw, tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(gx, (gz.double() @ w.double()).to(out))
    want = gz.double().t() @ x.double()
    assert torch.equal(gw, want.to(out))
    # accumulated onto another matrix, and in place
    base = _fill(N, K, g, out, ints=True)
    lib.ts_linear_grad_weight(gz, x, gw, base=base, tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(gw, (want + base.double()).to(out))
    want = want + base.double()
    lib.ts_linear_grad_weight(gz, x, base, base=base, tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(base, want.to(out))


@pytest.mark.parametrize("M,N,K", [(17, 64, 130), (300, 257, 515)])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act", ACTS[1:])
def test_gradient_through_activation(lib, M, N, K, out, act):
    g = _gen(M, N, K, act, 7)
    gz, w, pre = _fill(M, N, g, scale=0.1), _fill(N, K, g), _fill(M, K, g, out, scale=2.0)
    gx = _pitched(M, K, out)
    lib.ts_linear_grad_input(gz, w, gx, act=act, preact=pre)
    lib.ts_sync_and_check()
    s = gz.double() @ w.double()
    slope = _slope(pre.double(), act)
    S = gz.double().abs() @ w.double().abs()
    own = 2.0 ** -20 * (pre.double().abs() + 1)  # of the slope
    _close(gx, s * slope, SLOPE[act] * _sum_bound(S, N) + own * s.abs() + (2.0 ** -23 + 2 * HALF[out]) * (s * slope).abs(), act)


@pytest.mark.parametrize("M,N", [(1, 1), (1, 1000), (3, 64), (127, 65), (128, 512), (129, 513), (1000, 72), (4099, 130), (8192, 256)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("aligned", [True, False])
def test_act_grad(lib, M, N, dtype, act, aligned):
    g = _gen(M, N, act, 9)
    step = 8 if aligned else 1
    gy, pre = _fill(M, N, g, dtype, step=step), _fill(M, N, g, dtype, scale=2.0, step=step)
    gz = _pitched(M, N, dtype, step=step)
    gb = torch.full((N,), float("nan"), device="cuda")
    lib.ts_act_grad(gy, pre if act != "none" else None, gz, gb, act=act)
    lib.ts_sync_and_check()
    want = gy.double() * _slope(pre.double(), act)
    own = (2.0 ** -20 * (pre.double().abs() + 1) if act not in ("none", "relu") else 0) * gy.double().abs()
    _close(gz, want, own + (2.0 ** -23 + 2 * HALF[dtype]) * want.abs(), act)
    # each sum passes at most M / 8 / 32 + 1 additions in a thread, 32 in the CTA and 8 in the cluster
    adds = M / 32 + 42
    _close(gb, want.sum(0), own.sum(0) + adds * 2.0 ** -24 * want.abs().sum(0) if act not in ("none", "relu") else
           adds * 2.0 ** -24 * want.abs().sum(0) + 1e-30, "bias " + act)
    # the bias gradient alone, and in place
    if act == "none":
        gb2 = torch.empty_like(gb)
        lib.ts_act_grad(gy, None, None, gb2)
        assert torch.equal(gb, gb2)
    else:
        lib.ts_act_grad(gy, pre, pre, act=act)
        assert torch.equal(pre, gz)


def test_gradients_against_differences(lib):
    """The layer's gradients against central differences of its own fp32 forward pass."""
    M, N, K = 40, 72, 56
    g = _gen(11)
    x, w, bias = _fill(M, K, g), _fill(N, K, g, scale=0.2), torch.randn(N, device="cuda", generator=g)
    gy = _fill(M, N, g, F32)

    def loss(x, w, bias, act):
        y = torch.empty((M, N), device="cuda")
        lib.ts_linear(x, w, y, bias=bias, act=act)
        return float((y.double() * gy.double()).sum())

    for act in ACTS[1:]:
        z = torch.empty((M, N), device="cuda")
        lib.ts_linear(x, w, torch.empty_like(z), bias=bias, act=act, preact=z)
        gz32, gb = torch.empty_like(z), torch.empty(N, device="cuda")
        lib.ts_act_grad(gy, z, gz32, gb, act=act)
        gz = gz32.bfloat16()
        gx, gw = torch.empty((M, K), device="cuda"), torch.empty((N, K), device="cuda")
        lib.ts_linear_grad_input(gz, w, gx)
        lib.ts_linear_grad_weight(gz, x, gw)
        lib.ts_sync_and_check()
        eps = 2.0 ** -4
        for name, grad in (("bias", gb), ("x", gx), ("w", gw)):
            t = {"bias": bias, "x": x, "w": w}[name]
            d = torch.zeros_like(t)
            at = (3,) if name == "bias" else (3, 5)
            # steps that the type holds exactly
            lo, hi = t.clone(), t.clone()
            hi[at] = t[at] + eps
            lo[at] = t[at] - eps
            step = float(hi[at].double() - lo[at].double())
            args = lambda v: (v if name == "x" else x, v if name == "w" else w, v if name == "bias" else bias, act)  # noqa: E731
            num = (loss(*args(hi)) - loss(*args(lo))) / step
            # The gradient's own rounding (grad_z to bf16) against the sum of the magnitudes that make it,
            # and the difference's: y in fp32, and relu's corner or the third derivative over the step.
            size = {"bias": gz32[:, 3].abs().sum(), "x": (gz32[3].abs() * w[:, 5].float().abs()).sum(),
                    "w": (gz32[:, 3].abs() * x[:, 5].float().abs()).sum()}[name]
            move = {"bias": torch.ones(M, device="cuda"), "x": w[:, 5].float(), "w": x[:, 5].float()}[name].abs() * eps
            gys = {"bias": gy[:, 3], "x": gy[3], "w": gy[:, 3]}[name].abs()
            zs = {"bias": z[:, 3], "x": z[3], "w": z[:, 3]}[name]
            if act == "relu":  # outputs whose corner lies within the step
                curve = float((gys * move / eps * (zs.abs() <= move)).sum())
            else:  # |act'''| < 2.5, the central difference's remainder is a sixth of it times the step squared
                curve = float((gys * (move / eps) * 2.5 / 6 * move ** 2).sum())
            noise = float((gy.abs() * (z.abs() + 1)).sum()) * 2.0 ** -20 / step
            assert abs(num - float(grad[at])) <= curve + 2.0 ** -8 * float(size) + noise, (act, name)
            del d


def test_empty(lib):
    x, w = torch.zeros((3, 8), dtype=BF16, device="cuda")[:, :0], torch.zeros((5, 8), dtype=BF16, device="cuda")[:, :0]
    y, bias = torch.full((3, 5), 9.0, device="cuda"), torch.arange(5, device="cuda").float() - 2
    res, pre = torch.ones((3, 5), device="cuda"), torch.empty((3, 5), device="cuda")
    lib.ts_linear(x, w, y, bias=bias, act="relu", residual=res, preact=pre)
    lib.ts_sync_and_check()
    assert torch.equal(y, bias.relu().expand(3, 5) + 1) and torch.equal(pre, bias.expand(3, 5).contiguous())
    lib.ts_linear(torch.empty((0, 8), dtype=BF16, device="cuda"), torch.empty((5, 8), dtype=BF16, device="cuda"),
                  torch.empty((0, 5), device="cuda"))
    gw = torch.full((5, 8), 9.0, device="cuda")
    lib.ts_linear_grad_weight(torch.empty((0, 5), dtype=BF16, device="cuda"), torch.empty((0, 8), dtype=BF16, device="cuda"), gw)
    gb = torch.full((5,), 9.0, device="cuda")
    lib.ts_act_grad(torch.empty((0, 5), device="cuda"), None, None, gb)
    lib.ts_sync_and_check()
    assert not gw.any() and not gb.any()


def test_special_values(lib):
    """Infinities and NaN stay in the rows and columns that use them; activations keep their limits."""
    M, N, K = 200, 300, 128
    g = _gen(13)
    for act in ACTS:
        x, w = _fill(M, K, g), _fill(N, K, g, scale=0.1)
        x[5, 7], x[9, 3], w[4, 1] = float("nan"), float("inf"), float("inf")
        y = torch.empty((M, N), device="cuda")
        lib.ts_linear(x, w, y, act=act)
        lib.ts_sync_and_check()
        ok = torch.ones((M, N), dtype=torch.bool, device="cuda")
        ok[5], ok[9], ok[:, 4] = False, False, False
        assert torch.isfinite(y[ok]).all()
        assert torch.isnan(y[5]).all()
    # far arguments of the activations and of their slopes
    z = torch.tensor([[-1e30, -3e4, -100.0, -30.0, 0.0, 30.0, 100.0, 3e4, 1e30, float("nan")]], device="cuda")
    for act in ACTS[1:]:
        got, one = torch.empty_like(z), torch.ones_like(z)
        lib.ts_act_grad(one, z, got, act=act)
        lib.ts_sync_and_check()
        want = torch.tensor([[0, 0, 0, 0, 0.0 if act == "relu" else 0.5, 1, 1, 1, 1, float("nan")]], device="cuda")
        assert torch.allclose(got, want, atol=1e-6, rtol=0, equal_nan=True), act
        y = torch.empty_like(z)
        x0, w0 = torch.zeros((1, 8), dtype=BF16, device="cuda"), torch.zeros((10, 8), dtype=BF16, device="cuda")
        lib.ts_linear(x0, w0, y, bias=z[0].contiguous(), act=act)
        lib.ts_sync_and_check()
        want = torch.where(z > 0, z, torch.where(z != z, z, torch.zeros_like(z)))
        assert torch.allclose(y, want, atol=1e-6, rtol=1e-6, equal_nan=True), act
