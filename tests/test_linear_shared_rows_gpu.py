"""Operands and outputs that are column ranges of the same rows: a layer's state kept in one buffer."""
import pytest
import torch

from orth_accuracy import check, matrix

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _ints(g, *shape, dtype=BF16):
    return torch.randint(-3, 4, shape, device="cuda", generator=g).to(dtype)


# few tokens; tokens as columns; a cluster's shared K; persistent tiles
@pytest.mark.parametrize("M,N,K", [(3, 72, 200), (30, 304, 520), (60, 200, 640), (152, 203, 904), (700, 1500, 320), (1000, 2001, 1104)])
@pytest.mark.parametrize("order", ["xyrz", "zryx", "yxzr"])
def test_layer_in_one_buffer(lib, M, N, K, order):
    """x, y, residual and pre-activations side by side, and eight columns of sevens."""
    g = torch.Generator("cuda").manual_seed(M)
    wide = {"x": -(-K // 8) * 8, "y": N, "r": N, "z": N}
    total = sum(wide.values()) + 8
    buf = torch.full((M, -(-total // 8) * 8 + 8), 7.0, dtype=BF16, device="cuda")
    at, parts = 0, {}
    for name in order:
        if name == "x":
            at = -(-at // 8) * 8
        parts[name] = buf[:, at:at + (K if name == "x" else N)]
        at += wide[name]
    x, y, r, z = (parts[n] for n in "xyrz")
    w = _ints(g, N, K)
    x.copy_(_ints(g, M, K))
    r.copy_(_ints(g, M, N))
    x0, r0 = x.clone(), r.clone()
    lib.ts_linear(x, w, y, act="relu", residual=r, preact=z)
    lib.ts_sync_and_check()
    want = x0.double() @ w.double().t()
    assert torch.equal(z, want.to(BF16)) and torch.equal(y, (want.relu() + r0.double()).to(BF16))
    assert torch.equal(x, x0) and torch.equal(r, r0)
    for t in (x, y, r, z):
        t.fill_(7)
    assert bool((buf == 7).all())


@pytest.mark.parametrize("M,N,K", [(30, 304, 520), (152, 200, 904), (1000, 2000, 1104)])
def test_gradients_in_one_buffer(lib, M, N, K):
    g = torch.Generator("cuda").manual_seed(M)
    buf = torch.full((M, N + 2 * K + 8), 7.0, dtype=BF16, device="cuda")
    gz, gx, z = buf[:, :N], buf[:, N:N + K], buf[:, N + K:N + 2 * K]
    gz.copy_(_ints(g, M, N))
    z.copy_(_ints(g, M, K))
    w = _ints(g, N, K)
    gz0, z0 = gz.clone(), z.clone()
    lib.ts_linear_grad_input(gz, w, gx, act="relu", preact=z)
    lib.ts_sync_and_check()
    assert torch.equal(gx, ((gz0.double() @ w.double()) * (z0 > 0)).to(BF16))
    assert torch.equal(gz, gz0) and torch.equal(z, z0) and bool((buf[:, N + 2 * K:] == 7).all())
    # a weight gradient beside its base
    both = torch.zeros((N, 2 * K), device="cuda")
    both[:, :K] = _ints(g, N, K, dtype=F32)
    base = both[:, :K].clone()
    x = _ints(g, M, K)
    lib.ts_linear_grad_weight(gz, x, both[:, K:], base=both[:, :K])
    lib.ts_sync_and_check()
    assert torch.equal(both[:, K:].double(), base.double() + gz0.double().t() @ x.double()) and torch.equal(both[:, :K], base)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N", [(1, 5), (70, 33), (1000, 1024), (513, 4001)])
def test_activation_gradient_of_a_part(lib, dtype, M, N):
    g = torch.Generator("cuda").manual_seed(N)
    buf = torch.full((M, 3 * N + 4), 7.0, dtype=dtype, device="cuda")
    gy, z, gz = buf[:, :N], buf[:, N:2 * N], buf[:, 2 * N:3 * N]
    gy.copy_(_ints(g, M, N))
    z.copy_(_ints(g, M, N))
    gb = torch.empty(N, device="cuda")
    want = gy.double() * (z > 0)
    lib.ts_act_grad(gy, z, gz, gb, act="relu")
    lib.ts_sync_and_check()
    assert torch.equal(gz.double(), want) and torch.equal(gb.double(), want.sum(0))
    assert bool((buf[:, 3 * N:] == 7).all())


@pytest.mark.parametrize("n,R,C", [(3, 100, 64), (4, 130, 33), (3, 1300, 1104), (2, 2050, 700)])
def test_orthogonalised_side_by_side(lib, n, R, C):
    """Matrices of a batch that are column ranges of the same rows, as heads of one projection are."""
    g = torch.zeros((R, n * C + 8), dtype=BF16, device="cuda")[:, :n * C].unflatten(1, (n, C)).transpose(0, 1)
    g.copy_(matrix(R, C, n, lead=(n,), device="cuda"))
    keep = torch.full((R, n * C + 8), 7.0, dtype=BF16, device="cuda")
    out = keep[:, :n * C].unflatten(1, (n, C)).transpose(0, 1)
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    for i in range(n):
        check(out[i], g[i])
    assert bool((keep[:, n * C:] == 7).all())
    # and beside the result, in the same rows
    buf = torch.empty((R, 2 * C), dtype=BF16, device="cuda")
    buf[:, :C] = g[0]
    lib.ts_orthogonalise(buf[:, :C], buf[:, C:])
    lib.ts_sync_and_check()
    check(buf[:, C:], g[0])
    assert torch.equal(buf[:, :C], g[0])
