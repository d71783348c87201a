"""Offsets past 2^31 elements in a linear layer's operators, spot-checked at the far end."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _ints(*shape):
    return torch.randint(-3, 4, shape, device="cuda", dtype=torch.int8).to(BF16)


@pytest.mark.parametrize("extras", [False, True])
def test_output_past_2_31(lib, extras):
    M, N, K = 70001, 33000, 16  # y of 2.3e9 values
    x, w = _ints(M, K), _ints(N, K)
    y = torch.empty((M, N), dtype=BF16, device="cuda")
    res = _ints(M, N) if extras else None
    pre = torch.empty_like(y) if extras else None
    lib.ts_linear(x, w, y, act="relu", residual=res, preact=pre)
    lib.ts_sync_and_check()
    for rows in (slice(0, 3), slice(65534, 65538), slice(M - 3, M)):
        z = x[rows].float() @ w.float().t()
        assert torch.equal(y[rows], (z.relu() + (res[rows].float() if extras else 0)).to(BF16))
        if extras:
            assert torch.equal(pre[rows], z.to(BF16))


@pytest.mark.parametrize("M", [3, 20])
def test_weights_past_2_31(lib, M):
    N, K = 300000, 8192  # w of 2.5e9 values
    x, w = _ints(M, K), _ints(N, K)
    y = torch.empty((M, N), device="cuda")
    lib.ts_linear(x, w, y)
    gz, gx = _ints(M, N), torch.empty((M, K), device="cuda")
    lib.ts_linear_grad_input(gz, w, gx)
    lib.ts_sync_and_check()
    for rows in (slice(0, 3), slice(262140, 262148), slice(N - 3, N)):
        assert torch.equal(y[:, rows], x.float() @ w[rows].float().t())
    want = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    for i in range(0, N, 50000):
        want += gz[:, i:i + 50000].double() @ w[i:i + 50000].double()
    # integers below 2^24: exact in fp32 in any order
    assert torch.equal(gx.double(), want)


def test_weight_gradient_past_2_31(lib):
    M, N, K = 64, 70000, 33000
    gz, x = _ints(M, N), _ints(M, K)
    gw = torch.empty((N, K), dtype=BF16, device="cuda")
    lib.ts_linear_grad_weight(gz, x, gw)
    lib.ts_sync_and_check()
    for rows in (slice(0, 3), slice(65534, 65538), slice(N - 3, N)):
        assert torch.equal(gw[rows], (gz[:, rows].float().t() @ x.float()).to(BF16))


def test_activation_gradient_past_2_31(lib):
    M, N = 70000, 33000
    gy, z = _ints(M, N), _ints(M, N)
    gz, gb = torch.empty((M, N), dtype=BF16, device="cuda"), torch.empty(N, device="cuda")
    lib.ts_act_grad(gy, z, gz, gb, act="relu")
    lib.ts_sync_and_check()
    for rows in (slice(0, 3), slice(65534, 65538), slice(M - 3, M)):
        assert torch.equal(gz[rows], torch.where(z[rows] > 0, gy[rows], torch.zeros_like(gy[rows])))
    for cols in (slice(0, 2), slice(N - 2, N)):
        assert torch.equal(gb[cols].double(), torch.where(z[:, cols] > 0, gy[:, cols], torch.zeros_like(gy[:, cols])).double().sum(0))


def test_orthogonalised_batch_past_2_31(lib):
    n, R, C = 36, 60, 1 << 20  # 2.3e9 values
    g = torch.randn((n, R, C), device="cuda", dtype=BF16)
    out = torch.empty_like(g)
    lib.ts_orthogonalise(g, out, steps=1)
    lib.ts_sync_and_check()
    for i in (0, n - 1):
        x = g[i].double()
        x = x / (x.norm() + 1e-7)
        A = x @ x.t()
        want = 3.4445 * x + (-4.7750 * A + 2.0315 * A @ A) @ x
        # X, A, b A + c A^2 are rounded to fp16 (2^-12 each, their sums at most 4 times their values here) and
        # the result to bf16 (2^-8)
        assert float((out[i].double() - want).norm()) <= (2.0 ** -8 + 2.0 ** -8) * float(want.norm())
