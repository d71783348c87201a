"""A linear layer's product for few tokens and many columns: more tiles than run at once."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("M", [1, 8, 9, 15, 16, 32, 33, 64])
@pytest.mark.parametrize("N,K,out", [(38911, 136, BF16), (50001, 72, F32), (40000, 320, BF16)])
def test_few_tokens_many_columns(lib, M, N, K, out):
    """Small integers: exact sums, and residual, bias and preact beside them."""
    g = torch.Generator("cuda").manual_seed(M + N)

    def ints(r, c, dtype=BF16):
        return torch.randint(-3, 4, (r, c), device="cuda", generator=g).to(dtype)

    x, w, bias, res = ints(M, K), ints(N, K), ints(1, N, F32)[0], ints(M, N, out)
    y, z = torch.empty((M, N), dtype=out, device="cuda"), torch.empty((M, N), dtype=out, device="cuda")
    lib.ts_linear(x, w, y, bias=bias, act="relu", residual=res, preact=z)
    lib.ts_sync_and_check()
    want = x.double() @ w.double().t() + bias.double()
    assert torch.equal(z, want.to(out))
    assert torch.equal(y, (want.relu() + res.double()).to(out))


@pytest.mark.parametrize("M", [9, 32, 60])
def test_input_gradient_of_few_tokens(lib, M):
    """The same forms with the weights read the other way around."""
    N, K = 120, 40016
    g = torch.Generator("cuda").manual_seed(M)
    gz = torch.randint(-3, 4, (M, N), device="cuda", generator=g).to(BF16)
    w = torch.randint(-3, 4, (N, K), device="cuda", generator=g).to(BF16)
    gx = torch.empty((M, K), device="cuda")
    lib.ts_linear_grad_input(gz, w, gx)
    lib.ts_sync_and_check()
    assert torch.equal(gx.double(), gz.double() @ w.double())
