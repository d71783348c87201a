"""Residuals and pre-activations that TMA loads into staging buffers which plain stores have just left.

A subtile that N cuts off leaves by the lanes' own stores; the next tile's residual is loaded into the same buffer,
after all lanes have read it.  Many ragged tiles by few workers, residuals in place, one buffer (long K) and two."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _ints(g, *shape, dtype=BF16):
    return torch.randint(-3, 4, shape, device="cuda", generator=g).to(dtype)


@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("N", [8, 72, 136, 200, 264, 920])
@pytest.mark.parametrize("K", [64, 512, 1088])
@pytest.mark.parametrize("out", [BF16, F32])
def test_ragged_tiles_of_few_workers(lib, tile, N, K, out):
    g = torch.Generator("cuda").manual_seed(N * 10000 + K)
    M = 2200  # the last tile's rows end inside it
    x, w, res, z = _ints(g, M, K), _ints(g, N, K), _ints(g, M, N, dtype=out), _ints(g, M, N, dtype=out)
    want = x.double() @ w.double().t()
    for workers in (1, 3):
        y = res.clone()
        lib.ts_linear(x, w, y, act="relu", residual=y, tile=tile, max_workers=workers)
        gz = z.clone()
        lib.ts_linear_grad_input(x, w.t().contiguous(), gz, act="relu", preact=gz, tile=tile, max_workers=workers)
        lib.ts_sync_and_check()
        assert torch.equal(y, (want.relu() + res.double()).to(out))
        assert torch.equal(gz, (want * (z > 0)).to(out))
