"""The norm of an orthogonalised matrix over fp32's whole range, in both forms of ts_orthogonalise.

With no steps the result is the normalised matrix itself.  A norm is the root of a sum of squares of n values in fp32:
each square and each of the sums' levels rounds by at most 2^-24 of the sum so far.  A thread adds up at most 2^9 of
them here and the partial sums join in another 2^6, so the sum is off by 2^-24 * (2^9 + 2^6 + 1) < 2^-14 of itself and
the norm by half of that; the factors round a few times more.  An entry is off by that, 2^-14, and its rounding to bf16
by 2^-8 of itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TOL = 2.0 ** -8 + 2.0 ** -13


def _normal(R, C, seed, clip=3.2):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn((R, C), device="cuda", generator=g).clamp_(-clip, clip)


def _normalised(lib, g, eps=1e-7):
    out = torch.empty(g.shape, dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, out, steps=0, eps=eps)
    lib.ts_sync_and_check()
    return out.double()


def _check(lib, g, eps=1e-7):
    want = g.double() / (g.double().norm() + float(torch.tensor(eps, dtype=F32)))
    got = _normalised(lib, g, eps)
    # bf16's least normal value is 2^-126; below it a rounding is off by at most 2^-134
    assert bool(((got - want).abs() <= TOL * want.abs() + 2.0 ** -133).all())


@pytest.mark.parametrize("size", [1e-30, 1e-10, 1.0, 2.0 ** 30, 1e9, 3e9, 1e14, 5e15, 1e16, 2e16, 5e18, 1e19, 1e25, 1e37, 1e38])
@pytest.mark.parametrize("R,C", [(96, 160), (2048, 2048), (4096, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sizes(lib, size, R, C, dtype):
    """Where the squares, or their sum, pass fp32's range."""
    g = (_normal(R, C, 1) * size).to(dtype)
    _check(lib, g, 1e-35 if size < 1e-20 else 1e-7)


@pytest.mark.parametrize("base,outlier", [(5e15, 1.2e18), (1e16, 2.0 ** 60.2), (1e9, 1e19), (1e9, 1e25), (1.0, 3e38), (1e18, 3e38)])
def test_outlier(lib, base, outlier):
    """One value far above the others, in a share of its own."""
    for R, C in ((1024, 1024), (2048, 2048)):
        g = _normal(R, C, 2) * base
        g[3, 4] = outlier
        _check(lib, g)


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1e-30, 1e-7, 1.0, 1e12, 3e38])
@pytest.mark.parametrize("size", [0.0, 1e-45, 1e-42, 1e-38, 1e-32, 1e-25, 1e-20, 1e-10, 1e10, 1e30, 3e38])
def test_eps(lib, size, eps):
    """Norms above, about and below eps, from fp32's least value to its largest."""
    g = _normal(64, 96, 3, 1.0) * size if size else torch.zeros((64, 96), device="cuda")
    _check(lib, g, eps)


@pytest.mark.parametrize("steps", [0, 5])
@pytest.mark.parametrize("R,C", [(64, 96), (300, 500), (2048, 1024)])
@pytest.mark.parametrize("beside", [1.0, 1e17, 1e30, float("inf")])
def test_nan_beside_large_values(lib, R, C, beside, steps):
    """A matrix that holds a NaN gives NaNs, whatever else it holds."""
    g = _normal(R, C, 4)
    g[0, 0] = float("nan")
    g[R - 1, C - 1] = beside
    out = torch.empty((R, C), dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, out, steps=steps)
    lib.ts_sync_and_check()
    assert bool(torch.isnan(out).all())


@pytest.mark.parametrize("size", [1e-20, 1e10, 5e15, 1e16, 2e16, 1e19, 1e38])
@pytest.mark.parametrize("R,C", [(300, 500), (4096, 4096)])
def test_update_does_not_depend_on_the_size(lib, size, R, C):
    """Five steps from the same matrix times a power of two: the same update, by one launch and by a chain."""
    g = _normal(R, C, 5)
    scale = 2.0 ** round(torch.log2(torch.tensor(size, dtype=torch.float64)).item())
    scale = min(scale, 2.0 ** 126)
    want, got = (torch.empty((R, C), dtype=BF16, device="cuda") for _ in range(2))
    lib.ts_orthogonalise(g, want, eps=1e-35)
    lib.ts_orthogonalise(g * scale, got, eps=1e-35)
    lib.ts_sync_and_check()
    # the factors' roundings apart (2^-14 of X, which five steps raise by 3.4445^5 at most for its smallest singular
    # values), both round alike: 2^-7 is twice an output's rounding
    assert float((got.double() - want.double()).norm()) <= 2.0 ** -7 * float(want.double().norm())
    assert float(want.double().norm()) > 0.7 * min(R, C) ** 0.5
