"""Options of ts_orthogonalise that would mean something else once they are in fp32."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("coef", [(0, 0, 0), (1e-50, 0.0, 0.0), (1e-60, -1e-50, 1e-46), (0.0, -0.0, 0.0)])
def test_coefficients_of_zero(lib, coef):
    """Not the default ones in their place."""
    g = torch.randn((8, 16), device="cuda")
    out = torch.zeros((8, 16), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="coefficients"):
        lib.ts_orthogonalise(g, out, coefficients=coef)
    lib.ts_sync_and_check()
    assert not out.any()


def test_least_coefficients(lib):
    """fp32's least value is not 0: X becomes 0 by it."""
    g = torch.randn((8, 16), device="cuda")
    out = torch.ones((8, 16), dtype=torch.bfloat16, device="cuda")
    lib.ts_orthogonalise(g, out, steps=1, coefficients=(2.0 ** -149, 0.0, 0.0))
    lib.ts_sync_and_check()
    assert float(out.float().abs().max()) <= 2.0 ** -133


@pytest.mark.parametrize("coef", [(float("nan"), 1.0, 1.0), (1.0, float("nan"), 0.0), (1.0, 1.0, float("inf"))])
def test_coefficients_that_are_not_finite(lib, coef):
    g = torch.randn((8, 16), device="cuda")
    out = torch.zeros((8, 16), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.TsError):
        lib.ts_orthogonalise(g, out, coefficients=coef)
    lib.ts_sync_and_check()
    assert not out.any()
