"""ts_orthogonalise of matrices that run as a chain of launches: large, long and thin ones, and batches of them."""
import pytest
import torch

import test_orthogonalise_gpu as plain
from test_orthogonalise_gpu import BF16, F32, _check, _matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _bounded_norm(monkeypatch):
    """The reference's bound takes the largest singular value from a decomposition, minutes of them at these
    sizes.  Here it is bounded from above instead: s^64 is the largest eigenvalue of (X X^T)^32, which its
    Frobenius norm exceeds by n^(1/128) on s at most."""

    def norm(x, order):
        assert order == 2
        A = x @ x.t() if x.shape[0] <= x.shape[1] else x.t() @ x
        log = 0.0
        for _ in range(5):
            f = A.norm()
            if not f > 0:
                return f
            log = 2 * (log + float(f.log()))
            A = (A / f) @ (A / f)
        return torch.exp((log + A.norm().log()) / 64)

    monkeypatch.setattr(plain.torch.linalg, "matrix_norm", norm)


@pytest.mark.parametrize("R,C", [(2304, 1008), (2300, 1001), (1001, 2300), (2048, 2048), (20, 20000), (50, 30001), (30000, 50),
                                 (4097, 129)])
@pytest.mark.parametrize("dtype,extra", [(BF16, 0), (F32, 0), (BF16, 7)])
def test_long_and_large(lib, R, C, dtype, extra):
    g = _matrix(R, C, R + C, dtype, extra=extra)
    out = torch.full((R, C + extra), float("nan"), dtype=BF16, device="cuda")[:, :C]
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    _check(out, g, what=f"{R}x{C}")


@pytest.mark.parametrize("n,R,C", [(5, 419, 2259), (3, 1300, 1100), (40, 300, 500)])
def test_batches(lib, n, R, C):
    """A matrix that holds a NaN leaves the others alone, and a zero one stays zero."""
    g = _matrix(R, C, n, BF16, (n,))
    g[1] = 0
    g[2, 3, 4] = float("nan")
    out = torch.empty((n, R, C), dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    assert not out[1].any() and torch.isnan(out[2]).any()
    for i in range(n):
        if i not in (1, 2):
            _check(out[i], g[i], what=f"{i} of {n} {R}x{C}")
