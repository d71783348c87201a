"""ts_orthogonalise at its default five steps, and at others, held to the accuracy it states (orth_accuracy)."""
import pytest
import torch

from orth_accuracy import COEF, WHOLE, check, errors, iterate, matrix

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# one launch, and a chain of them: squares, wide and tall ones, odd ones, sizes off tiles and boxes
ONE = [(1, 1), (1, 50), (50, 1), (8, 8), (33, 65), (64, 200), (128, 128), (129, 127), (200, 64), (300, 300), (256, 1000), (513, 640),
       (777, 130), (1024, 768), (1000, 1001)]
CHAIN = [(2304, 1008), (2300, 1001), (1001, 2300), (2048, 2048), (20, 20000), (50, 30001), (30000, 50), (4097, 129), (129, 4097),
         (1537, 3001)]


def _run(lib, g, **kw):
    """The update of g, written into a wider matrix whose rest stays as it is."""
    *lead, R, C = g.shape
    extra = kw.pop("extra", 0)
    keep = torch.full((*lead, R + 1, C + extra), 7.0, dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, keep[..., :R, :C], **kw)
    lib.ts_sync_and_check()
    assert bool((keep[..., R:, :] == 7).all()) and bool((keep[..., C:] == 7).all())
    return keep[..., :R, :C]


@pytest.mark.parametrize("R,C", ONE + CHAIN)
@pytest.mark.parametrize("dtype,extra", [(BF16, 0), (F32, 0), (BF16, 7), (F32, 8)])
def test_five_steps(lib, R, C, dtype, extra):
    g = matrix(R, C, R * 1000 + C, dtype, extra=extra, device="cuda")
    check(_run(lib, g, extra=extra), g, what=f"{R}x{C}")


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 4, 6, 7])
@pytest.mark.parametrize("R,C", [(96, 130), (130, 96), (600, 500), (2300, 1001), (1100, 2500)])
def test_steps(lib, R, C, steps):
    g = matrix(R, C, 3, F32, device="cuda")
    check(_run(lib, g, steps=steps), g, steps)


@pytest.mark.parametrize("coef", [(2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)])
@pytest.mark.parametrize("R,C", [(160, 300), (300, 160), (1100, 2500), (2304, 1008)])
def test_coefficients(lib, R, C, coef):
    g = matrix(R, C, 4, device="cuda")
    check(_run(lib, g, steps=6, coefficients=coef), g, 6, coef)


@pytest.mark.parametrize("n,R,C", [(5, 64, 64), (5, 200, 136), (5, 136, 200), (7, 65, 33), (4, 513, 640), (200, 40, 72), (5, 419, 2259),
                                   (4, 1300, 1100), (40, 300, 500), (4, 2050, 700)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batches(lib, n, R, C, dtype):
    """Each matrix by itself, whatever its neighbours hold."""
    g = torch.zeros((n, R + 1, C + 8), dtype=dtype, device="cuda")[:, :R, :C]
    g.copy_(matrix(R, C, n, dtype, (n,), device="cuda"))
    g[1] *= 1000
    g[2] = 0
    g[3, 1, 2] = float("nan")
    out = _run(lib, g, extra=8)
    for i in range(n):
        if i == 2:
            assert not out[i].any()
        elif i == 3:
            assert bool(torch.isnan(out[i]).all())
        elif i < 8 or i + 2 >= n:
            check(out[i], g[i], what=f"{i} of {n} {R}x{C}")


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-3, 1.0, 1e9, 1e16, 1e20, 1e30, 3e37])
@pytest.mark.parametrize("R,C", [(96, 160), (2048, 1500)])
def test_magnitudes(lib, size, R, C):
    """Squares that leave fp32's range do not matter."""
    g = matrix(R, C, 8, F32, size=1.0, device="cuda")
    g = g / g.abs().max() * size
    eps = 1e-7 if size > 1e-3 else size * 1e-4
    check(_run(lib, g, eps=eps), g, eps=float(torch.tensor(eps, dtype=F32)))


@pytest.mark.parametrize("R,C", [(256, 512), (1001, 2300)])
def test_singular_values(lib, R, C):
    """They lie where five steps of the polynomial put them: an error moves them by no more than its own size."""
    g = matrix(R, C, 12, device="cuda")
    s = torch.linalg.svdvals(g.double().cpu())
    s = s / g.double().norm().cpu()
    for _ in range(5):
        s = COEF[0] * s + COEF[1] * s ** 3 + COEF[2] * s ** 5
    got = torch.linalg.svdvals(_run(lib, g).double().cpu())
    # Weyl, and Hoffman and Wielandt: the differences' root of squares is at most the error's Frobenius norm
    assert float((got.sort().values - s.sort().values).norm()) <= WHOLE * float(s.norm())


@pytest.mark.parametrize("R,C", [(300, 500), (1100, 1300)])
def test_replayed_with_another_matrix(lib, R, C):
    g = matrix(R, C, 14, F32, device="cuda")
    out = torch.empty((R, C), dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.ts_orthogonalise(g, out)
    for seed in (15, 16):
        g.copy_(matrix(R, C, seed, F32, device="cuda"))
        out.zero_()
        graph.replay()
        lib.ts_sync_and_check()
        check(out, g)


def test_error_is_that_of_the_emulation(lib):
    """No more than the formats take: within a tenth of what rounding at the same places gives in 64 bits."""
    from orth_accuracy import emulated

    for R, C in ((300, 500), (2048, 1500)):
        g = matrix(R, C, 17, device="cuda")
        want = iterate(g)
        got, same = errors(_run(lib, g), want)[0], errors(emulated(g), want)[0]
        # the roundings of some 10^5 values and more: their sum of squares varies by far less than that
        assert 0.9 * same <= got <= 1.1 * same
