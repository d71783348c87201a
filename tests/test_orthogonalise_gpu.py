"""ts_orthogonalise against its iteration in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
COEF = (3.4445, -4.7750, 2.0315)
U = 2.0 ** -12   # half a step of fp16, relative


def _reference(g, steps, coef=COEF, eps=1e-7):
    """The iteration on one matrix in 64 bits, and a bound of the kernels' error in the Frobenius norm.

    With E the error before a step: p is an odd polynomial of the singular values, so the step changes E by
    at most the largest |p'| on the singular values' range.  The step's own roundings to fp16: of X (already
    in E), of A (it enters b A + c A^2 with at most |b| + 2 |c| |A|), of b A + c A^2, and of the result; the
    accumulation in fp32 cuts at 23 bits (17 terms each time, on sums of magnitudes no larger than the
    Frobenius norms' product)."""
    a, b, c = coef
    x = g.double()
    x = x / (x.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    n = x.shape[0]
    err = U * float(x.norm())
    for _ in range(steps):
        A = x @ x.t()
        B = b * A + c * A @ A
        s = float(torch.linalg.matrix_norm(x, 2)) + err
        r = torch.linspace(0, s, 200, dtype=torch.float64)
        lip = float((a + 3 * b * r ** 2 + 5 * c * r ** 4).abs().max())
        cut = 17 * 2.0 ** -23 * -(-max(x.shape) // 16)
        y = a * x + B @ x
        own = ((U + cut) * float(A.norm()) * (abs(b) + 2 * abs(c) * s * s) + (U + cut) * float(B.norm())) * s
        err = lip * err + own + (U + cut) * float(y.norm())
        x = y
    x = x.t() if tall else x
    return x, err + 2.0 ** -8 * float(x.norm()) + 1e-30, n


def _check(out, g, steps=5, coef=COEF, eps=1e-7, what=""):
    want, bound, _ = _reference(g, steps, coef, eps)
    off = float((out.double() - want).norm())
    assert off <= bound, f"{what}: {off} past {bound} (of {float(want.norm())})"


def _matrix(R, C, seed, dtype=BF16, lead=(), extra=0, size=1e-3):
    g = torch.Generator("cuda").manual_seed(seed)
    u, v = torch.randn((*lead, R, 3), device="cuda", generator=g), torch.randn((*lead, 3, C), device="cuda", generator=g)
    t = torch.zeros((*lead, R, C + extra), dtype=dtype, device="cuda")[..., :C]
    t.copy_(size * (torch.randn((*lead, R, C), device="cuda", generator=g) + 0.5 * u @ v))
    return t


SIZES = [(1, 1), (1, 50), (50, 1), (8, 8), (33, 65), (64, 200), (128, 128), (129, 127), (200, 64), (300, 300), (256, 1000),
         (513, 640), (777, 130), (1024, 768)]


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("extra", [0, 3])
def test_sizes(lib, R, C, dtype, extra):
    g = _matrix(R, C, R * 1000 + C, dtype, extra=extra)
    out = torch.full((R, C + extra), float("nan"), dtype=BF16, device="cuda")[:, :C]
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    _check(out, g, what=f"{R}x{C}")


@pytest.mark.parametrize("steps", [0, 1, 2, 7])
@pytest.mark.parametrize("R,C", [(96, 130), (130, 96)])
def test_steps(lib, R, C, steps):
    g = _matrix(R, C, 3, F32)
    out = torch.empty((R, C), dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, out, steps=steps)
    lib.ts_sync_and_check()
    _check(out, g, steps)


@pytest.mark.parametrize("coef", [(2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)])
def test_coefficients(lib, coef):
    g = _matrix(160, 300, 4)
    out = torch.empty((160, 300), dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, out, steps=6, coefficients=coef)
    lib.ts_sync_and_check()
    _check(out, g, 6, coef)


@pytest.mark.parametrize("R,C", [(64, 64), (200, 136), (136, 200), (65, 33)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batch(lib, R, C, dtype):
    """Each matrix by itself, whatever its neighbours hold; matrices apart and rows strided."""
    n = 5
    g = torch.zeros((n, R + 1, C + 8), dtype=dtype, device="cuda")[:, :R, :C]
    g.copy_(_matrix(R, C, 6, dtype, (n,)))
    g[1] *= 1000
    g[2] = 0
    g[3, 1, 2] = float("nan")
    keep = torch.full((n, R + 2, C + 8), 7.0, dtype=BF16, device="cuda")
    out = keep[:, :R, :C]
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    for i in (0, 1, 4):
        _check(out[i], g[i], what=f"matrix {i}")
        single = torch.empty((R, C), dtype=BF16, device="cuda")
        lib.ts_orthogonalise(g[i], single)
        lib.ts_sync_and_check()
        assert float((single.double() - out[i].double()).norm()) <= 2.0 ** -7 * float(single.double().norm())
    assert not out[2].any()
    assert torch.isnan(out[3]).any()
    assert (keep[:, R:] == 7).all() and (keep[:, :, C:] == 7).all()


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-3, 1e20, 1e30, 3e37])
def test_magnitudes(lib, size):
    """Squares that leave fp32's range do not matter."""
    g = _matrix(96, 160, 8, F32, size=1.0)
    g = g / g.abs().max() * size
    out = torch.empty((96, 160), dtype=BF16, device="cuda")
    eps = 1e-30 if size < 1e-20 else 1e-7
    if size == 1e-38:
        eps = 1e-42
    if size == 1e-20:
        eps = 1e-25
    lib.ts_orthogonalise(g, out, eps=eps)
    lib.ts_sync_and_check()
    _check(out, g, eps=float(torch.tensor(eps, dtype=F32)))


def test_singular_values(lib):
    """The result's singular values lie where five steps of the polynomial put them."""
    g = _matrix(256, 512, 12)
    out = torch.empty((256, 512), dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    s = torch.linalg.svdvals(g.double())
    s = s / g.double().norm()
    for _ in range(5):
        s = COEF[0] * s + COEF[1] * s ** 3 + COEF[2] * s ** 5
    got = torch.linalg.svdvals(out.double())
    bound = _reference(g, 5)[1]
    assert float((got.sort().values - s.sort().values).abs().max()) <= bound


def test_same_on_every_run_and_in_a_graph(lib):
    g = _matrix(300, 500, 14)
    first, out = (torch.empty((300, 500), dtype=BF16, device="cuda") for _ in range(2))
    lib.ts_orthogonalise(g, first)
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        lib.ts_orthogonalise(g, out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        lib.ts_sync_and_check()
        assert torch.equal(first, out)
    g.mul_(-1)
    graph.replay()
    lib.ts_sync_and_check()
    assert torch.equal(out, -first)
