"""Edges of a linear layer's operators: strides, neighbours in memory, streams and graphs, waits that run out, a step."""
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _gen(*key):
    return torch.Generator("cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _ints(r, c, g, dtype=BF16, lo=-3, hi=4):
    return torch.randint(lo, hi, (r, c), device="cuda", generator=g).to(dtype)


def _window(r, c, dtype, top, left, right):
    """A matrix inside a larger one of sevens, and that one."""
    big = torch.full((r + top + 2, left + c + right), 7.0, dtype=dtype, device="cuda")
    return big[top:top + r, left:left + c], big


def _untouched(big, r, c, top, left):
    keep = big.clone()
    keep[top:top + r, left:left + c] = 7
    return bool((keep == 7).all())


# (M, N, K): few tokens; tokens as columns; a cluster's shared K; persistent tiles, narrow and wide
FORMS = [(3, 70, 200), (30, 300, 520), (60, 200, 640), (150, 200, 900), (700, 1500, 320), (1000, 2000, 1100)]


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("left,right", [(0, 0), (8, 8), (3, 2), (1, 0)])
def test_windows(lib, M, N, K, out, left, right):
    """Operands and outputs that are parts of larger matrices, whose rest is neither used nor written."""
    g = _gen(M, N, K, left)
    x, w = (_window(r, K, BF16, 1, 8, 8 + (-K) % 8)[0] for r in (M, N))
    x.copy_(_ints(M, K, g))
    w.copy_(_ints(N, K, g))
    (y, by), (z, bz), (res, _) = (_window(M, N, out, 2, left, right) for _ in range(3))
    res.copy_(_ints(M, N, g, out))
    bias = _ints(1, N, g, F32)[0]
    lib.ts_linear(x, w, y, bias=bias, act="relu", residual=res, preact=z)
    lib.ts_sync_and_check()
    want = x.double() @ w.double().t() + bias.double()
    assert torch.equal(y, (want.relu() + res.double()).to(out)) and torch.equal(z, want.to(out))
    assert _untouched(by, M, N, 2, left) and _untouched(bz, M, N, 2, left)
    # the gradients of the same layer, into windows of windows
    gz, _ = _window(M, N, BF16, 1, 8, 8 + (-N) % 8)
    gz.copy_(_ints(M, N, g))
    (gx, bx), (gw, bw) = _window(M, K, out, 2, left, right), _window(N, K, out, 2, left, right)
    lib.ts_linear_grad_input(gz, w, gx)
    lib.ts_linear_grad_weight(gz, x, gw)
    lib.ts_sync_and_check()
    assert torch.equal(gx, (gz.double() @ w.double()).to(out)) and _untouched(bx, M, K, 2, left)
    assert torch.equal(gw, (gz.double().t() @ x.double()).to(out)) and _untouched(bw, N, K, 2, left)


@pytest.mark.parametrize("M,N,K", FORMS)
def test_nan_beside_the_operands(lib, M, N, K):
    """What lies between and behind the rows of the operands is not multiplied, not even by zero."""
    K -= 3
    g = _gen(M, N, K)
    x, w = (torch.full((r, -(-K // 8) * 8 + 8), float("nan"), dtype=BF16, device="cuda")[:, :K] for r in (M, N))
    x.copy_(_ints(M, K, g))
    w.copy_(_ints(N, K, g))
    y = torch.empty((M, N), device="cuda")
    lib.ts_linear(x, w, y)
    lib.ts_sync_and_check()
    assert torch.equal(y.double(), x.double() @ w.double().t())
    gz = torch.full((M, -(-N // 8) * 8 + 8), float("nan"), dtype=BF16, device="cuda")[:, :N]
    gz.copy_(_ints(M, N, g))
    gx, gw = torch.empty((M, K), device="cuda"), torch.empty((N, K), device="cuda")
    lib.ts_linear_grad_input(gz, w, gx)
    lib.ts_linear_grad_weight(gz, x, gw)
    lib.ts_sync_and_check()
    assert torch.equal(gx.double(), gz.double() @ w.double())
    assert torch.equal(gw.double(), gz.double().t() @ x.double())


@pytest.mark.parametrize("M,N,K", FORMS)
def test_same_on_every_run(lib, M, N, K):
    g = _gen(M, N, K, 1)
    x, w = (torch.randn((r, -(-K // 8) * 8), device="cuda", generator=g).to(BF16)[:, :K] for r in (M, N))
    a, b = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    lib.ts_linear(x, w, a, act="gelu")
    for _ in range(5):
        lib.ts_linear(x, w, b, act="gelu")
        lib.ts_sync_and_check()
        assert torch.equal(a, b)


def test_captured_and_replayed(lib):
    g = _gen(3)
    jobs = []
    for M, N, K in FORMS:
        K = -(-K // 8) * 8
        N = -(-N // 8) * 8
        x, w = _ints(M, K, g), _ints(N, K, g)
        jobs.append((x, w, torch.empty((M, N), device="cuda"), torch.empty((M, K), device="cuda"),
                     torch.empty((N, K), device="cuda"), _ints(M, N, g), torch.empty(N, device="cuda")))

    def calls():
        for x, w, y, gx, gw, gz, gb in jobs:
            lib.ts_linear(x, w, y)
            lib.ts_act_grad(gz, None, None, grad_bias=gb)
            lib.ts_linear_grad_input(gz, w, gx)
            lib.ts_linear_grad_weight(gz, x, gw)

    calls()
    lib.ts_sync_and_check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for turn in range(3):
        for x, w, y, gx, gw, gz, gb in jobs:
            for t in (x, w, gz):
                t.copy_(_ints(*t.shape, g))
            for t in (y, gx, gw):
                t.fill_(float("nan"))
        graph.replay()
        lib.ts_sync_and_check()
        for x, w, y, gx, gw, gz, gb in jobs:
            assert torch.equal(y.double(), x.double() @ w.double().t())
            assert torch.equal(gx.double(), gz.double() @ w.double())
            assert torch.equal(gw.double(), gz.double().t() @ x.double())
            assert torch.equal(gb.double(), gz.double().sum(0))


def test_two_streams_at_once(lib):
    """Calls of all forms on two streams that may overlap, each with its inputs written on its own stream."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    g = _gen(5)
    work = []
    for s in streams:
        jobs = [(_ints(M, -(-K // 8) * 8, g), _ints(N, -(-K // 8) * 8, g), torch.empty((M, N), device="cuda"))
                for M, N, K in FORMS]
        m = torch.randn((120, 200), device="cuda", generator=g)
        work.append((jobs, m, torch.empty((120, 200), dtype=BF16, device="cuda"),
                     torch.randn((1100, 1300), device="cuda", generator=g), torch.empty((1100, 1300), dtype=BF16, device="cuda")))
    want = []
    for jobs, m, mo, big, bo in work:
        lib.ts_orthogonalise(m, mo)
        lib.ts_orthogonalise(big, bo)
        lib.ts_sync_and_check()
        want.append((mo.clone(), bo.clone()))
        mo.zero_(), bo.zero_()
    torch.cuda.synchronize()
    for turn in range(4):
        for s, (jobs, m, mo, big, bo) in zip(streams, work):
            for x, w, y in jobs:
                lib.ts_linear(x, w, y, stream=s)
            lib.ts_orthogonalise(m, mo, stream=s)
            lib.ts_orthogonalise(big, bo, stream=s)
    for s in streams:
        lib.ts_sync_and_check(s)
    for (jobs, m, mo, big, bo), (m_want, b_want) in zip(work, want):
        for x, w, y in jobs:
            assert torch.equal(y.double(), x.double() @ w.double().t())
        assert torch.equal(mo, m_want) and torch.equal(bo, b_want)


def test_two_graphs_at_once(lib):
    """Graphs of orthogonalised updates hold workspaces of their own."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    g = _gen(7)
    made = []
    for size in ((100, 180), (100, 180), (1100, 1300), (1100, 1300)):
        m, o = torch.randn(size, device="cuda", generator=g), torch.empty(size, dtype=BF16, device="cuda")
        lib.ts_orthogonalise(m, o)
        lib.ts_sync_and_check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.ts_orthogonalise(m, o)
        made.append((graph, o, o.clone(), m))  # a graph reads m where it lay when it was captured
    torch.cuda.synchronize()
    for turn in range(3):
        for i, (graph, o, _, _) in enumerate(made):
            with torch.cuda.stream(streams[i % 2]):
                o.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, o, want, _ in made:
            assert torch.equal(o, want)


@pytest.mark.parametrize("M,N,K,runs_out", [(40, 2048, 8192, False), (256, 256, 8192, False), (2048, 2048, 8192, True)])
def test_waits_that_run_out_are_reported(lib, M, N, K, runs_out):
    """A limit far below the time that the first data takes: a status, and a context that works afterwards.

    A poll of a barrier may suspend for longer than the whole of a short wait, which then ends unnoticed
    and the result is right; the epilogue of a persistent tile waits for a K loop, and notices."""
    g = _gen(M)
    x, w, y = _ints(M, K, g), _ints(N, K, g), torch.empty((M, N), device="cuda")
    lib.ts_linear(x, w, y, timeout_s=1e-9)
    try:
        lib.ts_sync_and_check()
        assert not runs_out
        assert torch.equal(y.double(), x.double() @ w.double().t())
    except lib.TsError as e:
        assert e.status == lib.TS_ERR_TIMEOUT
    lib.ts_sync_and_check()
    lib.ts_linear(x, w, y)
    lib.ts_sync_and_check()
    assert torch.equal(y.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("size", [(300, 500), (1500, 3000)])
def test_orthogonalisation_whose_waits_run_out(lib, size):
    g = torch.randn(size, device="cuda", generator=_gen(size))
    want, out = (torch.empty(size, dtype=BF16, device="cuda") for _ in range(2))
    lib.ts_orthogonalise(g, want)
    lib.ts_sync_and_check()
    lib.ts_orthogonalise(g, out, timeout_s=1e-9)
    with pytest.raises(lib.TsError) as e:
        lib.ts_sync_and_check()
    assert e.value.status == lib.TS_ERR_TIMEOUT
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    assert torch.equal(out, want)


def test_refusals_of_the_binding(lib, monkeypatch):
    x, w, y = (torch.zeros(s, dtype=BF16, device="cuda") for s in ((4, 16), (8, 16), (4, 8)))
    f = torch.zeros((4, 8), device="cuda")
    for bad in (lambda: lib.ts_linear(x, w, y.t()), lambda: lib.ts_linear(x[:, ::2], w[:, ::2], y),
                lambda: lib.ts_linear(x, w[:, :8], y), lambda: lib.ts_linear(x[:1].expand(4, 16), w, y),
                lambda: lib.ts_linear(x, w, y, bias=torch.zeros(7, device="cuda")),
                lambda: lib.ts_linear(x, w, y, residual=y[:3]),
                lambda: lib.ts_linear(x, w, torch.zeros((1, 8), dtype=BF16, device="cuda").expand(4, 8)),
                lambda: lib.ts_linear_grad_input(y, w, y), lambda: lib.ts_linear_grad_weight(y, x, y),
                lambda: lib.ts_act_grad(f, f[:2], f, act="relu"), lambda: lib.ts_act_grad(f, None, None, torch.zeros(4, device="cuda")),
                lambda: lib.ts_orthogonalise(x, x[:2]), lambda: lib.ts_orthogonalise(x, torch.empty_like(x), steps=-1),
                lambda: lib.ts_orthogonalise(x, torch.empty_like(x), eps=0.0),
                lambda: lib.ts_orthogonalise(x, torch.empty_like(x), coefficients=(0, 0, 0)),
                lambda: lib.ts_orthogonalise(x[None].expand(3, 4, 16), torch.empty((3, 4, 16), dtype=BF16, device="cuda")),
                lambda: lib.ts_orthogonalise(x, torch.empty_like(x)[:, :8])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.ts_linear(x.float(), w, y), lambda: lib.ts_linear(x, w, y.half()),
                lambda: lib.ts_linear(x, w, y, residual=f), lambda: lib.ts_linear(x, w, f, preact=y),
                lambda: lib.ts_linear(x, w, y, bias=torch.zeros(8, device="cuda").half()),
                lambda: lib.ts_linear_grad_weight(y, x, torch.zeros((8, 16), device="cuda"), base=w),
                lambda: lib.ts_act_grad(f, y, f, act="relu"), lambda: lib.ts_orthogonalise(x, x.float()),
                lambda: lib.ts_orthogonalise(x, torch.empty_like(x), workspace=torch.zeros(8))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lib.ts_linear(x, w, y, residual=y, preact=y), lambda: lib.ts_linear(x, x, x[:, :4]),
                lambda: lib.ts_orthogonalise(x, x), lambda: lib.ts_act_grad(f, None, f, act="relu"),
                lambda: lib.ts_linear_grad_input(y, w, x.clone(), act="relu"),
                lambda: lib.ts_orthogonalise(x, torch.empty_like(x), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(lib.TsError) as e:
            bad()
        assert e.value.status == lib.TS_ERR_INVALID_ARG
    with pytest.raises(KeyError):
        lib.ts_linear(x, w, y, act="mish")
    # tensors of another device than the current one
    monkeypatch.setattr(lib, "_raw_device", lambda: 1)
    for bad in (lambda: lib.ts_linear(x, w, y), lambda: lib.ts_linear_grad_input(y, w, x), lambda: lib.ts_linear_grad_weight(y, x, w),
                lambda: lib.ts_act_grad(f, None, f), lambda: lib.ts_orthogonalise(x, torch.empty_like(x))):
        with pytest.raises(ValueError, match="current device"):
            bad()
    monkeypatch.undo()
    lib.ts_sync_and_check()


def test_workspace_that_is_passed(lib):
    g = torch.randn((3, 200, 130), device="cuda", generator=_gen(9))
    a, b = (torch.empty(g.shape, dtype=BF16, device="cuda") for _ in range(2))
    lib.ts_orthogonalise(g, a)
    need = lib.ts_orthogonalise_workspace(3, 200, 130)
    ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    lib.ts_orthogonalise(g, b, workspace=ws[:need])
    lib.ts_sync_and_check()
    assert torch.equal(a, b) and bool((ws[need:] == 0xAB).all())


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_training_step(lib, act):
    """A residual block of two layers: forward, backward and the orthogonalised updates, one call after another."""
    T, D, H = 300, 256, 640
    g = _gen(act)
    x = torch.randn((T, D), device="cuda", generator=g).to(BF16)
    w1, w2 = (torch.randn(s, device="cuda", generator=g).mul_(s[1] ** -0.5).to(BF16) for s in ((H, D), (D, H)))
    b1, b2 = (0.1 * torch.randn(n, device="cuda", generator=g) for n in (H, D))
    gy = torch.randn((T, D), device="cuda", generator=g).to(BF16)
    new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    z, h, y = new(T, H), new(T, H), new(T, D)
    lib.ts_linear(x, w1, h, bias=b1, act=act, preact=z)
    lib.ts_linear(h, w2, y, bias=b2, residual=x)
    gb2, gw2, gz, gb1, gw1, gx = new(D, dtype=F32), new(D, H, dtype=F32), new(T, H), new(H, dtype=F32), new(H, D, dtype=F32), new(T, D)
    lib.ts_act_grad(gy, None, None, gb2)
    lib.ts_linear_grad_weight(gy, h, gw2)
    lib.ts_linear_grad_input(gy, w2, gz, act=act, preact=z)
    lib.ts_act_grad(gz, None, None, gb1)
    lib.ts_linear_grad_weight(gz, x, gw1)
    lib.ts_linear_grad_input(gz, w1, gx)
    u1, u2 = new(H, D), new(D, H)
    lib.ts_orthogonalise(gw1, u1)
    lib.ts_orthogonalise(gw2, u2)
    lib.ts_sync_and_check()

    d = torch.float64
    F = torch.nn.functional
    leaves = [t.to(d).requires_grad_() for t in (x, w1, b1, w2, b2)]
    X, W1, B1, W2, B2 = leaves
    Z = X @ W1.t() + B1
    A = {"gelu": F.gelu, "silu": F.silu, "relu": F.relu}[act](Z)
    Y = A @ W2.t() + B2 + X
    Y.backward(gy.to(d))
    # Relative errors in the Frobenius norm.  A rounding to bf16 is off by at most 2^-8 of each value, so by that
    # much of the norm; a product passes its operands' roundings on (times at most 4 here: the operands' own
    # norms against the product's, for these well-conditioned Gaussian matrices).  z, h, gz and the outputs
    # are rounded; at a relu's corner z's rounding may also switch a slope: |z| < 2^-8 |z| cannot, so none.
    u = 2.0 ** -8

    def close(got, want, roundings, what):
        off = float((got.to(d) - want).norm() / want.norm())
        assert off <= roundings * 4 * u, f"{what}: {off}"

    close(y, Y.detach(), 2, "y")
    close(gw2, W2.grad, 1, "grad_w2")
    close(gb2, B2.grad, 1, "grad_b2")
    close(gw1, W1.grad, 2, "grad_w1")
    close(gb1, B1.grad, 2, "grad_b1")
    close(gx, X.grad - gy.to(d), 3, "grad_x")
    for u_, gw in ((u1, gw1), (u2, gw2)):
        s = torch.linalg.svdvals(gw.to(d))
        s = s / s.square().sum().sqrt()
        for _ in range(5):
            s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
        got = torch.linalg.svdvals(u_.to(d))
        assert float((got.sort().values - s.sort().values).abs().max()) < 0.05
