"""A linear layer's operators at the largest sizes that they take, 2^31 - 512, and with row strides past 2^32.

Inputs are zeros but for some integers at the ends, about powers of two and at random places, so that every sum is
exact and what an offset that wrapped would read or write shows."""
import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

BF16, F32 = torch.bfloat16, torch.float32
MOST = 2 ** 31 - 512


@pytest.fixture(autouse=True)
def _memory():
    """Tens of GB each: given back before and after."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _places(n, seed=0):
    """Where values lie along an axis of n: its ends, about the powers of two, and some others."""
    g = torch.Generator().manual_seed(seed)
    p = [0, 1, 2, 7, 8, 9, n - 1, n - 2, n - 8, n - 9, n - 33, n - 64, n - 129, n // 2, n // 2 + 1]
    p += [2 ** k + d for k in range(24, 31) for d in (-1, 0, 1)]
    return torch.tensor(sorted({i for i in p if 0 <= i < n} | set(torch.randint(0, n, (200,), generator=g).tolist())), device="cuda")


def _values(r, c, seed=1):
    g = torch.Generator("cuda").manual_seed(seed)
    v = torch.randint(1, 4, (r, c), device="cuda", generator=g) * (2 * torch.randint(0, 2, (r, c), device="cuda", generator=g) - 1)
    return v.to(BF16)


def _elsewhere_zero(t, places, dim):
    """All values of t outside of `places` along dim are zero."""
    t.index_fill_(dim, places, 0)
    return not bool(t.any())


@pytest.mark.parametrize("M,N", [(1, 1), (2, 3)])
@pytest.mark.parametrize("K", [MOST, MOST - 511])
def test_few_tokens_of_the_longest_rows(lib, M, N, K):
    at = _places(K)
    x, w = (torch.zeros((r, -(-K // 8) * 8), dtype=BF16, device="cuda")[:, :K] for r in (M, N))
    x[:, at], w[:, at] = _values(M, len(at)), _values(N, len(at), 2)
    y = torch.empty((M, N), device="cuda")
    lib.ts_linear(x, w, y)
    lib.ts_sync_and_check()
    assert torch.equal(y.double(), x[:, at].double() @ w[:, at].double().t())


@pytest.mark.parametrize("tile", ["auto", "128x128", "128x256", "256x256"])
def test_most_rows(lib, tile):
    M, N, K = MOST, 1, 8
    at = _places(M)
    x, w = torch.zeros((M, K), dtype=BF16, device="cuda"), _values(N, K)
    x[at] = _values(len(at), K, 2)
    y = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    lib.ts_linear(x, w, y, act="relu", tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(y[at].double(), (x[at].double() @ w.double().t()).relu())
    assert _elsewhere_zero(y, at, 0)


@pytest.mark.parametrize("M,tile", [(1, "auto"), (1, "128x128"), (1, "128x256"), (1, "256x256"), (9, "auto")])
def test_most_columns(lib, M, tile):
    """With a bias and a residual: every offset along the columns."""
    N, K = MOST, 8
    at = _places(N)
    x, w = _values(M, K), torch.zeros((N, K), dtype=BF16, device="cuda")
    w[at] = _values(len(at), K, 2)
    bias = torch.zeros(N, dtype=BF16, device="cuda")
    bias[at] = _values(1, len(at), 3)[0]
    y = torch.zeros((M, N), dtype=BF16, device="cuda")
    y[:, at] = _values(M, len(at), 4)
    want = (x.double() @ w[at].double().t() + bias[at].double()).relu() + y[:, at].double()
    lib.ts_linear(x, w, y, bias=bias, act="relu", residual=y, tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(y[:, at].double(), want)
    assert _elsewhere_zero(y, at, 1)


@pytest.mark.parametrize("M", [1, 9, 70])
def test_strides_past_2_32(lib, M):
    """Two rows of w, and M rows of one value each, far apart."""
    far = 2 ** 32 + 8
    buf = torch.zeros(far + 4096, dtype=BF16, device="cuda")
    N, K = 2, 1000
    w = torch.as_strided(buf, (N, K), (far, 1))
    w.copy_(_values(N, K))
    x = _values(M, K, 2)
    y = torch.empty((M, N), device="cuda")
    lib.ts_linear(x, w, y, tile="auto")
    lib.ts_sync_and_check()
    assert torch.equal(y.double(), x.double() @ w.double().t())
    gz, gx = _values(M, 8, 3)[:, :N], torch.empty((M, K), device="cuda")
    lib.ts_linear_grad_input(gz, w, gx)
    lib.ts_sync_and_check()
    assert torch.equal(gx.double(), gz.double() @ w.double())


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("rows", [2, 3])
def test_outputs_with_strides_past_2_32(lib, rows, odd):
    far, N, K = 2 ** 32 + 8 + odd, 500, 64
    x, w = _values(rows, K), _values(N, K, 2)
    want = x.double() @ w.double().t()
    for tile in ("auto", "128x128", "128x256", "256x256"):
        buf = torch.zeros((rows - 1) * far + N, dtype=BF16, device="cuda")
        y = torch.as_strided(buf, (rows, N), (far, 1))
        y.copy_(_values(rows, N, 3))
        kept = y.double()
        lib.ts_linear(x, w, y, residual=y, tile=tile)
        lib.ts_sync_and_check()
        assert torch.equal(y, (want + kept).to(BF16))
        y.zero_()
        assert not bool(buf.any())
        del buf, y
        torch.cuda.empty_cache()
    buf = torch.zeros((rows - 1) * far + N, dtype=BF16, device="cuda")
    gy = torch.as_strided(buf, (rows, N), (far, 1))
    gy.copy_(_values(rows, N, 3))
    # gy as its own pre-activation: relu's slope is 1 where it is above 0
    want, gb = gy.double(), torch.empty(N, device="cuda")
    lib.ts_act_grad(gy, gy, gy, gb, act="relu")
    lib.ts_sync_and_check()
    assert torch.equal(gy.double(), want.relu()) and torch.equal(gb.double(), want.relu().sum(0))


@pytest.mark.parametrize("tile", ["auto", "128x128"])
def test_longest_sum(lib, tile):
    """K loops of some seconds by one CTA, with the default limit of a wait."""
    M, N = MOST, 8
    at = _places(M)
    x, gw = torch.zeros((M, N), dtype=BF16, device="cuda"), torch.empty((N, N), device="cuda")
    x[at] = _values(len(at), N)
    lib.ts_linear_grad_weight(x, x, gw, tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(gw.double(), x[at].double().t() @ x[at].double())


def test_longest_rows_of_nine_tokens(lib):
    M, N, K = 9, 1, MOST
    at = _places(K)
    x, w = (torch.zeros((r, K), dtype=BF16, device="cuda") for r in (M, N))
    x[:, at], w[:, at] = _values(M, len(at)), _values(N, len(at), 2)
    y = torch.empty((M, N), device="cuda")
    lib.ts_linear(x, w, y)
    lib.ts_sync_and_check()
    assert torch.equal(y.double(), x[:, at].double() @ w[:, at].double().t())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_activation_gradient_of_most_columns(lib, dtype, act):
    N = MOST
    at = _places(N)
    gy = torch.zeros((1, N), dtype=dtype, device="cuda")
    gy[:, at] = _values(1, len(at)).to(dtype)
    gb = torch.full((N,), 7.0, device="cuda")
    want = gy[0, at].double()
    if act == "relu":
        want = want.relu()
        lib.ts_act_grad(gy, gy, gy, gb, act=act)
    else:
        lib.ts_act_grad(gy, None, None, gb)
    lib.ts_sync_and_check()
    assert torch.equal(gb[at].double(), want) and torch.equal(gy[0, at].double(), want)
    assert _elsewhere_zero(gb, at, 0) and _elsewhere_zero(gy, at, 1)


@pytest.mark.parametrize("N", [1, 8])
def test_activation_gradient_of_most_rows(lib, N):
    M = MOST
    at = _places(M)
    gy = torch.zeros((M, N), dtype=BF16, device="cuda")
    gy[at] = _values(len(at), N)
    gb = torch.empty(N, device="cuda")
    want = gy[at].double().relu()
    lib.ts_act_grad(gy, gy, gy, gb, act="relu")
    lib.ts_sync_and_check()
    assert torch.equal(gb.double(), want.sum(0)) and torch.equal(gy[at].double(), want)
    assert _elsewhere_zero(gy, at, 0)
