"""Every tile's kernel with every activation: products of several tiles a worker, their residuals fetched ahead, in place too."""
import math

import pytest
import torch

from test_linear_gpu import ACTS, BF16, F32, HALF, SLOPE, _act, _close, _fill, _gen, _pitched, _slope, _sum_bound

pytestmark = pytest.mark.gpu

# one staging buffer and two (K above and below 1024), edges that vectors do and do not fill, one worker and several
CASES = [(300, 1100, 200, 2), (260, 530, 1100, 3), (1030, 776, 640, 0), (600, 1001, 130, 1)]


@pytest.mark.parametrize("M,N,K,workers", CASES)
@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
def test_forward(lib, M, N, K, workers, tile, out, act):
    g = _gen(M, N, K, tile, act)
    x, w = _fill(M, K, g, scale=1.5), _fill(N, K, g, scale=1 / math.sqrt(K))
    bias = torch.randn(N + 1, device="cuda", generator=g)[1:]  # off a 16-byte boundary
    bias = bias if K % 3 else bias.to(BF16)
    z = x.double() @ w.double().t() + bias.double()
    S = x.double().abs() @ w.double().abs().t() + bias.double().abs()
    err = _sum_bound(S, K)
    own = 2.0 ** -20 * (z.abs() + 1) if act not in ("none", "relu") else 0
    for pre, in_place in ((False, False), (False, True), (True, False), (True, True)):
        res = _fill(M, N, g, out)
        before = res.double()
        y = res if in_place else _pitched(M, N, out)
        keep = _pitched(M, N, out) if pre else None
        lib.ts_linear(x, w, y, bias=bias, act=act, residual=res, preact=keep, tile=tile, max_workers=workers)
        lib.ts_sync_and_check()
        want = _act(z, act) + before
        _close(y, want, SLOPE[act] * err + own + 2.0 ** -23 * (want.abs() + before.abs()) + 2 * HALF[out] * want.abs(), act)
        if pre:
            _close(keep, z, err + 2 * HALF[out] * z.abs(), f"preact {act}")


@pytest.mark.parametrize("M,N,K,workers", CASES)
@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act", ACTS[1:])
def test_backward(lib, M, N, K, workers, tile, out, act):
    """Through the activation before, into another matrix and over the pre-activations themselves (N and K swap)."""
    g = _gen(M, N, K, tile, act, 1)
    gz, w = _fill(M, K, g, scale=0.1), _fill(K, N, g)
    s = gz.double() @ w.double()
    S = gz.double().abs() @ w.double().abs()
    for in_place in (False, True):
        pre = _fill(M, N, g, out, scale=2.0)
        z = pre.double()
        slope = _slope(z, act)
        gx = pre if in_place else _pitched(M, N, out)
        lib.ts_linear_grad_input(gz, w, gx, act=act, preact=pre, tile=tile, max_workers=workers)
        lib.ts_sync_and_check()
        own = 2.0 ** -20 * (z.abs() + 1)
        _close(gx, s * slope, SLOPE[act] * _sum_bound(S, K) + own * s.abs() + (2.0 ** -23 + 2 * HALF[out]) * (s * slope).abs(), act)


@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("K", [192, 2048])
def test_waits_that_run_out_with_a_residual(lib, tile, out, K):
    """Loads of residuals that are under way when a wait gives up are waited for, and the next call is right."""
    M, N = 1000, 2000
    g = _gen(K, tile)
    x, w, res = _fill(M, K, g, ints=True), _fill(N, K, g, ints=True), _fill(M, N, g, out, ints=True)
    y = _pitched(M, N, out)
    try:
        lib.ts_linear(x, w, y, residual=res, tile=tile, timeout_s=1e-9)
        lib.ts_sync_and_check()
    except lib.TsError as e:
        assert "timed out" in str(e)
    lib.ts_linear(x, w, y, residual=res, tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(y, (x.double() @ w.double().t() + res.double()).to(out))
