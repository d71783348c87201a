"""Argument checks of a linear layer's operators that need no GPU: they precede every CUDA call."""
import ctypes

import pytest
import torch

P = 1 << 20  # an address that is never touched


def _linear(ts, M=64, N=64, K=64, out=1, x=P, w=2 * P, y=4 * P, **opts):
    return ts._lib.ts_linear(x, w, y, M, N, K, out, ts.LinearOpts(**opts), None)


def _gin(ts, M=64, N=64, K=64, out=1, g=P, w=2 * P, d=4 * P, **opts):
    return ts._lib.ts_linear_grad_input(g, w, d, M, N, K, out, ts.LinearGradOpts(**opts), None)


def _gw(ts, M=64, N=64, K=64, out=1, g=P, x=2 * P, d=4 * P, **opts):
    return ts._lib.ts_linear_grad_weight(g, x, d, M, N, K, out, ts.LinearGradOpts(**opts), None)


def test_linear_refuses(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    assert _linear(ts, M=-1) == E and _linear(ts, K=1 << 31) == E and _linear(ts, N=(1 << 31) - 511) == E
    assert "sizes" in ts.ts_last_error_detail()
    assert _linear(ts, out=2) == E and _linear(ts, out=-1) == E
    assert _linear(ts, act=5) == E and _linear(ts, act=-1) == E and "act" in ts.ts_last_error_detail()
    assert _linear(ts, tile=4) == E and _linear(ts, max_workers=-1) == E
    assert _linear(ts, timeout_s=-1.0) == E and _linear(ts, timeout_s=float("nan")) == E
    assert _linear(ts, bias=P, bias_type=2) == E
    assert _linear(ts, ldx=56) == E and _linear(ts, ldw=56) == E and _linear(ts, ldy=63) == E
    assert _linear(ts, residual=8 * P, ld_residual=63) == E and _linear(ts, preact=8 * P, ld_preact=1) == E
    assert _linear(ts, x=0) == E and _linear(ts, w=0) == E and _linear(ts, y=0) == E
    assert _linear(ts, y=4 * P + 2) == E and _linear(ts, residual=8 * P + 1) == E and _linear(ts, preact=8 * P + 2) == E
    assert _linear(ts, bias=8 * P + 2, bias_type=1) == E and _linear(ts, bias=8 * P + 1) == E
    assert _linear(ts, x=P + 8) == U and _linear(ts, w=2 * P + 2) == U and _linear(ts, ldx=68) == U and _linear(ts, K=60) == U
    assert "16-byte" in ts.ts_last_error_detail()
    # outputs over operands, the residual elsewhere on y, preact on anything
    assert _linear(ts, y=P) == E and _linear(ts, y=2 * P + 64) == E
    assert _linear(ts, residual=4 * P + 4) == E and _linear(ts, residual=4 * P, ld_residual=128) == E
    assert _linear(ts, preact=4 * P) == E and _linear(ts, preact=8 * P, residual=8 * P) == E and _linear(ts, preact=P) == E
    assert _linear(ts, bias=4 * P) == E
    assert _linear(ts, M=0) == ts.TS_OK and _linear(ts, N=0, x=0, w=0, y=0) == ts.TS_OK


def test_gradient_products_refuse(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    for f in (_gin, _gw):
        assert f(ts, M=-1) == E and f(ts, K=1 << 31) == E and f(ts, out=2) == E and f(ts, act=5) == E
        assert f(ts, tile=-1) == E and f(ts, max_workers=-1) == E and f(ts, timeout_s=-1.0) == E
        assert f(ts, ldg=63) == E and f(ts, ldb=63) == E and f(ts, ldd=63) == E
        assert f(ts, g=0) == E and f(ts, d=0) == E and f(ts, d=4 * P + 2) == E
        assert f(ts, g=P + 2) == U and f(ts, ldg=65) == U and f(ts, ldb=70) == U and f(ts, N=60) == U
        assert f(ts, d=P) == E and "overlaps" in ts.ts_last_error_detail()
    assert _gin(ts, w=0) == E and _gw(ts, x=0) == E
    # an activation and its pre-activations come together; a weight gradient has neither
    assert _gin(ts, act=1) == E and _gin(ts, aux=8 * P) == E and _gw(ts, act=1) == E
    assert _gin(ts, act=1, aux=4 * P, ld_aux=128) == E and _gw(ts, aux=4 * P + 4) == E and _gw(ts, aux=8 * P, ld_aux=3) == E
    assert _gin(ts, M=0) == ts.TS_OK and _gin(ts, K=0) == ts.TS_OK and _gw(ts, N=0) == ts.TS_OK


def test_act_grad_refuses(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED

    def call(M=64, N=64, gy=P, z=2 * P, gz=4 * P, gb=8 * P, dtype=1, act=1, ldy=0, ldp=0, ldg=0):
        return ts._lib.ts_act_grad(gy, z, gz, gb, M, N, dtype, act, ldy, ldp, ldg, None)

    assert call(M=-1) == E and call(N=1 << 31) == E and call(dtype=2) == E and call(act=5) == E
    assert call(z=0) == E and call(act=0) == E and call(gz=0, gb=0) == E and call(gy=0) == E
    assert call(ldy=63) == E and call(ldp=3) == E and call(ldg=1) == E
    assert call(gy=P + 2) == E and call(gb=8 * P + 2) == E
    assert call(gz=P + 16) == E and call(gz=P, ldg=128) == E and call(gb=P) == E and call(gb=4 * P + 64) == E
    assert call(N=0) == ts.TS_OK and call(M=0, gb=0) == ts.TS_OK
    assert U == ts.TS_ERR_UNSUPPORTED


def test_orthogonalise_refuses(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    need = ts.ts_orthogonalise_workspace(2, 64, 32)
    assert need > 0 and ts.ts_orthogonalise_workspace(0, 64, 32) == 0 and ts.ts_orthogonalise_workspace(1, 1 << 21, 32) == 0
    assert ts.ts_orthogonalise_workspace(1, 1 << 20, 1 << 20) >= 4 << 40 and ts.ts_orthogonalise_workspace(2, 1 << 20, 1 << 20) == 0
    assert ts.ts_orthogonalise_workspace(1, 64, 32, 0) < 1024

    def call(n=2, R=64, C=32, G=P, O=2 * P, ws=16 * P, size=None, g_type=0, **opts):  # noqa: E741
        return ts._lib.ts_orthogonalise(G, O, n, R, C, g_type, ts.OrthOpts(**opts), ws, need if size is None else size, None)

    assert call(n=-1) == E and call(R=-1) == E and call(C=(1 << 20) + 1) == E and call(n=65536) == U
    assert call(n=2, R=1 << 20, C=1 << 20) == U and call(g_type=2) == E
    assert call(steps=65) == E and call(eps=-1.0) == E and call(eps=float("inf")) == E and call(eps=float("nan")) == E
    assert call(a=float("nan")) == E and call(b=float("inf")) == E and call(timeout_s=-1.0) == E
    assert call(ldg=31) == E and call(ldo=31) == E and call(g_matrix=64) == E and call(o_matrix=2047) == E
    assert call(G=0) == E and call(O=0) == E and call(G=P + 1) == E and call(O=2 * P + 1) == E and call(G=P + 2, g_type=1) == E
    assert call(ws=0) == E and call(size=need - 1) == E and call(ws=16 * P + 128) == E and "256" in ts.ts_last_error_detail()
    assert call(O=P) == E and call(ws=P) == E and call(O=16 * P) == E
    assert call(n=0) == ts.TS_OK and call(R=0) == ts.TS_OK and call(C=0, G=0, O=0, ws=0) == ts.TS_OK


def test_options_have_the_packed_layout(ts):
    """The binding packs options into bytes; they must lie as the structures do."""
    for packed, struct in ((ts._PACK_LINEAR, ts.LinearOpts), (ts._PACK_LINEAR_GRAD, ts.LinearGradOpts),
                           (ts._PACK_ORTH, ts.OrthOpts)):
        assert packed.size == ctypes.sizeof(struct)
        values = list(range(1, len(struct._fields_) + 1))
        o = struct.from_buffer_copy(packed.pack(*values))
        assert [getattr(o, n) or 0 for n, _ in struct._fields_] == values


def test_binding_refuses_host_tensors(ts):
    a, y = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((4, 4))
    with pytest.raises(TypeError):
        ts.ts_linear(a, a, y)
    with pytest.raises(TypeError):
        ts.ts_linear_grad_input(a, a, y)
    with pytest.raises(TypeError):
        ts.ts_linear_grad_weight(a, a, y)
    with pytest.raises(TypeError):
        ts.ts_act_grad(y, None, y)
    with pytest.raises(TypeError):
        ts.ts_orthogonalise(a, a)
