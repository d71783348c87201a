"""Argument checks of the mixture-of-experts operators that need no GPU: they precede every CUDA call."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that is never touched


def _fp8(ts, M=64, N=64, K=64, out=None, A=P, SA=P, B=2 * P, SB=P, D=4 * P, groups=None, offsets=P, **opts):
    o = ts.Fp8Opts(**opts)
    out = ts.TS_OUT_F32 if out is None else out
    if groups is None:
        return ts._lib.ts_gemm_fp8(A, SA, B, SB, D, M, N, K, out, o, None)
    return ts._lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, offsets, groups, M, N, K, out, o, None)


def test_products_refuse(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    assert _fp8(ts, M=-1) == E and _fp8(ts, K=1 << 31) == E
    assert "sizes" in ts.ts_last_error_detail()
    assert _fp8(ts, out=2) == E
    assert _fp8(ts, a_type=2) == E and _fp8(ts, b_type=-1) == E and _fp8(ts, b_scale=2) == E
    assert _fp8(ts, trans_b=2) == E and _fp8(ts, tile=4) == E and _fp8(ts, max_workers=-1) == E
    assert _fp8(ts, timeout_s=-1.0) == E and _fp8(ts, sa_row=-1) == E
    assert _fp8(ts, lda=48) == E and _fp8(ts, ldb=48) == E and _fp8(ts, ldd=63) == E
    assert _fp8(ts, b_scale=1, trans_b=1) == U and _fp8(ts, b_scale=1, groups=2) == U
    assert _fp8(ts, D=0) == E and _fp8(ts, D=4 * P + 2) == E
    assert _fp8(ts, A=0) == E and _fp8(ts, SB=0) == E and _fp8(ts, SA=P + 2) == E
    assert _fp8(ts, A=P + 8) == U and _fp8(ts, lda=72) == U and _fp8(ts, K=60) == U
    assert "16-byte" in ts.ts_last_error_detail()
    assert _fp8(ts, D=P) == E and "overlap" in ts.ts_last_error_detail()
    assert _fp8(ts, groups=-1) == E and _fp8(ts, groups=1025) == U
    assert _fp8(ts, groups=2, offsets=0) == E and _fp8(ts, groups=2, offsets=P + 4) == E
    assert _fp8(ts, groups=2, b_group=64) == E and _fp8(ts, groups=2, b_group=64 * 64 + 8) == U
    # nothing to do: no CUDA call either
    assert _fp8(ts, M=0) == ts.TS_OK and _fp8(ts, N=0) == ts.TS_OK and _fp8(ts, groups=0) == ts.TS_OK


def test_quantiser_refuses(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED

    def call(M=64, N=256, x=P, q=4 * P, s=8 * P, x_type=0, q_type=0, **opts):
        return ts._lib.ts_quant_fp8(x, q, s, M, N, x_type, q_type, ts.QuantOpts(**opts), None)

    assert call(M=-1) == E and call(N=1 << 31) == E and call(x_type=2) == E and call(q_type=2) == E
    assert call(transpose=2) == E and call(transpose=1, rows=P) == U and call(rows=P, out_rows=4, rows_div=-1) == E
    assert call(ldx=255) == E and call(ldq=255) == E and call(transpose=1, ldq=63) == E
    assert call(x=0) == E and call(q=0) == E and call(s=0) == E and call(x=P + 1) == E and call(s=8 * P + 2) == E
    assert call(rows=P + 2, out_rows=4) == E
    assert call(q=P) == E and "overlap" in ts.ts_last_error_detail()
    assert call(N=1 << 30, q=1 << 50) == U
    assert call(M=0) == ts.TS_OK and call(N=0) == ts.TS_OK and call(rows=P, out_rows=0) == ts.TS_OK


def test_router_refuses(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED

    def call(T=4, n=64, k=4, dtype=1, x=P, e=P, w=P, **opts):
        return ts._lib.ts_moe_route(x, e, w, T, n, k, dtype, ts.RouteOpts(**opts), None)

    assert call(T=-1) == E and call(n=0) == E and call(k=0) == E and call(k=65) == E and call(dtype=2) == E
    assert call(n=1025) == U and call(n=64, k=33) == U
    assert call(score=2) == E and call(no_renorm=2) == E and call(groups=5) == E and call(groups=-1) == E
    assert call(groups=64) == U and call(groups=8, keep_groups=9) == E and call(groups=32, keep_groups=1) == E
    assert call(group_best=3) == E and call(ldx=63) == E and call(x=0) == E and call(x=P + 2) == E
    assert call(T=0, x=0, e=0, w=0) == ts.TS_OK
    grad = lambda **kw: ts._lib.ts_moe_route_grad(P, P, P, P, kw.get("T", 4), kw.get("n", 64), kw.get("k", 4), 1,  # noqa: E731
                                                  ts.RouteOpts(**kw.get("opts", {})), None)
    assert grad(k=65) == E and grad(opts={"ldg": 3}) == E and grad(T=0) == ts.TS_OK


def test_plan_refuses(ts):
    E, U = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    call = lambda n=8, e=4, ws=0, size=0, experts=P, off=P: ts._lib.ts_moe_plan(experts, off, P, P, n, e, ws, size, None)  # noqa: E731
    assert call(n=-1) == E and call(e=0) == E and call(e=1025) == U and call(off=0) == E and call(experts=0) == E
    assert call(off=P + 4) == E
    need = ts.ts_moe_plan_workspace(1 << 20, 64)
    assert need > 0 and ts.ts_moe_plan_workspace(8, 64) == 0
    assert call(n=1 << 20, e=64) == E and call(n=1 << 20, e=64, ws=P, size=need - 1) == E
    assert "workspace" in ts.ts_last_error_detail()


def test_combine_refuses(ts):
    E = ts.TS_ERR_INVALID_ARG

    def call(T=4, k=2, N=64, R=8, dtype=0, y=P, pos=P, w=P, out=4 * P, ldy=0, ldo=0):
        return ts._lib.ts_moe_combine(y, pos, w, out, T, k, N, R, dtype, ldy, ldo, None)

    assert call(T=-1) == E and call(R=1 << 31) == E and call(k=-1) == E and call(k=1025) == E and call(dtype=3) == E
    assert call(ldy=63) == E and call(ldo=63) == E and call(y=0) == E and call(out=0) == E and call(pos=0) == E
    assert call(out=4 * P + 1) == E and call(pos=P + 2) == E and call(out=P) == E
    assert call(T=0) == ts.TS_OK and call(N=0) == ts.TS_OK

    def grad(T=4, k=2, N=64, R=8, go=P, y=2 * P, pos=P, gy=4 * P, gw=P, ldg=0):
        return ts._lib.ts_moe_combine_grad(go, y, pos, P, gy, gw, T, k, N, R, 0, 0, 0, ldg, None)

    assert grad(ldg=63) == E and grad(go=0) == E and grad(gy=0) == E and grad(pos=0) == E
    assert grad(gy=P) == E and grad(gy=2 * P) == E and grad(gw=P + 2) == E
    assert grad(T=0) == ts.TS_OK and grad(k=0) == ts.TS_OK


def test_binding_structs_match_the_header_layout(ts, tmp_path):
    structs = {"ts_fp8_opts": ts.Fp8Opts, "ts_quant_opts": ts.QuantOpts, "ts_route_opts": ts.RouteOpts}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "tsgemm.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = {tuple(x.split()[:2]): int(x.split()[2])
           for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()}
    for name, cls in structs.items():
        assert got[(name, "size")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(name, f)] == getattr(cls, f).offset, f"{name}.{f}"


@pytest.mark.parametrize("name,cls", [("_PACK_FP8", "Fp8Opts"), ("_PACK_QUANT", "QuantOpts"), ("_PACK_ROUTE", "RouteOpts")])
def test_packed_options_are_the_structures(ts, name, cls):
    cls, packer = getattr(ts, cls), getattr(ts, name)
    values = [i + 1 for i in range(len(cls._fields_))]
    o = cls.from_buffer_copy(packer.pack(*values))
    assert [getattr(o, f) for f, _ in cls._fields_] == values


@pytest.mark.parametrize("name,value", [("TS_FP8_E4M3", 0), ("TS_FP8_E5M2", 1), ("TS_SCALE_BLOCK", 0), ("TS_SCALE_ROW", 1),
                                        ("TS_SCORE_SOFTMAX", 0), ("TS_SCORE_SIGMOID", 1)])
def test_constants(ts, name, value):
    assert getattr(ts, name) == value


@pytest.mark.parametrize("trans", [0, 1])
def test_groups_of_one_row_keep_the_callers_pitch(ts, trans):
    # B's groups of a single row, one after another: the default distance is that row's length (or ldb)
    U, E = ts.TS_ERR_UNSUPPORTED, ts.TS_ERR_INVALID_ARG
    one = dict(N=100, K=1, trans_b=1, lda=16) if trans else dict(N=1, K=100, lda=112)
    assert _fp8(ts, groups=2, **one) == U and "b_group" in ts.ts_last_error_detail()
    assert _fp8(ts, groups=2, ldb=104, **one) == U and _fp8(ts, groups=2, ldb=96, **one) == E
    assert _fp8(ts, groups=2, b_group=1 << 40, **one) == E and _fp8(ts, groups=2, ldb=1 << 40, **one) == E
    assert _fp8(ts, groups=2, b_group=120, ldb=96, **one) == U  # given, it leaves a single row's pitch unused
    # a padded row: the second group ends 1024 + 100 bytes behind B's start
    assert _fp8(ts, groups=2, D=2 * P + 1024 + 96, ldb=1024, **one) == E and "overlap" in ts.ts_last_error_detail()


@pytest.fixture
def no_cuda_scratch(ts, monkeypatch):
    """The plan's scratch on the CPU: its streams are integers, and `capturing` says which of them capture."""
    import contextlib

    import torch

    current, capturing = [0], set()

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        try:
            yield
        finally:
            current.pop()

    class Stream(int):
        cuda_stream = property(int)

        def __new__(cls, handle, device=None):
            return int.__new__(cls, handle)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: int(current[-1]) in capturing)
    monkeypatch.setattr(ts, "_stream_of", lambda s: int(current[-1] if s is None else s))
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(int(current[-1])) or empty(*a, **kw))
    return current, capturing, made, lambda stream=None, n=1000: ts._scratch_for(n, torch.device("cpu"), stream)


def test_threads_on_one_stream_do_not_share_a_plans_scratch(no_cuda_scratch):
    import threading

    *_, scratch = no_cuda_scratch
    mine = scratch(7)
    assert scratch(7) is mine, "kept from call to call"
    got = []
    t = threading.Thread(target=lambda: got.append(scratch(7)))
    t.start()
    t.join()
    assert got[0].data_ptr() != mine.data_ptr()


def test_a_captured_plans_scratch_is_its_graphs(no_cuda_scratch):
    current, capturing, made, scratch = no_cuda_scratch
    kept = scratch(7)
    made.clear()
    # a capture that forks: the current stream (0) captures too, and the plan runs on 7
    capturing |= {0, 7}
    first = scratch(7)
    assert made == [7] and first.data_ptr() != kept.data_ptr(), "allocated on the stream that uses it"
    assert scratch().data_ptr() != first.data_ptr() and made == [7, 0]
    # only the plan's stream captures: the graph must not record the kept scratch
    capturing.discard(0)
    assert scratch(7).data_ptr() not in (kept.data_ptr(), first.data_ptr())
    # and nothing of a graph is kept for later calls
    capturing.clear()
    assert scratch(7) is kept
    # only the current stream captures: the call is no part of the graph
    capturing.add(0)
    assert scratch(7) is kept


def test_grouped_rows_stay_below_2_31(ts):
    # a group may start at any row, and its tiles reach up to 255 rows past its last one
    U, top = ts.TS_ERR_UNSUPPORTED, (1 << 31) - 256
    assert _fp8(ts, M=top + 1, groups=2, D=1 << 50) == U and "rows" in ts.ts_last_error_detail()
    assert _fp8(ts, M=(1 << 31) - 1, groups=2, D=1 << 50) == U
    # at the limit, the next check answers
    assert _fp8(ts, M=top, groups=2, D=0) == ts.TS_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [0, -0.0, 1e-50, -1e-50, 2.0 ** -150])
def test_a_routing_scale_that_is_zero_in_32_bits(ts, scale):
    # the options hold it in fp32, where 0 stands for the default of 1
    with pytest.raises(ValueError, match="scale"):
        ts.ts_moe_route(None, None, None, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        ts.ts_moe_route_grad(None, None, None, None, scale=scale)
    assert ts._PACK_ROUTE.unpack(ts._PACK_ROUTE.pack(*[0] * 6, 2.0 ** -149, 0, 0, 0))[6] == 2.0 ** -149
