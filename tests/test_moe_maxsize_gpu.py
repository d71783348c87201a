"""Offsets past 2^31 elements in the mixture-of-experts operators, spot-checked at the far end."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_product_output_past_2_31(lib):
    M, N, K = 70001, 33000, 16  # D of 2.3e9 values
    A = torch.randint(-4, 5, (M, K), device="cuda").float().to(torch.float8_e4m3fn)
    B = torch.randint(-4, 5, (N, K), device="cuda").float().to(torch.float8_e4m3fn)
    SA = torch.full((1, M), 0.5, device="cuda").t()
    SB = torch.full((-(-N // 128), 1), 2.0, device="cuda")
    D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    lib.ts_gemm_fp8(A, SA, B, SB, D)
    lib.ts_sync_and_check()
    for rows in (slice(0, 3), slice(65534, 65538), slice(M - 3, M)):
        assert torch.equal(D[rows], (A[rows].float() @ B.float().t()).bfloat16())


@pytest.mark.parametrize("transpose", [False, True])
def test_quantisation_past_2_31(lib, transpose):
    M, N = 70000, 31000  # 2.2e9 values
    x = torch.randint(-8, 9, (M, N), device="cuda", dtype=torch.int8).bfloat16()
    x[:, ::100] = 14  # every block's largest magnitude is 14: its factor, 32, is exact
    x[::100] = 14
    qr, qc = (N, M) if transpose else (M, N)
    q = torch.empty((qr, qc), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((-(-qc // 128), qr), device="cuda").t()
    lib.ts_quant_fp8(x, q, s, transpose=transpose)
    lib.ts_sync_and_check()
    # the last block along a row of q is short and may hold no 14
    assert bool((s[:, :-1] == 14.0 / 448.0).all())
    for rows in (slice(0, 2), slice(qr - 2, qr)):
        want = (x[:, rows].t() if transpose else x[rows]).float()
        factor = torch.full((2, s.shape[1]), 32.0, device="cuda")
        factor[:, -1] = 448.0 / want[:, 128 * (s.shape[1] - 1):].abs().amax(1)
        want = (want * factor.repeat_interleave(128, 1)[:, :qc]).to(torch.float8_e4m3fn)
        assert torch.equal(q[rows].float(), want.float())


def test_combine_past_2_31(lib):
    R, N, T = 70000, 33000, 8  # y and grad_y of 2.3e9 values
    y = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    y[R - 5:] = torch.randn((5, N), device="cuda").bfloat16()
    pos = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    pos[0, 0], pos[3, 1], pos[7, 0] = R - 1, R - 5, R - 3
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    lib.ts_moe_combine(y, pos, out)
    go = torch.randn((T, N), device="cuda").bfloat16()
    gy = torch.zeros_like(y)
    lib.ts_moe_combine_grad(go, y, pos, None, gy)
    lib.ts_sync_and_check()
    assert torch.equal(out[0], y[R - 1]) and torch.equal(out[3], y[R - 5]) and torch.equal(out[7], y[R - 3])
    assert torch.equal(gy[R - 1], go[0]) and torch.equal(gy[R - 5], go[3]) and not gy[:R - 5].any()


def test_plan_of_many_slots(lib):
    T, k, E = 1 << 20, 2, 100  # more tiles than one placing CTA sums by itself
    e = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int64, device="cuda")
    order = torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos = torch.empty((T, k), dtype=torch.int32, device="cuda")
    lib.ts_moe_plan(e, off, order, pos)
    lib.ts_sync_and_check()
    ref = e.flatten().long().sort(stable=True).indices
    assert torch.equal(order.long(), ref)
    assert torch.equal(off[1:], torch.bincount(e.flatten().long(), minlength=E).cumsum(0))
    assert torch.equal(pos.flatten()[ref].long(), torch.arange(T * k, device="cuda"))


def test_plan_on_another_stream(lib):
    # the scratch that the call keeps belongs to the stream it runs on
    e = torch.randint(0, 16, (40000, 2), dtype=torch.int32, device="cuda")
    outs = []
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams * 3:
        off = torch.empty(17, dtype=torch.int64, device="cuda")
        order = torch.empty(80000, dtype=torch.int32, device="cuda")
        pos = torch.empty((40000, 2), dtype=torch.int32, device="cuda")
        lib.ts_moe_plan(e, off, order, pos, stream=st)
        outs.append((off, order, pos))
    torch.cuda.synchronize()
    lib.ts_sync_and_check()
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(outs[0], o))
