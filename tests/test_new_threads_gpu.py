"""Calls from threads that have not touched the GPU: no call of theirs has made a context current yet."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _in_new_thread(f):
    got = []

    def body():
        try:
            f()
            got.append(None)
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if got[0] is not None:
        raise got[0]


# few tokens; tokens as columns; a cluster's shared K; persistent tiles
@pytest.mark.parametrize("M,N,K", [(3, 72, 200), (30, 304, 520), (152, 200, 904), (1000, 2000, 1104)])
def test_linear_layer(lib, M, N, K):
    g = torch.Generator("cuda").manual_seed(M)
    x, w, gz = (torch.randint(-3, 4, s, device="cuda", generator=g).to(BF16) for s in ((M, K), (N, K), (M, N)))
    y, gx, gw, gb = (torch.empty(s, device="cuda") for s in ((M, N), (M, K), (N, K), (N,)))
    torch.cuda.synchronize()
    _in_new_thread(lambda: lib.ts_linear(x, w, y))
    _in_new_thread(lambda: lib.ts_linear_grad_input(gz, w, gx))
    _in_new_thread(lambda: lib.ts_linear_grad_weight(gz, x, gw))
    _in_new_thread(lambda: lib.ts_act_grad(gz, None, None, gb))
    lib.ts_sync_and_check()
    assert torch.equal(y.double(), x.double() @ w.double().t()) and torch.equal(gx.double(), gz.double() @ w.double())
    assert torch.equal(gw.double(), gz.double().t() @ x.double()) and torch.equal(gb.double(), gz.double().sum(0))


@pytest.mark.parametrize("R,C", [(100, 200), (2048, 1024)])
def test_orthogonalise(lib, R, C):
    g = torch.randn((R, C), device="cuda")
    want, out = torch.empty((R, C), dtype=BF16, device="cuda"), torch.empty((R, C), dtype=BF16, device="cuda")
    lib.ts_orthogonalise(g, want)
    ws = torch.empty(lib.ts_orthogonalise_workspace(1, R, C), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _in_new_thread(lambda: lib.ts_orthogonalise(g, out, workspace=ws))
    lib.ts_sync_and_check()
    assert torch.equal(out, want)


def test_gemm(lib):
    A, B = (torch.randint(-3, 4, (300, 128), device="cuda").to(BF16) for _ in range(2))
    D = torch.empty((300, 300), device="cuda")
    torch.cuda.synchronize()
    _in_new_thread(lambda: lib.ts_gemm_bf16(A, B, D))
    lib.ts_sync_and_check()
    assert torch.equal(D.double(), A.double() @ B.double().t())
