"""The workspace that the binding takes for ts_orthogonalise is the call's own."""
import threading

import pytest
import torch

from orth_accuracy import check, matrix

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_nothing_is_kept(lib):
    g = matrix(2048, 1024, 1, device="cuda")
    out = torch.empty_like(g)
    lib.ts_sync_and_check()
    before = torch.cuda.memory_allocated()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        lib.ts_orthogonalise(g, out, stream=stream)
        lib.ts_sync_and_check(side)
        lib.ts_sync_and_check()
        assert torch.cuda.memory_allocated() == before
        check(out, g)


def test_memory_that_is_handed_out_again(lib):
    """What is allocated behind a call on its stream may lie where the call's workspace was."""
    side = torch.cuda.Stream()
    need = lib.ts_orthogonalise_workspace(1, 700, 900)
    g = matrix(700, 900, 2, device="cuda")
    outs = [torch.empty_like(g) for _ in range(6)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        stream = side if i % 2 else None
        lib.ts_orthogonalise(g, out, stream=stream)
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xAB)
    torch.cuda.synchronize()
    lib.ts_sync_and_check()
    for out in outs:
        check(out, g)
        assert torch.equal(out, outs[0])


def test_threads_that_share_a_stream(lib):
    jobs = [(matrix(300 + 10 * i, 400, i, device="cuda"), torch.empty((300 + 10 * i, 400), dtype=BF16, device="cuda")) for i in range(4)]
    torch.cuda.synchronize()

    def work(g, out):
        for _ in range(10):
            lib.ts_orthogonalise(g, out)

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    lib.ts_sync_and_check()
    for g, out in jobs:
        check(out, g)
