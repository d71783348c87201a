"""Waits of ts_orthogonalise that run out at any point: a status, or the right result, and a context that works."""
import time

import pytest
import torch

from orth_accuracy import matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,C", [(40, 60), (300, 500), (1000, 1001), (2048, 1500)])
def test_limits_of_all_lengths(lib, R, C):
    """Limits about the length of the grid barrier's waits, the first loads' and the K loops', so that some CTAs and
    warps give up and others do not.  A CTA leaves with all of its threads, and waits once at most."""
    g = matrix(R, C, 1, device="cuda")
    want, out = (torch.empty((R, C), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.ts_orthogonalise(g, want)
    lib.ts_sync_and_check()
    gave_up = 0
    for limit in (1e-9, 1e-6, 2e-6, 3e-6, 4e-6, 6e-6, 1e-5, 1e-4):
        for _ in range(4):
            out.fill_(float("nan"))
            torch.cuda.synchronize()
            t0 = time.monotonic()
            lib.ts_orthogonalise(g, out, timeout_s=limit)
            try:
                lib.ts_sync_and_check()
                assert torch.equal(out, want)
            except lib.TsError as e:
                assert e.status == lib.TS_ERR_TIMEOUT
                gave_up += 1
            # each of 17 products' CTAs drains for 0.2 s at most
            assert time.monotonic() - t0 < 4
    assert gave_up > 0
    lib.ts_orthogonalise(g, out)
    lib.ts_sync_and_check()
    assert torch.equal(out, want)
