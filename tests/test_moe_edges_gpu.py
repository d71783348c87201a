"""Edges of the mixture-of-experts operators: empty batches, streams and threads, far rows, extreme values."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _plan_buffers(T, k, E):
    return (torch.full((E + 1,), -5, dtype=torch.int64, device="cuda"),
            torch.full((T * k,), -5, dtype=torch.int32, device="cuda"),
            torch.full((T, k), -5, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("E", [1, 31, 33, 64, 256, 700, 1024])
def test_plan_without_slots_after_one_with_some(lib, E):
    # the counts of the first plan are what the second would find in shared memory that it did not clear
    full = torch.randint(0, E, (250, 8), dtype=torch.int32, device="cuda")
    empty = torch.empty((0, 8), dtype=torch.int32, device="cuda")
    kept = [_plan_buffers(250, 8, E) for _ in range(20)]
    offs = [_plan_buffers(0, 8, E) for _ in range(20)]
    for a, b in zip(kept, offs):
        lib.ts_moe_plan(full, *a)
        lib.ts_moe_plan(empty, *b)
    lib.ts_sync_and_check()
    assert all(not off.any() for off, _, _ in offs)
