"""Which matrices overlap, without a GPU: every call here is refused, for one reason or for another behind it."""
import random

P = 1 << 20  # an address that is never touched


def _bytes(at, rows, width, pitch):
    return {at + r * pitch + i for r in range(rows) for i in range(width)}


def test_windows_of_one_buffer(ts):
    """Rows of one pitch: refused where a byte is shared, and only there.  A misaligned bias is refused behind that."""
    rng = random.Random(1)
    shared = apart = 0
    for _ in range(4000):
        M, N, K, pitch = rng.randint(1, 4), rng.randint(1, 12), 8 * rng.randint(1, 2), 8 * rng.randint(3, 6)
        at = [P + 2 * rng.randint(0, 2 * pitch) for _ in range(3)]
        x = P + 16 * rng.randint(0, 12)
        y, res, pre = at
        opts = {"bias": P + 1, "residual": res, "preact": pre, "ldx": pitch, "ldw": pitch, "ldy": pitch, "ld_residual": pitch, "ld_preact": pitch}
        assert ts._lib.ts_linear(x, 16 * P, y, M, N, K, 0, ts.LinearOpts(**opts), None) == ts.TS_ERR_INVALID_ARG
        by, br, bp = (_bytes(a, M, 2 * N, 2 * pitch) for a in at)
        bx = _bytes(x, M, 2 * K, 2 * pitch)
        clash = by & bx or (by & br and y != res) or bp & (by | br | bx)
        detail = ts.ts_last_error_detail()
        assert ("overlaps" in detail) == bool(clash), (M, N, K, pitch, x, at, detail)
        assert clash or "bias is not aligned" in detail
        shared, apart = shared + bool(clash), apart + (not clash)
    assert shared > 500 and apart > 100


def test_batches_and_workspaces(ts):
    """Matrices behind one another and side by side.  A workspace over G is refused behind the check of O and G."""
    rng = random.Random(2)
    seen = {"matrices": 0, "O overlaps G": 0, "workspace overlaps": 0}
    for _ in range(4000):
        n, R, C = rng.randint(2, 3), rng.randint(1, 3), rng.randint(1, 6)
        ld, matrix = rng.randint(C, 30), rng.randint(C, 40)
        if rng.random() < 0.5:
            matrix = ld * rng.randint(1, 4)
        G, O = P, P + 2 * rng.randint(0, 60)  # noqa: E741
        opts = {"ldg": ld, "ldo": ld, "g_matrix": matrix, "o_matrix": matrix}
        assert ts._lib.ts_orthogonalise(G, O, n, R, C, 0, ts.OrthOpts(**opts), P, 1 << 19, None) == ts.TS_ERR_INVALID_ARG
        detail = ts.ts_last_error_detail()
        rows = [[_bytes(a + 2 * z * matrix, R, 2 * C, 2 * ld) for z in range(n)] for a in (G, O)]
        inside = sum(len(b) for b in rows[0]) != len(set().union(*rows[0]))
        both = set().union(*rows[0]) & set().union(*rows[1])
        kind = next(k for k in seen if k in detail)
        seen[kind] += 1
        if inside:
            assert kind == "matrices"
        elif both:
            assert kind in ("matrices", "O overlaps G")
        # what is taken shares nothing
        if kind == "workspace overlaps":
            assert not inside and not both
    assert min(seen.values()) > 100, seen
    # side by side, and windows of rows that both have: taken up to the workspace
    for opts, off in (({"ldg": 32, "ldo": 32, "g_matrix": 8, "o_matrix": 8}, 32), ({"ldg": 64, "ldo": 64, "g_matrix": 512, "o_matrix": 512}, 64),
                      ({"ldg": 64, "ldo": 64}, 64)):
        assert ts._lib.ts_orthogonalise(P, P + off, 2, 8, 8, 0, ts.OrthOpts(**opts), P, 1 << 19, None) == ts.TS_ERR_INVALID_ARG
        assert "workspace overlaps" in ts.ts_last_error_detail()


def test_act_grad_windows_that_share(ts):
    def call(gz, gy=P, z=0, gb=0, ld=64, N=16, M=4, act=0):
        return ts._lib.ts_act_grad(gy, z, gz, gb, M, N, 1, act, ld, ld, ld, None)

    for gz in (P + 4, P + 60, P + 3 * 256, P + 256 - 60, P - 4, P - 256 + 200):
        assert call(gz) == ts.TS_ERR_INVALID_ARG and "overlaps an input" in ts.ts_last_error_detail()
    assert call(0, gb=P + 256) == ts.TS_ERR_INVALID_ARG and call(P + 64, z=P + 96, act=1) == ts.TS_ERR_INVALID_ARG
