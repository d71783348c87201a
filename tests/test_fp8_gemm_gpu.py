"""Block-scaled 8-bit products, plain and grouped by rows, against a 64-bit reference.

Two kinds of inputs.  Small integers with power-of-two scales: every product, K-block sum and scaled
sum is exact in fp32, so the result must be the reference's to the bit (rounded once to bf16).  Random
values with arbitrary scales: within a bound derived from the arithmetic below.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _cdiv(a, b):
    return -(-a // b)


def _pitched(r, c, dtype, step=16, extra=0):
    return torch.zeros((r, _cdiv(c, step) * step + extra), dtype=dtype, device="cuda")[:, :c]


def _operand(r, c, fmt, rng, ints, lead=()):
    v = rng.integers(-4, 5, (*lead, r, c)).astype(np.float32) if ints else \
        rng.standard_normal((*lead, r, c)).astype(np.float32) * 8
    q = torch.zeros((*lead, r, _cdiv(max(c, 1), 16) * 16), dtype=FORMATS[fmt], device="cuda")[..., :c]
    q.copy_(torch.from_numpy(v).to("cuda").to(FORMATS[fmt]))
    return q, q.to(torch.float64).cpu()


def _scale(shape, rng, ints, row_contiguous):
    v = 2.0 ** rng.integers(-2, 3, shape) if ints else np.exp(rng.standard_normal(shape))
    t = torch.from_numpy(v.astype(np.float32))
    if row_contiguous:
        d = torch.empty((*shape[:-2], shape[-1], shape[-2]), device="cuda").transpose(-1, -2)
        d.copy_(t)
    else:
        d = t.cuda()
    return d, t.double()


def _expand(s, rows, cols, row_step):
    return s.repeat_interleave(row_step, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]


def _problem(M, N, K, seed, ints=False, a="e4m3", b="e4m3", row=False, trans=False, sa_rows=True, groups=None):
    rng = np.random.default_rng(seed)
    A, a64 = _operand(M, K, a, rng, ints)
    lead = () if groups is None else (groups,)
    R, C = (K, N) if trans else (N, K)
    B, b64 = _operand(R, C, b, rng, ints, lead)
    SA, sa64 = _scale((M, _cdiv(K, 128)), rng, ints, sa_rows)
    SB, sb64 = _scale((*lead, R if row else _cdiv(R, 128), _cdiv(C, 128)), rng, ints, False)
    a64 = a64 * _expand(sa64, M, K, 1)
    b64 = b64 * _expand(sb64, R, C, 1 if row else 128)
    return A, SA, B, SB, a64, b64 if trans else b64.transpose(-1, -2)


def _check(D, ref, S, K, exact, what):
    got = D.double().cpu()
    assert torch.isfinite(got).all(), what
    if exact:
        assert torch.equal(D.cpu(), ref.to(D.dtype)), what
        return
    # One MMA adds 32 products and the running sum, each aligned to the largest and cut at no less than 23
    # bits: 33 * 2^-23 of the block's sum of magnitudes, four MMAs a block; then a rounding for the product
    # of the scales and one for each block's fused multiply-add; the output's own rounding.
    bound = (132 * 2.0 ** -23 + (_cdiv(K, 128) + 2) * 2.0 ** -24) * S
    bound += (2.0 ** -8 if D.dtype == torch.bfloat16 else 2.0 ** -23) * ref.abs() + 1e-30
    err = (got - ref).abs()
    assert bool((err <= bound).all()), f"{what}: error {float((err - bound).max())} past the bound"


SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 512), (3, 17, 40), (33, 129, 129), (127, 65, 300), (128, 128, 128),
         (129, 256, 1024), (200, 383, 777), (257, 640, 2048), (513, 512, 4096), (1023, 1025, 255)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", ["block", "trans", "row"])
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("ints", [True, False])
def test_product(lib, M, N, K, form, out, ints):
    A, SA, B, SB, a, b = _problem(M, N, K, M + N + K, ints, row=form == "row", trans=form == "trans")
    D = torch.full((M, N), float("nan"), dtype=out, device="cuda")
    lib.ts_gemm_fp8(A, SA, B, SB, D, trans_b=form == "trans")
    lib.ts_sync_and_check()
    _check(D, a @ b, a.abs() @ b.abs(), K, ints, f"{form} {M}x{N}x{K}")


@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("form", ["block", "trans", "row"])
@pytest.mark.parametrize("M,N,K", [(1, 100, 48), (300, 520, 1000), (777, 1280, 640)])
def test_tiles_agree(lib, M, N, K, form, tile):
    A, SA, B, SB, a, b = _problem(M, N, K, 3, True, row=form == "row", trans=form == "trans")
    D = torch.full((M, N), float("nan"), device="cuda")
    lib.ts_gemm_fp8(A, SA, B, SB, D, trans_b=form == "trans", tile=tile)
    lib.ts_sync_and_check()
    _check(D, a @ b, None, K, True, tile)


@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("b", ["e4m3", "e5m2"])
def test_formats_mix(lib, a, b):
    M, N, K = 150, 200, 450
    A, SA, B, SB, x, y = _problem(M, N, K, 11, False, a=a, b=b)
    D = torch.empty((M, N), device="cuda")
    lib.ts_gemm_fp8(A, SA, B, SB, D)
    lib.ts_sync_and_check()
    _check(D, x @ y, x.abs() @ y.abs(), K, False, f"{a} x {b}")


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("extra", [0, 1, 8])
def test_strides(lib, out, extra):
    # rows of D at odd pitches, scales with the blocks contiguous, operands inside wider ones
    M, N, K = 140, 210, 390
    A, SA, B, SB, a, b = _problem(M, N, K, 5, True, sa_rows=False)
    wide = torch.full((M + 2, N + extra + 3), float("nan"), dtype=out, device="cuda")
    D = wide[1:M + 1, extra:N + extra]
    lib.ts_gemm_fp8(A, SA, B, SB, D)
    lib.ts_sync_and_check()
    _check(D, a @ b, None, K, True, "strided")
    assert torch.isnan(wide[0]).all() and torch.isnan(wide[-1]).all(), "rows around D were written"
    assert torch.isnan(wide[:, :extra]).all() and torch.isnan(wide[:, N + extra:]).all(), "columns around D were written"


def test_empty_sizes(lib):
    for M, N, K in ((0, 5, 16), (5, 0, 16), (5, 7, 0)):
        A, SA, B, SB, _, _ = _problem(M, N, K, 1, True)
        D = torch.full((M, N), 3.0, device="cuda")
        lib.ts_gemm_fp8(A, SA, B, SB, D)
        lib.ts_sync_and_check()
        assert (D == 0).all() if K == 0 else D.numel() == 0


def test_not_a_number_stays_in_its_row_and_column(lib):
    M, N, K = 200, 300, 260
    A, SA, B, SB, a, b = _problem(M, N, K, 9, True)
    A[7, 200] = float("nan")
    B[130, 3] = float("nan")
    SA[150, 1] = float("inf")
    D = torch.zeros((M, N), device="cuda")
    lib.ts_gemm_fp8(A, SA, B, SB, D)
    lib.ts_sync_and_check()
    bad = ~torch.isfinite(D)
    assert bad[7].all() and bad[:, 130].all()
    bad[7] = bad[150] = False
    bad[:, 130] = False
    assert not bad.any()
    keep = torch.ones((M, N), dtype=torch.bool)
    keep[7] = keep[150] = False
    keep[:, 130] = False
    ref = (a.nan_to_num() @ b.nan_to_num()).float()
    assert torch.equal(D.cpu()[keep], ref[keep])


def test_another_stream_and_repeats(lib):
    M, N, K = 700, 900, 1100
    A, SA, B, SB, a, b = _problem(M, N, K, 21, False)
    D = [torch.empty((M, N), device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        lib.ts_gemm_fp8(A, SA, B, SB, D[0])
        SA2 = SA * 2  # written on this stream, read by the next product
        lib.ts_gemm_fp8(A, SA2, B, SB, D[1])
        lib.ts_gemm_fp8(A, SA, B, SB, D[2])
    lib.ts_sync_and_check(st)
    assert torch.equal(D[0], D[2]), "the same product twice differs"
    assert torch.equal(D[0] * 2, D[1])


def _grouped_ref(offsets, a, b, N):
    ref = torch.zeros((a.shape[0], N), dtype=torch.float64)
    for g in range(len(offsets) - 1):
        ref[offsets[g]:offsets[g + 1]] = a[offsets[g]:offsets[g + 1]] @ b[g]
    return ref


OFFSETS = [
    [0, 0], [0, 1], [0, 5, 5, 6], [0, 0, 0, 300], [3, 40, 168, 168, 297, 300], [0, 128, 256, 384],
    list(range(0, 65)), [10, 10, 10, 200, 201],
]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("case", range(len(OFFSETS)))
def test_grouped(lib, case, trans, out):
    off = OFFSETS[case]
    M, N, K, G = off[-1] + 7, 200, 300, len(off) - 1
    A, SA, B, SB, a, b = _problem(M, N, K, case, True, trans=trans, groups=G)
    D = torch.full((M, N), -777.0, dtype=out, device="cuda")
    lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, torch.tensor(off, device="cuda"), trans_b=trans)
    lib.ts_sync_and_check()
    ref = _grouped_ref(off, a, b, N)
    assert torch.equal(D.cpu()[off[0]:off[-1]], ref.to(out)[off[0]:off[-1]])
    assert (D[:off[0]] == -777.0).all() and (D[off[-1]:] == -777.0).all(), "rows outside every group were written"


@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
def test_grouped_tiles_agree(lib, tile):
    rng = np.random.default_rng(8)
    off = [0] + np.cumsum(rng.integers(0, 400, 9)).tolist()
    M, N, K, G = off[-1], 520, 384, 9
    A, SA, B, SB, a, b = _problem(M, N, K, 4, True, groups=G)
    D = torch.empty((M, N), device="cuda")
    lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, torch.tensor(off, device="cuda"), tile=tile)
    lib.ts_sync_and_check()
    assert torch.equal(D.cpu(), _grouped_ref(off, a, b, N).float())


def test_grouped_most_groups(lib):
    G = 1024
    off = torch.arange(G + 1) // 3  # mostly empty or of one row
    M, N, K = int(off[-1]), 64, 64
    A, SA, B, SB, a, b = _problem(M, N, K, 2, True, groups=G)
    D = torch.empty((M, N), device="cuda")
    lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, off.cuda())
    lib.ts_sync_and_check()
    assert torch.equal(D.cpu(), _grouped_ref(off.tolist(), a, b, N).float())


def test_grouped_keeps_a_neighbours_not_a_number_out(lib):
    off = [0, 100, 200]
    A, SA, B, SB, a, b = _problem(200, 128, 256, 6, True, groups=2)
    A[:100] = float("nan")
    D = torch.zeros((200, 128), device="cuda")
    lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, torch.tensor(off, device="cuda"))
    lib.ts_sync_and_check()
    assert torch.isnan(D[:100]).all()
    assert torch.equal(D[100:].cpu(), (a[100:] @ b[1]).float())


@pytest.mark.parametrize("off,bad", [([0, 50, 40, 100], 1), ([0, 50, 101, 101], 1), ([-1, 50, 60, 100], 0)])
def test_grouped_bad_offsets_are_reported(lib, off, bad):
    A, SA, B, SB, a, b = _problem(100, 64, 64, 6, True, groups=3)
    D = torch.zeros((100, 64), device="cuda")
    lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, torch.tensor(off, device="cuda"))
    with pytest.raises(lib.TsError) as e:
        lib.ts_sync_and_check()
    assert e.value.status == lib.TS_ERR_INVALID_ARG and "offsets" in e.value.detail
    lib.ts_sync_and_check()  # reported once


def test_grouped_empty_sum(lib):
    off = torch.tensor([2, 5, 6], device="cuda")
    D = torch.full((8, 20), 4.0, device="cuda")
    z = lambda *s: torch.empty(s, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    lib.ts_gemm_fp8_grouped(z(8, 0), f(8, 0), z(2, 20, 0), f(2, 1, 0), D, off)
    lib.ts_sync_and_check()
    assert (D[2:6] == 0).all() and (D[:2] == 4).all() and (D[6:] == 4).all()


def test_refusals(lib):
    A, SA, B, SB, _, _ = _problem(64, 64, 64, 1, True)
    D = torch.empty((64, 64), device="cuda")
    with pytest.raises(TypeError):
        lib.ts_gemm_fp8(A.float(), SA, B, SB, D)
    with pytest.raises(TypeError):
        lib.ts_gemm_fp8(A, SA.double(), B, SB, D)
    with pytest.raises(TypeError):
        lib.ts_gemm_fp8(A.cpu(), SA, B, SB, D)
    with pytest.raises(TypeError):
        lib.ts_gemm_fp8(A, SA, B, SB, D.half())
    with pytest.raises(ValueError):
        lib.ts_gemm_fp8(A, SA, B[:, :48], SB, D)
    with pytest.raises(ValueError):
        lib.ts_gemm_fp8(A, SA[:32], B, SB, D)
    with pytest.raises(ValueError):
        lib.ts_gemm_fp8(A, SA, B, SB.expand(3, 1), D)
    with pytest.raises(ValueError):
        lib.ts_gemm_fp8(A.t(), SA, B, SB, D)
    with pytest.raises(lib.TsError) as e:  # rows of 72 bytes
        lib.ts_gemm_fp8(torch.zeros((64, 72), dtype=torch.float8_e4m3fn, device="cuda")[:, :64], SA, B, SB, D)
    assert e.value.status == lib.TS_ERR_UNSUPPORTED
    with pytest.raises(lib.TsError) as e:
        lib.ts_gemm_fp8(A[:16], SA[:16], B[:16], SB, A.view(torch.float32)[:16, :16])
    assert e.value.status == lib.TS_ERR_INVALID_ARG and "overlap" in e.value.detail
    B3, SB3 = B[None], SB[None]
    with pytest.raises(TypeError):
        lib.ts_gemm_fp8_grouped(A, SA, B3, SB3, D, torch.tensor([0, 64], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        lib.ts_gemm_fp8_grouped(A, SA, B3, SB3, D, torch.tensor([0, 1, 64], device="cuda"))
    lib.ts_sync_and_check()


def test_expanded_tensors(lib):
    # scales broadcast along one dimension are taken as they are; what cannot be told apart or shares rows is refused
    M, N, K = 130, 140, 300
    A, SA, B, SB, a, b = _problem(M, N, K, 13, True)
    one = SA[:, :1].contiguous()
    D = torch.empty((M, N), device="cuda")
    lib.ts_gemm_fp8(A, one.expand(M, 3), B, SB, D)
    lib.ts_sync_and_check()
    ref = (A.double().cpu() * one.double().cpu()) @ b
    assert torch.equal(D.cpu(), ref.float())
    row = SA[:1].contiguous()
    lib.ts_gemm_fp8(A, row.expand(M, 3), B, SB, D)
    lib.ts_sync_and_check()
    ref = (A.double().cpu() * _expand(row.double().cpu(), 1, K, 1)) @ b
    assert torch.equal(D.cpu(), ref.float())
    for bad in (lambda: lib.ts_gemm_fp8(A, SA[:1, :1].expand(M, 3), B, SB, D),
                lambda: lib.ts_gemm_fp8(A[:1].expand(M, K), SA, B, SB, D),
                lambda: lib.ts_gemm_fp8(A, SA, B, SB, D[:1].expand(M, N)),
                lambda: lib.ts_gemm_fp8_grouped(A, SA, B[None].expand(2, N, K), SB[None].repeat(2, 1, 1), D,
                                                torch.tensor([0, 10, M], device="cuda"))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("N,before,after", [(520, 8, 16), (520, 2, 8), (518, 1, 1), (517, 0, 0), (517, 8, 11), (393, 3, 1)])
def test_grouped_output_pitches(lib, N, before, after, tile, out):
    # D's rows and base on 16-, 4- and 2-byte boundaries; groups that end inside a warp's 32 rows
    off = [2, 70, 71, 71, 230, 262]
    M, K = off[-1] + 3, 200
    A, SA, B, SB, a, b = _problem(M, N, K, N + before, True, groups=len(off) - 1)
    wide = torch.full((M, before + N + after), -777.0, dtype=out, device="cuda")
    D = wide[:, before:before + N]
    lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, torch.tensor(off, device="cuda"), tile=tile)
    lib.ts_sync_and_check()
    ref = torch.full(wide.shape, -777.0, dtype=torch.float64)
    ref[off[0]:off[-1], before:before + N] = _grouped_ref(off, a, b, N)[off[0]:off[-1]]
    assert torch.equal(wide.cpu(), ref.to(out))


@pytest.mark.parametrize("workers", [1, 3, 7, 40])
def test_worker_cap(lib, workers):
    # few tiles and a long K: without a cap each tile's K blocks are shared by several workers
    M, N, K = 9, 300, 4096
    A, SA, B, SB, a, b = _problem(M, N, K, 21, True)
    D = torch.full((M, N), float("nan"), device="cuda")
    lib.ts_gemm_fp8(A, SA, B, SB, D, max_workers=workers)
    lib.ts_sync_and_check()
    _check(D, a @ b, None, K, True, f"{workers} workers")


def test_unsplit_results_are_the_same_on_every_tile_and_for_every_batch(lib):
    # (random values: the order of the fp32 sums is the K blocks' on every tile)
    off = [0, 30, 30, 211, 611]
    A, SA, B, SB, _, _ = _problem(off[-1], 520, 1000, 4, False, groups=4)
    o = torch.tensor(off, device="cuda")
    D = [torch.empty((off[-1], 520), device="cuda") for _ in range(4)]
    for d, tile in zip(D, ("128x128", "128x256", "256x256")):
        lib.ts_gemm_fp8_grouped(A, SA, B, SB, d, o, tile=tile)
    for g in range(4):  # eleven rows at a time, on short tiles
        for i in range(off[g], off[g + 1], 11):
            j = min(i + 11, off[g + 1])
            lib.ts_gemm_fp8_grouped(A[i:j], SA[i:j], B[g:g + 1], SB[g:g + 1], D[3][i:j],
                                    torch.tensor([0, j - i], device="cuda"))
    lib.ts_sync_and_check()
    for d in D[1:]:
        assert torch.equal(D[0], d)
