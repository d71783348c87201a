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


@pytest.mark.parametrize("pitch", [0, 256, 400])
@pytest.mark.parametrize("trans", [False, True])
def test_groups_of_one_row_through_the_c_entry(lib, trans, pitch):
    # B [groups][1][128] (or, K = 1, its transpose), the groups one after another at the row's pitch
    G, R, L = 5, 3, 128
    rng = torch.Generator().manual_seed(pitch + trans)
    step = pitch or L
    M, N, K = G * R, (L if trans else 1), (1 if trans else L)
    buf = torch.randint(-4, 5, (G, step), generator=rng).float()  # what lies between the groups is not zero
    B = buf.to(torch.float8_e4m3fn).cuda()
    a = torch.randint(-4, 5, (M, K), generator=rng).float()
    A = torch.zeros((M, -(-K // 16) * 16), dtype=torch.float8_e4m3fn, device="cuda")
    A[:, :K] = a.to(torch.float8_e4m3fn).cuda()
    SA, SB = torch.ones((1, M), device="cuda"), torch.full((G,), 2.0, device="cuda")
    off = torch.arange(0, M + 1, R, device="cuda")
    D = torch.full((M, N), float("nan"), device="cuda")
    o = lib.Fp8Opts(trans_b=int(trans), lda=A.shape[1], ldb=pitch)
    st = lib._lib.ts_gemm_fp8_grouped(A.data_ptr(), SA.data_ptr(), B.data_ptr(), SB.data_ptr(), D.data_ptr(),
                                      off.data_ptr(), G, M, N, K, lib.TS_OUT_F32, o,
                                      torch.cuda.current_stream().cuda_stream)
    assert st == lib.TS_OK, lib.ts_last_error_detail()
    lib.ts_sync_and_check()
    rows = buf[:, :L].repeat_interleave(R, 0)
    want = 2 * (a * rows if trans else (a * rows).sum(1, keepdim=True))
    assert torch.equal(D.cpu(), want)


def test_plans_of_threads_on_one_stream(lib):
    # more slots than one CTA sorts: each call is two launches that share the scratch it keeps
    import threading

    T, E, threads, calls = 9000, 64, 4, 30
    start, errors = threading.Barrier(threads, timeout=60), []

    def work(seed):
        try:
            g = torch.Generator().manual_seed(seed)
            e = [torch.randint(0, E, (T, 2), generator=g, dtype=torch.int32) for _ in range(calls)]
            dev = [x.cuda() for x in e]
            bufs = [_plan_buffers(T, 2, E) for _ in range(calls)]
            torch.cuda.synchronize()
            start.wait()
            for x, b in zip(dev, bufs):
                lib.ts_moe_plan(x, *b)  # all on the default stream
            torch.cuda.synchronize()
            for x, (_, order, _) in zip(e, bufs):
                assert torch.equal(order.cpu().long(), x.flatten().sort(stable=True).indices)
        except Exception as err:  # noqa: BLE001
            errors.append(err)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(threads)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    lib.ts_sync_and_check()
    assert not errors, errors[0]


def _captured_plan(lib, e, bufs, fork):
    """A graph of one plan, on a side stream that the capture forks to or that captures alone; then an
    allocation on the capturing stream, filled before the fork joins."""
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    main = torch.cuda.Stream()
    if fork:
        with torch.cuda.graph(graph, stream=main):
            side.wait_stream(main)
            lib.ts_moe_plan(e, *bufs, stream=side)
            other = [torch.empty(lib.ts_moe_plan_workspace(e.numel(), bufs[0].numel() - 1), dtype=torch.uint8,
                                 device="cuda").fill_(255) for _ in range(4)]
            main.wait_stream(side)
        return graph, other
    with torch.cuda.stream(main):
        graph.capture_begin(capture_error_mode="relaxed")
    with torch.cuda.stream(side):
        lib.ts_moe_plan(e, *bufs, stream=main)
    with torch.cuda.stream(main):
        graph.capture_end()
    return graph, None


@pytest.mark.parametrize("fork", [True, False])
def test_captured_plan_on_a_stream_that_is_passed(lib, fork):
    T, E = 20000, 64
    e = torch.randint(0, E, (T, 2), dtype=torch.int32, device="cuda")
    bufs, eager = _plan_buffers(T, 2, E), _plan_buffers(T, 2, E)
    lib.ts_moe_plan(e, *eager)
    torch.cuda.synchronize()
    graph, other = _captured_plan(lib, e, bufs, fork)
    for _ in range(10):
        bufs[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, eager))
    lib.ts_sync_and_check()
    assert other is None or all((o == 255).all() for o in other)


@pytest.mark.parametrize("form", ["block", "row"])
def test_scales_of_more_than_2_29_rows(lib, form):
    # four bytes a scale: the distance to the last one, in bytes, passes 2^31
    n = 2 ** 29 + 256
    codes = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    long = torch.zeros((n, 16), dtype=torch.uint8, device="cuda")
    long.view(-1, 4, 16)[:, :, 0] = codes
    long = long.view(torch.float8_e4m3fn)
    scales = torch.empty((1, n), device="cuda")
    scales.view(-1, 8)[:] = torch.tensor([1.0, 1.0, 1.0, 1.0, 2.0, 2.0, 2.0, 2.0], device="cuda")
    one = torch.ones((1, 16), device="cuda").to(torch.float8_e4m3fn)
    unit = torch.ones((1, 1), device="cuda")
    if form == "block":
        D = torch.full((n, 1), float("nan"), device="cuda")
        lib.ts_gemm_fp8(long, scales.t(), one, unit, D)
    else:
        D = torch.full((1, n), float("nan"), device="cuda")
        lib.ts_gemm_fp8(one, unit, long, scales.t(), D)
    lib.ts_sync_and_check()
    want = torch.tensor([1.0, 2.0, 3.0, 4.0, 2.0, 4.0, 6.0, 8.0], device="cuda")
    assert bool((D.view(-1, 8) == want).all())


@pytest.mark.parametrize("M,G,N", [(1280, 64, 300), (2 ** 29, 1024, 1)])
def test_disordered_groups_make_no_more_tiles_than_ordered_ones(lib, M, G, N):
    # offsets 0, M, 0, M, ...: every other group is all rows, and 512 of those have 2^31 tiles.  All groups
    # have the same weights, so it does not matter which of them writes a row.
    codes = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    A = torch.zeros((M, 16), dtype=torch.uint8, device="cuda")
    A.view(-1, 4, 16)[:, :, 0] = codes
    A = A.view(torch.float8_e4m3fn)
    SA = torch.full((1, M), 0.5, device="cuda").t()
    B = torch.ones((G, N, 16), device="cuda").to(torch.float8_e4m3fn)
    SB = torch.ones((G, -(-N // 128), 1), device="cuda")
    off = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    off[1::2] = M
    D = torch.full((M, N), float("nan"), device="cuda")
    lib.ts_gemm_fp8_grouped(A, SA, B, SB, D, off)
    with pytest.raises(lib.TsError) as err:
        lib.ts_sync_and_check()
    assert "offsets" in err.value.detail
    want = torch.tensor([[0.5], [1.0], [1.5], [2.0]], device="cuda")
    assert bool((D.view(-1, 4, N) == want).all())


def test_routing_scale_of_the_smallest_normal_number(lib):
    x = torch.zeros((1, 4), device="cuda")
    e, w = torch.empty((1, 2), dtype=torch.int32, device="cuda"), torch.empty((1, 2), device="cuda")
    lib.ts_moe_route(x, e, w, scale=2.0 ** -126)
    lib.ts_sync_and_check()
    assert w.tolist() == [[2.0 ** -127] * 2]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_gradient_of_chosen_scores_whose_reciprocal_overflows(lib, score):
    # chosen scores of some 6e-39 (softmax: experts that a bias chose, far below the largest logit)
    x = torch.full((3, 40), -88.0, device="cuda")
    x[:, 1::2] = -88.2
    if score == "softmax":
        x += 88.0
        x[:, 7] = 88.0 - 8.0 / 1024
    e = torch.tensor([[0, 1], [5, 38], [-1, 3]], dtype=torch.int32, device="cuda")
    gw = torch.tensor([[30.0, -20.0], [-5.0, 40.0], [3.0, 7.0]], device="cuda")
    gx = torch.full_like(x, float("nan"))
    lib.ts_moe_route_grad(x, e, gw, gx, score=score)
    lib.ts_sync_and_check()
    there = (e >= 0).double()
    xd = x.double()
    s = torch.sigmoid(xd) if score == "sigmoid" else torch.softmax(xd, 1)
    share = s.gather(1, e.clamp_min(0).long()) * there
    share = share / share.sum(1, keepdim=True)
    g = gw.double() * there
    v = (g - (g * share).sum(1, keepdim=True)) * share
    want = torch.zeros_like(xd).scatter_add_(1, e.clamp_min(0).long(), v)
    if score == "sigmoid":
        want *= torch.sigmoid(-xd)
    # a score: two units of expf and of the subnormal grid here (2^-22 each), a rounding or two; its share
    # twice that, the difference twice again
    assert bool(((gx.double() - want).abs() <= 2.0 ** -18 * gw.double().abs().amax()).all())


@pytest.mark.parametrize("form", ["block", "row"])
@pytest.mark.parametrize("a,b", [(100, -100), (-120, 126), (-100, -40), (60, 60), (0, -149)])
def test_scales_far_apart(lib, form, a, b):
    # powers of two whose product fp32 holds (a subnormal one too): the small whole numbers' sums stay exact
    M, N, K = 40, 200, 384
    g = torch.Generator().manual_seed(a)
    x, y = (torch.randint(-2, 3, s, generator=g).float() for s in ((M, K), (N, K)))
    A, B = x.to(torch.float8_e4m3fn).cuda(), y.to(torch.float8_e4m3fn).cuda()
    SA = torch.full((M, 3), 2.0 ** a, device="cuda")
    SB = torch.full((2 if form == "block" else N, 3), 2.0 ** b, device="cuda")
    D = torch.full((M, N), float("nan"), device="cuda")
    lib.ts_gemm_fp8(A, SA, B, SB, D)
    lib.ts_sync_and_check()
    assert torch.equal(D.double().cpu(), (x.double() @ y.double().t()) * 2.0 ** (a + b))
