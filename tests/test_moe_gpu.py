"""Routing, planning, 8-bit quantisation and the combine, against references in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

NEG = float("-inf")


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ routing
def _route_ref(x, k, score, bias=None, groups=1, keep=0, best=1, renorm=True, scale=1.0):
    """Experts and weights of logits x (float64), and the gap below which a choice could go either way."""
    T, E = x.shape
    keep = keep or groups
    masked = ~(x > NEG)
    if score == "sigmoid":
        s = 1 / (1 + np.exp(-np.where(masked, 0, x)))
    else:
        top = np.max(np.where(masked, -1e300, x), 1, keepdims=True)
        e = np.where(masked, 0, np.exp(np.where(masked, 0, x - top)))
        s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    s = np.where(masked, 0, s)
    c = np.where(masked, NEG, s + (0 if bias is None else bias))
    gap = np.full(T, np.inf)
    if groups > 1:
        n = E // groups
        o = -np.sort(-c.reshape(T, groups, n), 2)
        gs = o[:, :, 0].copy()
        if best == 2 and n > 1:
            gs = np.where(o[:, :, 1] > NEG, gs + o[:, :, 1], gs)
        order = np.argsort(-gs, 1, kind="stable")
        if keep < groups:
            r = np.take_along_axis(gs, order, 1)
            with np.errstate(invalid="ignore"):
                d = r[:, keep - 1] - r[:, keep]
            gap = np.minimum(gap, np.where(np.isnan(d) | (d == 0), np.inf, d))
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, order[:, :keep], True, 1)
        c = np.where(np.repeat(kept, n, 1), c, NEG)
    order = np.argsort(-c, 1, kind="stable")
    r = np.take_along_axis(c, order, 1)
    m = min(k + 1, E)
    with np.errstate(invalid="ignore"):
        d = r[:, :m - 1] - r[:, 1:m]
    d = np.where(np.isnan(d) | (d == 0), np.inf, d)
    if d.size:
        gap = np.minimum(gap, d.min(1))
    e = np.where(r[:, :k] > NEG, order[:, :k], -1)
    w = np.where(e >= 0, np.take_along_axis(s, order[:, :k], 1), 0)
    if renorm:
        t = w.sum(1, keepdims=True)
        w = np.where(t > 0, w / np.maximum(t, 1e-300), 0)
    return e.astype(np.int32), w * scale, s, gap


def _run_route(lib, x, k, **kw):
    T = x.shape[0]
    e = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    lib.ts_moe_route(x, e, w, **kw)
    lib.ts_sync_and_check()
    return e, w


ROUTES = [
    dict(T=1, E=256, k=8, score="sigmoid", groups=8, keep_groups=4, group_best=2, bias=True, scale=2.5),
    dict(T=33, E=1, k=1, score="softmax"), dict(T=5, E=7, k=7, score="softmax"),
    dict(T=64, E=32, k=4, score="sigmoid", renorm=False), dict(T=17, E=33, k=3, score="softmax", renorm=False),
    dict(T=129, E=64, k=6, score="softmax", bias=True), dict(T=100, E=160, k=6, score="softmax", groups=8, keep_groups=3),
    dict(T=50, E=96, k=32, score="sigmoid", groups=32, keep_groups=16, group_best=2),
    dict(T=41, E=512, k=8, score="sigmoid", bias=True), dict(T=40, E=1000, k=10, score="softmax", groups=4, keep_groups=1),
    dict(T=9, E=1024, k=2, score="sigmoid", groups=2, keep_groups=1, group_best=1, bias=True),
    dict(T=2000, E=128, k=2, score="softmax"), dict(T=11, E=12, k=5, score="sigmoid", groups=12, keep_groups=5, group_best=2),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masks", [False, True])
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route(lib, case, masks, dtype):
    kw = dict(ROUTES[case])
    T, E, k = kw.pop("T"), kw.pop("E"), kw.pop("k")
    g = torch.Generator().manual_seed(case)
    x = (2 * torch.randn((T, E), generator=g)).to(dtype)
    if masks:
        x = x.masked_fill(torch.rand((T, E), generator=g) < 0.4, NEG)
        x[T // 2] = NEG  # nothing is left
        x[0, E // 2] = torch.finfo(dtype).min  # a mask of the type's lowest value: still a number
    b = torch.round(30 * torch.randn(E, generator=g)) * 0.001 if kw.pop("bias", False) else None
    e, w = _run_route(lib, x.cuda(), k, bias=None if b is None else b.cuda(), **kw)
    ref = {"keep": kw.get("keep_groups", 0), "best": kw.get("group_best", 1), "groups": kw.get("groups", 1),
           "renorm": kw.get("renorm", True), "scale": kw.get("scale", 1.0)}
    re_, rw, s, gap = _route_ref(x.double().numpy(), k, kw["score"], None if b is None else b.double().numpy(), **ref)
    # Scores carry a few roundings (exp within 2 units, a sum of depth 10, a division, the bias): two that are
    # nearer than 2^-19 may come in either order in fp32.  Equal ones (gap inf or exact ties) may not.
    sure = torch.from_numpy(gap > 2.0 ** -19)
    assert sure.float().mean() > 0.7
    e, w = e.cpu(), w.cpu().double()
    assert torch.equal(e[sure], torch.from_numpy(re_)[sure])
    rw = torch.from_numpy(rw)
    assert bool(((w - rw).abs()[sure] <= 2.0 ** -18 * rw.abs()[sure] + 1e-37).all())
    if masks and T > 1:  # a single row is row 0, which has an expert again
        assert (e[T // 2] == -1).all() and (w[T // 2] == 0).all()


def test_route_ties_go_to_the_lowest_index(lib):
    x = torch.zeros((3, 200), device="cuda")
    x[1, 150:] = 1.0
    x[2, ::7] = -1.0
    e, w = _run_route(lib, x, 5)
    assert e.tolist() == [[0, 1, 2, 3, 4], [150, 151, 152, 153, 154], [1, 2, 3, 4, 5]]
    assert torch.allclose(w, torch.full_like(w, 0.2), rtol=1e-6)
    e, _ = _run_route(lib, x[:1], 5, score="sigmoid", groups=8, keep_groups=2, group_best=2)
    assert e.tolist() == [[0, 1, 2, 3, 4]]
    # -0.0 and +0.0 are equal choices
    b = torch.full((200,), -0.5, device="cuda")  # sigmoid(0) - 0.5 = 0
    b[3] = -0.5
    e, _ = _run_route(lib, x[:1], 3, score="sigmoid", bias=b)
    assert e.tolist() == [[0, 1, 2]]


def test_route_infinities_and_not_a_number(lib):
    x = torch.zeros((4, 40), device="cuda")
    x[0, 5] = float("inf")
    x[1, 6] = float("nan")
    x[2, :] = float("nan")
    x[3, 39] = -1e38
    for score in ("softmax", "sigmoid"):
        e, w = _run_route(lib, x, 2, score=score)
        assert e[0].tolist() == [5, 0] and torch.isfinite(w[0]).all()
        assert e[1].tolist() == [0, 1] and torch.isnan(w[1]).all()
        assert e[2].tolist() == [-1, -1] and torch.isnan(w[2]).all()
        assert e[3].tolist() == [0, 1]


def test_route_choice_is_the_definition_to_the_bit(lib):
    # near ties by the thousand: the choice must be that of the fp32 definition, operation by operation
    T, E, k = 4096, 256, 8
    x = 1.5 * torch.randn((T, E), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    b = 0.001 * torch.round(30 * torch.randn(E, device="cuda", generator=torch.Generator("cuda").manual_seed(2)))
    for score in ("sigmoid", "softmax"):
        if score == "sigmoid":
            s = torch.reciprocal(1 + torch.exp(-x))
        else:
            p = torch.exp(x - x.amax(1, keepdim=True))
            t = p
            while t.shape[1] > 1:
                t = t[:, :t.shape[1] // 2] + t[:, t.shape[1] // 2:]
            s = p / t
        ref = (s + b).sort(dim=1, descending=True, stable=True).indices[:, :k]
        e, _ = _run_route(lib, x, k, score=score, bias=b)
        assert torch.equal(e, ref.to(torch.int32)), score


def test_route_strided_rows(lib):
    wide = torch.randn((20, 100), device="cuda")
    x = wide[:, 7:70]
    e, w = _run_route(lib, x, 4)
    e2, w2 = _run_route(lib, x.contiguous(), 4)
    assert torch.equal(e, e2) and torch.equal(w, w2)


def _grad_ref(x, e, gw, score, renorm, scale):
    """By torch's differentiation in 64 bits."""
    x = x.clone().requires_grad_(True)
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    there = e >= 0
    w = torch.where(there, s.gather(1, e.clamp_min(0).long()), torch.zeros((), dtype=x.dtype))
    if renorm:
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / torch.where(t > 0, t, torch.ones_like(t)), torch.zeros_like(w))
    (scale * w * gw).sum().backward()
    return x.grad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (37, 64, 6), (20, 300, 8), (9, 1024, 32), (6, 5, 5)])
def test_route_grad(lib, T, E, k, score, renorm, dtype):
    g = torch.Generator().manual_seed(E + k)
    x = (2 * torch.randn((T, E), generator=g)).to(dtype)
    x[T // 2, : E // 2] = -40.0 if dtype == torch.float32 else -20.0
    xc = x.cuda()
    e, _ = _run_route(lib, xc, k, score=score)
    e[0, k - 1] = -1  # a dropped slot
    gw = torch.randn((T, k), generator=g)
    gx = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    lib.ts_moe_route_grad(xc, e, gw.cuda(), gx, score=score, renorm=renorm, scale=1.5)
    lib.ts_sync_and_check()
    ref = _grad_ref(x.double(), e.cpu(), gw.double(), score, renorm, 1.5)
    # differences of terms of size |g| / S: 2^-18 of the largest term per row, and the output's rounding
    row = (1.5 * gw.double().abs()).amax(1, keepdim=True)
    s = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), 1)
    S = torch.where(e.cpu() >= 0, s.gather(1, e.cpu().clamp_min(0).long()), torch.zeros((), dtype=torch.float64)).sum(1, keepdim=True)
    bound = 2.0 ** -18 * k * row * (2 / S if renorm else 1) * s + (2.0 ** -8 if dtype == torch.bfloat16 else 0) * ref.abs()
    assert bool(((gx.double().cpu() - ref).abs() <= bound + 1e-30).all())


def test_route_grad_against_differences(lib):
    T, E, k, h = 6, 24, 4, 1e-2
    x = torch.randn((T, E), device="cuda")
    gw = torch.randn((T, k), device="cuda")
    for score in ("softmax", "sigmoid"):
        e, _ = _run_route(lib, x, k, score=score)
        gx = torch.empty_like(x)
        lib.ts_moe_route_grad(x, e, gw, gx, score=score)
        lib.ts_sync_and_check()

        def value(y):
            s = torch.sigmoid(y) if score == "sigmoid" else torch.softmax(y, 1)
            w = s.gather(1, e.long())
            return (w / w.sum(1, keepdim=True) * gw.double()).sum(1)

        xd = x.double()
        for c in range(E):
            d = torch.zeros_like(xd)
            d[:, c] = h
            num = (value(xd + d) - value(xd - d)) / (2 * h)
            # central differences: the third derivative of these functions is below 8 |g|
            assert bool(((num - gx[:, c].double()).abs() <= 8 * gw.abs().amax() * h * h + 1e-6).all())


def test_route_refusals(lib):
    x = torch.zeros((4, 32), device="cuda")
    e = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    for kw in (dict(groups=5), dict(groups=4, keep_groups=5), dict(groups=16, keep_groups=0, group_best=3),
               dict(score=7), dict(groups=32, keep_groups=1)):
        with pytest.raises(lib.TsError) as err:
            lib.ts_moe_route(x, e, w, **kw)
        assert err.value.status == lib.TS_ERR_INVALID_ARG
    with pytest.raises(lib.TsError) as err:
        lib.ts_moe_route(torch.zeros((4, 2048), device="cuda"), e, w)
    assert err.value.status == lib.TS_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        lib.ts_moe_route(x.half(), e, w)
    with pytest.raises(ValueError):
        lib.ts_moe_route(x, e, w[:3])
    with pytest.raises(TypeError):
        lib.ts_moe_route(x, e.long(), w)
    with pytest.raises(ValueError):
        lib.ts_moe_route(x, e, w, scale=0.0)
    with pytest.raises(ValueError):
        lib.ts_moe_route_grad(x, e, w, x, scale=0.0)
    # an expert index past the last is reported, and gives nothing
    e[1, 0] = 32
    gx = torch.full((4, 32), 1.0, device="cuda")
    lib.ts_moe_route_grad(x, e, torch.ones((4, 2), device="cuda"), gx, renorm=False)
    with pytest.raises(lib.TsError) as err:
        lib.ts_sync_and_check()
    assert "expert" in err.value.detail


# --------------------------------------------------------------------- plan
@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 256), (100, 3, 5), (2048, 1, 7), (1000, 8, 64),
                                   (1025, 8, 1024), (8191, 6, 128), (20000, 2, 3), (70001, 1, 300),
                                   (1200, 2, 700), (40000, 2, 760), (70000, 1, 640), (66000, 1, 1024), (300000, 1, 33)])
def test_plan(lib, T, k, E):
    g = torch.Generator().manual_seed(T + E)
    e = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    if E > 4:
        e[e == 2] = 3  # an expert without slots
    off = torch.full((E + 1,), -5, dtype=torch.int64, device="cuda")
    order = torch.full((T * k,), -5, dtype=torch.int32, device="cuda")
    pos = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    lib.ts_moe_plan(e.cuda(), off, order, pos)
    lib.ts_sync_and_check()
    key = torch.where(e < 0, E, e).flatten().long()
    ref = key.sort(stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    n = int(counts.sum())
    assert off.cpu().tolist() == [0] + counts.cumsum(0).tolist()
    assert torch.equal(order.cpu()[:n].long(), ref[:n]) and (order[n:] == -1).all()
    want = torch.full((T * k,), -1, dtype=torch.int32)
    want[ref[:n]] = torch.arange(n, dtype=torch.int32)
    assert torch.equal(pos.cpu().flatten(), want)


def test_plan_reports_an_expert_past_the_last(lib):
    e = torch.tensor([[0, 9], [1, 0]], dtype=torch.int32, device="cuda")
    off = torch.empty(3, dtype=torch.int64, device="cuda")
    order = torch.empty(4, dtype=torch.int32, device="cuda")
    pos = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    lib.ts_moe_plan(e, off, order, pos)
    with pytest.raises(lib.TsError) as err:
        lib.ts_sync_and_check()
    assert "slot 1" in err.value.detail
    assert off.tolist() == [0, 2, 3] and order.tolist() == [0, 3, 2, -1] and pos.tolist() == [[0, -1], [2, 1]]


def test_plan_in_graphs_that_replay_at_once(lib):
    # many slots, no workspace passed: each graph has its own
    T, E = 30000, 64
    runs = []
    for i in range(2):
        e = torch.randint(0, E, (T, 2), generator=torch.Generator().manual_seed(i), dtype=torch.int32).cuda()
        off = torch.empty(E + 1, dtype=torch.int64, device="cuda")
        order = torch.empty(T * 2, dtype=torch.int32, device="cuda")
        pos = torch.empty((T, 2), dtype=torch.int32, device="cuda")
        lib.ts_moe_plan(e, off, order, pos)
        lib.ts_sync_and_check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.ts_moe_plan(e, off, order, pos)
        runs.append((graph, order, order.clone(), torch.cuda.Stream(), e, off, pos))
    for _, order, *_ in runs:
        order.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, _, _, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    lib.ts_sync_and_check(runs[0][3])
    torch.cuda.synchronize()
    for _, order, want, *_ in runs:
        assert torch.equal(order, want)


# ----------------------------------------------------------------- quantise
TOPS = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


def _quant_ref(x, dtype):
    """x [r, c] on the device, fp32: the definition's q and scales, each operation rounded to fp32."""
    r, c = x.shape
    nb = _cdiv(c, 128)
    v = torch.nn.functional.pad(x, (0, nb * 128 - c)).view(r, nb, 128)
    a = v.abs().amax(2).clamp_min(2.0 ** -100)
    f = torch.full_like(a, TOPS[dtype]) / a
    q = (v * f[:, :, None]).clamp(-TOPS[dtype], TOPS[dtype]).view(r, -1)[:, :c].to(dtype)
    return q, a.double() / TOPS[dtype]


def _same_quant(q, s, x, dtype):
    rq, rs = _quant_ref(x, dtype)
    assert torch.equal(q.float(), rq.float())
    assert bool(((s.double() - rs).abs() <= 2.0 ** -24 * rs).all())
    # and what it is for: x within half a step of the 8-bit grid (a normal number's, or the smallest)
    bits = 4 if dtype == torch.float8_e4m3fn else 3
    least = 2.0 ** -10 if dtype == torch.float8_e4m3fn else 2.0 ** -17
    back = q.double() * s.double().repeat_interleave(128, 1)[:, :x.shape[1]]
    step = torch.maximum(x.double().abs() * 2.0 ** -bits, s.double().repeat_interleave(128, 1)[:, :x.shape[1]] * least)
    assert bool(((back - x.double()).abs() <= step * (1 + 2.0 ** -20)).all())


def _x(r, c, dtype, seed, pitch=0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((r, c + pitch), device="cuda", generator=g) * torch.exp(3 * torch.randn((r, 1), device="cuda", generator=g))
    x[: r // 3, : c // 2] = 0  # whole blocks of zeros
    return x.to(dtype)[:, :c]


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("r,c,pitch", [(1, 1, 0), (1, 128, 0), (3, 130, 0), (16, 1024, 0), (17, 1000, 3), (129, 257, 8),
                                       (300, 64, 0), (65, 2048, 0), (128, 4104, 0)])
def test_quant(lib, r, c, pitch, transpose, dtype, fmt):
    x = _x(r, c, dtype, r + c, pitch)
    qr, qc = (c, r) if transpose else (r, c)
    wide = torch.full((qr, qc + pitch), 1.0, device="cuda").to(fmt)
    q = wide[:, :qc]
    s = torch.full((_cdiv(qc, 128), qr), float("nan"), device="cuda").t()
    lib.ts_quant_fp8(x, q, s, transpose=transpose)
    lib.ts_sync_and_check()
    _same_quant(q, s, x.float().t() if transpose else x.float(), fmt)
    assert (wide[:, qc:].float() == 1).all(), "the pitch's padding was written"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quant_gather(lib, dtype):
    x = _x(40, 520, dtype, 3)
    rows = torch.randint(0, 120, (1000,), device="cuda", dtype=torch.int32)
    rows[::9] = -1
    q = torch.ones((1000, 528), device="cuda").to(torch.float8_e4m3fn)[:, :520]
    s = torch.empty((1000, 5), device="cuda")  # blocks contiguous
    lib.ts_quant_fp8(x, q, s, rows=rows, rows_div=3)
    lib.ts_sync_and_check()
    there = rows >= 0
    _same_quant(q[there], s[there], x.float()[(rows[there] // 3).long()], torch.float8_e4m3fn)
    assert (q[~there].float() == 0).all() and (s[~there] == 0).all()
    # a row past the input: reported, and zeros
    rows[5] = 120
    lib.ts_quant_fp8(x, q, s, rows=rows, rows_div=3)
    with pytest.raises(lib.TsError) as err:
        lib.ts_sync_and_check()
    assert "output row 5" in err.value.detail and (q[5].float() == 0).all()


@pytest.mark.parametrize("transpose", [False, True])
def test_quant_extremes(lib, transpose):
    x = torch.zeros((256, 256), device="cuda")
    x[0, 0] = float("nan")
    x[0, 1] = 3.0
    x[130, 130] = float("inf")
    x[5, 140] = 3e38
    x[6, 141] = 1e-42  # below the least amax: not scaled up to the top
    x[140, 6] = 1e-36  # below 2^-100 too
    q = torch.empty((256, 256), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((256, 2), device="cuda")
    lib.ts_quant_fp8(x, q, s, transpose=transpose)
    lib.ts_sync_and_check()
    at = (lambda i, j: (j, i)) if transpose else (lambda i, j: (i, j))
    f = q.float()
    assert torch.isnan(f[at(0, 0)]) and torch.isnan(f).sum() == 2  # the NaN, and inf * 0
    if not transpose:
        assert f[0, 1] == 448 and torch.isinf(s[130, 1])
    assert torch.isfinite(s).sum() == s.numel() - 1
    assert f[at(5, 140)] == 448 and f[at(140, 6)] == 0 and f[at(6, 141)] == 0


def test_quant_refusals(lib):
    x = torch.zeros((4, 256), device="cuda")
    q = torch.zeros((4, 256), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros((4, 2), device="cuda")
    rows = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: lib.ts_quant_fp8(x.half(), q, s), lambda: lib.ts_quant_fp8(x, q.float(), s),
                lambda: lib.ts_quant_fp8(x, q, s.double()), lambda: lib.ts_quant_fp8(x, q, s, rows=rows.long())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lib.ts_quant_fp8(x, q[:3], s), lambda: lib.ts_quant_fp8(x, q, s[:, :1]),
                lambda: lib.ts_quant_fp8(x, q, s, transpose=True), lambda: lib.ts_quant_fp8(x.t(), q, s),
                lambda: lib.ts_quant_fp8(x, q, s, rows=rows, rows_div=0),
                lambda: lib.ts_quant_fp8(x, q, s, rows=rows, transpose=True)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib.TsError) as err:
        lib.ts_quant_fp8(x, x.view(torch.float8_e4m3fn)[:, :256], s)
    assert err.value.status == lib.TS_ERR_INVALID_ARG and "overlap" in err.value.detail
    lib.ts_quant_fp8(x[:0], q[:0], s[:0])
    lib.ts_sync_and_check()


# ------------------------------------------------------------------ combine
def _combine_inputs(T, k, N, dtype, seed, pitch=0):
    g = torch.Generator("cuda").manual_seed(seed)
    R = T * k + 3
    y = torch.randn((R, N + pitch), device="cuda", generator=g).to(dtype)[:, :N]
    pos = torch.randperm(R, device="cuda", generator=g)[:T * k].to(torch.int32).view(T, k)
    pos = torch.where(torch.rand((T, k), device="cuda", generator=g) < 0.2, torch.full_like(pos, -1), pos)
    if T:
        pos[T // 2] = -1  # every slot dropped
    w = torch.randn((T, k), device="cuda", generator=g)
    go = torch.randn((T, N + pitch), device="cuda", generator=g).to(dtype)[:, :N]
    return y, pos, w, go


COMBINES = [(1, 1, 1, 0), (3, 2, 8, 0), (7, 8, 100, 0), (5, 9, 2048, 0), (33, 20, 4104, 8), (300, 4, 257, 1), (64, 3, 4096, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,N,pitch", COMBINES)
def test_combine(lib, T, k, N, pitch, weighted, dtype):
    y, pos, w, _ = _combine_inputs(T, k, N, dtype, N + k, pitch)
    out = torch.full((T, N + pitch), 5.0, dtype=dtype, device="cuda")
    lib.ts_moe_combine(y, pos, out[:, :N], weights=w if weighted else None)
    lib.ts_sync_and_check()
    wj = torch.where(pos >= 0, w.double() if weighted else 1.0, 0.0)
    rows = y.double()[pos.clamp_min(0).long()] * wj[:, :, None]
    ref, mag = rows.sum(1), rows.abs().sum(1)
    # k fused multiply-adds in fp32, then the output's rounding
    bound = k * 2.0 ** -24 * mag + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * ref.abs() + 1e-37
    assert bool(((out[:, :N].double() - ref).abs() <= bound).all())
    assert (out[:, N:] == 5).all() and (out[T // 2, :N] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,N,pitch", COMBINES)
def test_combine_grad(lib, T, k, N, pitch, weighted, dtype):
    y, pos, w, go = _combine_inputs(T, k, N, dtype, N + k, pitch)
    gy = torch.full((y.shape[0], N + pitch), 7.0, dtype=dtype, device="cuda")
    gw = torch.full((T, k), float("nan"), device="cuda")
    lib.ts_moe_combine_grad(go, y, pos, w if weighted else None, gy[:, :N], gw)
    lib.ts_sync_and_check()
    there = pos >= 0
    rows = y.double()[pos.clamp_min(0).long()]
    prod = torch.where(there[:, :, None], rows * go.double()[:, None, :], 0.0)
    # at most N fused multiply-adds in a chain, more in the tree
    bound = (N + 16) * 2.0 ** -24 * prod.abs().sum(2) + 1e-37
    assert bool(((gw.double() - prod.sum(2)).abs() <= bound).all())
    ref = torch.full_like(gy[:, :N], 7.0)
    scaled = go.float()[:, None, :] * (w if weighted else torch.ones_like(w))[:, :, None]
    ref[pos[there].long()] = scaled[there].to(dtype)
    assert torch.equal(gy[:, :N], ref), "grad_y differs, or a row that no slot takes was written"
    assert (gy[:, N:] == 7).all()


def test_combine_grad_against_differences(lib):
    T, k, N, h = 4, 3, 16, 1e-2
    y, pos, w, go = _combine_inputs(T, k, N, torch.float32, 5)
    gy = torch.zeros_like(y)
    gw = torch.zeros_like(w)
    lib.ts_moe_combine_grad(go, y, pos, w, gy, gw)
    lib.ts_sync_and_check()

    def value(yy, ww):
        out = torch.empty((T, N), device="cuda")
        lib.ts_moe_combine(yy, pos, out, weights=ww)
        return float((out.double() * go.double()).sum())

    # the function is linear in each of y and w: differences are exact but for rounding
    for i in range(T):
        for j in range(k):
            d = torch.zeros_like(w)
            d[i, j] = h
            assert abs((value(y, w + d) - value(y, w - d)) / (2 * h) - float(gw[i, j])) < 2e-3
    for r in range(0, y.shape[0], 3):
        d = torch.zeros_like(y)
        d[r, r % N] = h
        assert abs((value(y + d, w) - value(y - d, w)) / (2 * h) - float(gy[r, r % N])) < 2e-3


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,N", [(5, 3, 31), (5, 3, 33), (9, 9, 1023), (9, 5, 1025), (3, 8, 2049), (3, 1, 4095),
                                   (9, 5, 1026), (7, 9, 444), (5, 2, 36), (5, 2, 6), (4, 3, 4092)])
def test_combine_odd_rows(lib, T, k, N, dtype):
    # rows off the 16-byte grid: dense rows of odd length, of 2 or 4 values more, and a base off it
    y, pos, w, go = _combine_inputs(T, k, N, dtype, N, 0)
    flat = torch.full((T * N + 2,), 5.0, dtype=dtype, device="cuda")
    out = flat[1:-1].view(T, N)
    lib.ts_moe_combine(y, pos, out, weights=w)
    aligned = torch.empty((T, N), dtype=dtype, device="cuda")
    lib.ts_moe_combine(y, pos, aligned, weights=w)
    assert torch.equal(out, aligned)
    gy, gw = torch.full_like(y, 7.0), torch.empty_like(w)
    lib.ts_moe_combine_grad(go, y, pos, w, gy, gw)
    lib.ts_sync_and_check()
    there = pos >= 0
    rows = y.double()[pos.clamp_min(0).long()] * there[:, :, None]
    terms = rows * w.double()[:, :, None]
    ref, mag = terms.sum(1), terms.abs().sum(1)
    # k fused multiply-adds in fp32, then the output's rounding
    bound = k * 2.0 ** -24 * mag + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * ref.abs() + 1e-37
    assert bool(((out.double() - ref).abs() <= bound).all())
    assert flat[0] == 5 and flat[-1] == 5
    prod = rows * go.double()[:, None, :]
    assert bool(((gw.double() - prod.sum(2)).abs() <= (N + 16) * 2.0 ** -24 * prod.abs().sum(2) + 1e-37).all())
    want = torch.full_like(y, 7.0)
    want[pos[there].long()] = (go.float()[:, None, :] * w[:, :, None])[there].to(dtype)
    assert torch.equal(gy, want)


def test_combine_refusals(lib):
    y, pos, w, go = _combine_inputs(4, 2, 64, torch.float32, 1)
    out = torch.zeros((4, 64), device="cuda")
    for bad in (lambda: lib.ts_moe_combine(y, pos, out.bfloat16()), lambda: lib.ts_moe_combine(y, pos.long(), out),
                lambda: lib.ts_moe_combine(y, pos, out, weights=w.double()), lambda: lib.ts_moe_combine(y.half(), pos, out)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lib.ts_moe_combine(y, pos, out[:3]), lambda: lib.ts_moe_combine(y, pos, out, weights=w[:3]),
                lambda: lib.ts_moe_combine(y, pos, out[:, :63])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib.TsError) as err:
        lib.ts_moe_combine(y, pos, y[:4])
    assert err.value.status == lib.TS_ERR_INVALID_ARG
    pos[1, 1] = y.shape[0]
    lib.ts_moe_combine(y, pos, out, weights=w)
    with pytest.raises(lib.TsError) as err:
        lib.ts_sync_and_check()
    assert "slot 3" in err.value.detail
