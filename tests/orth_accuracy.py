"""How far ts_orthogonalise may be from its iteration in 64 bits, and how that is checked.

Relative to the result's Frobenius norm: the rounding of the result to bf16 takes at most 2^-8.  The roundings inside
the iteration (X, A and b A + c A^2 to fp16, 2^-12 of each value) have no useful worst-case bound, because each step
may raise an error 3.4445 times, so they are emulated: `emulated` rounds at the same places, and with five or seven
steps it is off by at most another 2^-8 on every matrix of these tests (test_orthogonalise_host.py holds it to that; it
finds 1.1e-3 to 3.7e-3).  Together 2^-7.  bf16 in the places of fp16 is off by more (8.7e-3 and up).

That is for the whole matrix; a wrong tile of a large one would hide in it.  So each block of 64 x 64 is held to twice
as much, 2^-6, of the norm that as many values have on average (the emulation's blocks reach 3.1e-3)."""
import torch

COEF = (3.4445, -4.7750, 2.0315)
SCALE = 4096.0
WHOLE, BLOCK = 2.0 ** -7, 2.0 ** -6


def same(x):
    return x


def to_fp16(x):
    return (x * SCALE).to(torch.float16).double() / SCALE


def to_bf16(x):
    return x.to(torch.bfloat16).double()


def iterate(g, steps=5, coef=COEF, eps=1e-7, inner=same, last=same):
    """The iteration on one matrix in 64 bits; `inner` rounds X, A and b A + c A^2, `last` the result."""
    a, b, c = coef
    x = g.double()
    x = x / (x.norm() + eps)
    if steps == 0:
        return last(x)
    tall = x.shape[0] > x.shape[1]
    x = inner(x.t() if tall else x)
    for i in range(steps):
        A = inner(x @ x.t())
        B = inner(b * A + c * A @ A)
        x = (last if i + 1 == steps else inner)(a * x + B @ x)
    return x.t() if tall else x


def emulated(g, steps=5, coef=COEF, eps=1e-7):
    return iterate(g, steps, coef, eps, to_fp16, to_bf16)


def errors(out, want):
    """Relative error of the whole, and the worst of a block of 64 x 64 against the norm its size has on average."""
    off, norm = out.double() - want, want.norm()
    R, C = want.shape
    sq = torch.nn.functional.pad(off.square(), (0, -C % 64, 0, -R % 64))
    blocks = sq.view(sq.shape[0] // 64, 64, sq.shape[1] // 64, 64).sum((1, 3))
    rows = torch.full((blocks.shape[0], 1), 64.0, dtype=torch.float64, device=off.device)
    cols = torch.full((1, blocks.shape[1]), 64.0, dtype=torch.float64, device=off.device)
    rows[-1], cols[0, -1] = R - 64 * (blocks.shape[0] - 1), C - 64 * (blocks.shape[1] - 1)
    worst = (blocks / (rows * cols)).max().sqrt() * (R * C) ** 0.5
    return float(off.norm() / norm), float(worst / norm)


def close(out, want):
    whole, block = errors(out, want)
    return whole <= WHOLE and block <= BLOCK  # false for NaNs


def check(out, g, steps=5, coef=COEF, eps=1e-7, what=""):
    want = iterate(g, steps, coef, eps)
    whole, block = errors(out, want)
    assert whole <= WHOLE and block <= BLOCK, f"{what}: off by {whole} of the norm, a block by {block}"


def matrix(R, C, seed, dtype=torch.bfloat16, lead=(), extra=0, size=1e-3, device="cpu"):
    """Noise with a part of rank three, as gradients have; `extra` columns of zeros behind each row."""
    g = torch.Generator(device).manual_seed(seed)
    u, v = (torch.randn((*lead, *s), device=device, generator=g) for s in ((R, 3), (3, C)))
    t = torch.zeros((*lead, R, C + extra), dtype=dtype, device=device)[..., :C]
    t.copy_(size * (torch.randn((*lead, R, C), device=device, generator=g) + 0.5 * u @ v))
    return t
