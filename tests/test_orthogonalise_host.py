"""The check that ts_orthogonalise is held to: what it passes and what it must not pass."""
import pytest
import torch

from orth_accuracy import COEF, check, close, emulated, errors, iterate, matrix, to_bf16, to_fp16

SIZES = [(1, 50), (50, 1), (8, 8), (33, 65), (64, 200), (128, 128), (129, 127), (300, 300), (777, 130), (513, 640), (20, 20000)]


@pytest.mark.parametrize("R,C", SIZES + [(1, 1)])
@pytest.mark.parametrize("steps", [1, 5, 7])
def test_roundings_of_the_iteration(R, C, steps):
    """What the tolerance grants the roundings inside the iteration is what they take; it is met with them."""
    g = matrix(R, C, R * 1000 + C)
    want = iterate(g, steps)
    inside = iterate(g, steps, inner=to_fp16)
    assert float((inside - want).norm()) <= 2.0 ** -8 * float(want.norm())
    check(emulated(g, steps), g, steps)


@pytest.mark.parametrize("coef", [(2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)])
def test_other_coefficients(coef):
    g = matrix(160, 300, 4)
    check(emulated(g, 6, coef), g, 6, coef)


@pytest.mark.parametrize("R,C", SIZES)
def test_wrong_results_do_not_pass(R, C):
    g = matrix(R, C, R * 1000 + C)
    want = iterate(g)
    good = emulated(g)
    assert close(good, want)
    wrong = {"zeros": torch.zeros_like(want), "negated": -good, "a step too few": emulated(g, 4), "a step too many": emulated(g, 6),
             "NaN": torch.full_like(want, float("nan")), "another matrix's": emulated(matrix(R, C, 1)),
             "one percent larger": good * 1.01}
    if min(R, C) > 8:  # of a few values the roundings may cancel
        wrong["bf16 inside"] = iterate(g, inner=to_bf16, last=to_bf16)
    for name, out in wrong.items():
        assert not close(out, want), f"{name}: {errors(out, want)}"


@pytest.mark.parametrize("R,C", [(300, 300), (513, 640), (777, 130)])
def test_wrong_places_do_not_pass(R, C):
    """A tile, a row or a column that is missing, or a neighbour's; the last row shifted by one."""
    g = matrix(R, C, 7)
    want, good = iterate(g), emulated(g)
    for part in ((slice(64, 128), slice(64, 128)), (slice(R - 4, R), slice(None)), (slice(None), slice(C - 2, C)),
                 (slice(0, 32), slice(32, 64))):
        out = good.clone()
        out[part] = 0
        assert not close(out, want)
        out = good.clone()
        out[part] = good.roll(1, 1)[part]
        assert not close(out, want)


def test_wrong_formulas_do_not_pass():
    g = matrix(200, 300, 9)
    want = iterate(g)
    a, b, c = COEF
    for coef in ((a, b, c * 1.02), (a, b * 1.02, c), (a * 1.02, b, c), (a, c, b)):
        assert not close(iterate(g, coef=coef, last=to_bf16), want)
