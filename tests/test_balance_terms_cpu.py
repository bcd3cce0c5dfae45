"""What the element-by-element test of the balance losses' gradient tells apart:
gradients with a term left out, at each of its shapes."""
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_balance_terms import SHAPES, BF16, F16, F32, expected, make, terms  # noqa: E402


@pytest.mark.parametrize("T, E, k, cuts", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_a_gradient_without_a_term_is_found(T, E, k, cuts, dtype):
    l, ids, counts, tokens, dloss, dz = make(T, E, k, cuts, dtype)
    t = terms(l, ids, cuts, counts, tokens, dloss, dz)
    want, tol = expected(t, dtype, E)
    af, am, bl, b = t
    # elements with a gradient at all
    live = b != 0
    for name, wrong in [("nothing", torch.zeros_like(want)), ("no mean", af + bl), ("no shares", bl - am), ("no z", af - am),
                        ("half of z", af - am + bl / 2)]:
        found = ((wrong - want).abs() > tol)[live].double().mean()
        print(name, float(found))
        # (an expert without tokens has no share to leave out)
        least = 0.9 * float((af != 0)[live].double().mean()) if name == "no shares" else 0.9
        assert found >= least, "%s: %.3f of the wrong elements found" % (name, float(found))
