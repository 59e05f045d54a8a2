"""The losses where their inputs leave the ordinary range. Formulas and bounds:
tests/loss_formulas.py."""
import pytest

from gpu_util import say
from test_gpu_losses import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [33, 300])
@pytest.mark.parametrize("dt,k", [("bf16", 1e-31), ("bf16", 1e31), ("f16", 1e-31)])
def test_upstream_gradients_without_a_scale(dt, k, M):
    """Coefficients outside 1e-30 .. 1e30, under which G has no scale: what the
    teacher's entries add to grad_bias is there all the same."""
    c = make("distill", 23, M, 64, 150, dt, True)
    c["grad"] *= k
    say("no scale", dt, k, M)
    check(c)
