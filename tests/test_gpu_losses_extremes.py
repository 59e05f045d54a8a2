"""The losses where their inputs leave the ordinary range. Formulas and bounds:
tests/loss_formulas.py."""
import math

import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say
from test_gpu_losses import KW, call, check, make, reference

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


@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_an_advantage_that_is_no_number(M, kl):
    """NaN, or a ratio of 0 times infinity, inside and outside the clip: loss and
    gradient of the row are NaN, those of the others as without it."""
    c = make("policy", 5, M, 64, 200, "bf16", True, mask=0.0)
    kw = dict(KW["policy"], kl_coef=kl)
    reference(c, 0.5, kw)
    *clean, saved = call(c, 0.5, kw)
    dh = L.loss_backward(c["grad"], c["weight"], saved)[0]
    for bad, old in ((math.nan, 0.0), (math.nan, 30.0), (math.nan, -30.0), (math.inf, 200.0), (-math.inf, 200.0)):
        say("policy advantage", bad, "old", old, "kl", kl, "M", M)
        c2 = dict(c, advantage=c["advantage"].clone(), old=c["old"].clone())
        c2["advantage"][7] = bad
        c2["old"][7] = clean[1][7] + old  # r = e^-old
        loss, logp, saved = call(c2, 0.5, kw)
        gh, gw, gb = L.loss_backward(c["grad"], c["weight"], saved)
        others = torch.arange(M, device=DEV) != 7
        assert bool(loss[7].isnan()) and torch.equal(logp, clean[1]) and torch.equal(loss[others], clean[0][others])
        assert bool(gh[7].isnan().all()) and bool(gw.isnan().all()) and bool(gb.isnan().all())
        assert bool(gh[others].isfinite().all())
