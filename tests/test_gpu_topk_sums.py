"""logits_topk: the log-sum-exp of rows whose logits, divided by the temperature, are
so large that one step of fp32 there is a factor of e^88 and more. The row's largest
term is 1 and nothing is above it, so that lse is that of the largest logit whatever
the steps below it; it is infinite only past fp32's range. Bounds: test_gpu_topk.py."""
import math

import pytest
import torch

from gpu_util import DEV, say
from test_gpu_topk import DT, check, logits

pytestmark = pytest.mark.gpu
V = 20011


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M", [1, 515])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_rows_of_one_low_value(dt, M, T):
    """Rows of nothing but the type's lowest value, or of -1e9, as a mask leaves them:
    several segments a row, and one."""
    for k in (1, 2, 64, 300, 1024):
        say(f"topk lowest {dt} M={M} T={T} k={k}")
        lse = check(torch.full((M, V), torch.finfo(DT[dt]).min, dtype=DT[dt], device=DEV), k, T)[2]
        assert bool(lse.isfinite().all())
        if dt != "f16":
            assert bool(check(torch.full((M, V), -1e9, dtype=DT[dt], device=DEV), k, 0.7)[2].isfinite().all())
            x = logits(k, M, V, dt)  # ... with one row of numbers among them, and the mask over half of another
            x[1:] = torch.finfo(DT[dt]).min
            x[0, ::2] = torch.finfo(DT[dt]).min
            assert bool(check(x, k, T)[2].isfinite().all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 600])
def test_large_quotients(dt, M):
    """The largest logit's product with log2(e) / T past 2^31: half a step of it is
    an exponent of 128."""
    for top, T in ((5e9, 1.0), (5.3e9, 0.7), (7.7e9, 1.0), (1e12, 1.0), (-9e9, 1.0), (100.0, 1e-8), (93.7, 3e-9), (9e29, 1e-8),
                   (3e38, 1.0), (-3e38, 1.0), (9e29, 1e-9), (-9e29, 1e-9)):
        for k in (1, 20, 300):
            say(f"topk top={top} T={T} {dt} M={M} k={k}")
            x = logits(k, M, V, dt)
            if top < 0:  # every logit far below 0
                x = x.float().abs().mul_(top * 1e-2).add_(top).to(DT[dt])
            else:
                at = torch.arange(M, device=DEV)
                x[at, (at * 7919 + 40) % V] = top
                x[at, (at * 104729 + 19000) % V] = top * 0.99
            check(x, k, T)


@pytest.mark.parametrize("dt", list(DT))
def test_the_least_temperatures(dt):
    """log2(e) / T past fp32's range."""
    for T in (1e-38, 1e-39, 1e-40):
        for M in (1, 600):
            say("topk T", T, dt, M)
            lse = check(torch.zeros(M, V, dtype=DT[dt], device=DEV), 7, T)[2]
            assert bool(((lse - math.log(V)).abs() < 1e-4).all())
            x = logits(5, M, V, dt)
            for y in (x, -x.abs() - 1):  # -1.0005 / 1e-38 is a number yet; the others are infinite
                check(y, 7, T)
