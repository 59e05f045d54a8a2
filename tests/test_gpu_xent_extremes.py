"""Softmax cross entropy where fp32's range or precision ends: masks of the
type's lowest value, logits near its largest, against the formula in 64 bits."""
import math

import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F = torch.finfo(torch.float32)
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def grid(seed, M, H, V, dt):
    """Inputs whose products and sums over H are exact in fp32: hidden in
    quarters up to 1, weight in eighths up to 1/2, 32 (128 H) < 2^24."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randint(-4, 5, (M, H), generator=g).div(4).to(DT[dt]).to(DEV)
    W = torch.randint(-4, 5, (V, H), generator=g).div(8).to(DT[dt]).to(DEV)
    y = torch.randint(0, V, (M,), generator=g).to(DEV)
    return h, W, y


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,V", [(9, 300), (70, 2000)])
def test_lowest_value_as_a_mask(M, V, dt):
    """Columns with the lowest value for a bias: probability 0, the bits that a
    -inf mask gives; a target there has the finite loss lse - t."""
    H = 64
    say(f"xent lowest-value mask M={M} V={V} {dt}")
    h, W, y = grid(1, M, H, V, dt)
    masked = torch.arange(V, device=DEV) % 3 == 0
    masked[:256] = V > 300  # a whole tile
    b = torch.where(masked, F.min, 0.25)
    binf = torch.where(masked, -math.inf, 0.25)
    free = torch.nonzero(~masked)[:, 0]
    y = free[y % len(free)]
    hit = torch.tensor([0, 5, M - 1], device=DEV)
    y[hit] = torch.nonzero(masked)[:, 0][hit]
    loss, lse = L.xent_forward(h, W, y, 1.0, b)
    loss_inf, lse_inf = L.xent_forward(h, W, y, 1.0, binf)
    assert torch.equal(lse, lse_inf)
    other = torch.ones(M, dtype=torch.bool, device=DEV)
    other[hit] = False
    assert torch.equal(loss[other], loss_inf[other]) and bool((loss_inf[hit] == math.inf).all())
    # t rounds to the lowest value itself (what is added to it is below half
    # its step); lse - t adds two roundings
    want = lse.double()[hit] - F.min
    assert bool(loss[hit].isfinite().all()) and bool(((loss[hit].double() - want).abs() <= 2 * U * want).all())
    gl = torch.full((M,), 1.0 / M, device=DEV)
    a, c = L.xent_backward(gl, h, W, y, lse, 1.0, b), L.xent_backward(gl, h, W, y, lse, 1.0, binf)
    for p, q in zip(a, c):
        assert torch.equal(p, q) and bool(p.isfinite().all())
    assert bool((a[2][y[hit]] < 0).all())  # a masked target's column: only the targets' -gl


@pytest.mark.parametrize("V", [40, 700])
def test_every_column_at_the_lowest_value(V):
    """The row's log-sum-exp is finite: log V is far below half a step there."""
    M, H = 5, 32
    say("xent all columns at the lowest value", V)
    h, W, y = grid(2, M, H, V, "bf16")
    b = torch.full((V,), F.min, device=DEV)
    loss, lse = L.xent_forward(h, W, y, 1.0, b)
    assert bool((lse == F.min).all()) and bool(loss.isfinite().all())


def sum_error(V):
    """Relative error of a row's sum of exponentials and of its fold, the
    arguments' own errors aside: exp2 (2 u), 16 additions per lane, two lane and
    four wave folds of two roundings and a factor, the tiles' folds."""
    return (24 + 3 * ((V + 255) // 256 // 16 + 18)) * U


@pytest.mark.parametrize("V", [40, 700])
def test_loss_where_every_column_is_at_the_lowest_value(V):
    """Equal logits: log V, though lse has no digits of that size left."""
    say("xent loss at the lowest value", V)
    h, W, y = grid(2, 5, 32, V, "bf16")
    loss, _ = L.xent_forward(h, W, y, 1.0, torch.full((V,), F.min, device=DEV))
    assert bool(((loss.double() - math.log(V)).abs() <= sum_error(V) + 4 * U * math.log(V)).all())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("top", [64.0, 4096.0])
def test_loss_of_a_confident_token(top, dt):
    """A largest logit of `top`, two columns 3 and 6 below it, the others 40 and
    more below: the loss is log(1 + e^-3 + e^-6 + ...), or that plus 3, in an
    lse whose half step is 2^-24 top. Exact logits: every one is the bias."""
    H, V = 32, 520
    say("xent confident", top, dt)
    h, W, _ = grid(4, 3, H, V, dt)
    h.zero_()
    b = torch.full((V,), top - 40.0, device=DEV)
    b[:7] = 0.0
    b[300], b[310], b[5] = top, top - 3, top - 6
    y = torch.tensor([300, 310, 300], device=DEV)
    loss, lse = L.xent_forward(h, W, y, 1.0, b)
    s = torch.exp(b.double() - top).sum()
    want = torch.log(s) + (top - b.double()[y])
    # the sum's terms past the largest weigh e^-3 and less; their arguments are
    # off by the product's and the constant's rounding, 2 u x relatively
    terms = torch.exp(b.double() - top)
    arg = 2 * U * float(((top - b.double()) * terms).sum() / s)
    tol = sum_error(V) + arg + 4 * U * want
    err = (loss.double() - want).abs()
    say(f"  worst {float((err / tol).max()):.3f} of the bound")
    assert bool((err <= tol).all())
    assert bool(((lse.double() - top - torch.log(s)).abs() <= U * top + sum_error(V) + arg + 4 * U).all())


def test_logits_near_the_largest_value():
    """A finite logit of 3e38 (its product with log2 e would be inf): certainty."""
    M, H, V = 6, 32, 300
    say("xent near the largest value")
    h, W, y = grid(3, M, H, V, "bf16")
    b = torch.zeros(V, device=DEV)
    b[7] = 3e38
    y[:3], y[3:] = 7, 200
    loss, lse = L.xent_forward(h, W, y, 1.0, b)
    assert bool((lse == b[7]).all()) and bool((loss[:3] == 0).all()) and bool((loss[3:] == b[7]).all())
    gl = torch.ones(M, device=DEV)
    dh, dw, db = L.xent_backward(gl, h, W, y, lse, 1.0, b)
    want = torch.zeros(V, device=DEV)
    want[7], want[200] = 3.0, -3.0
    assert torch.equal(db, want) and bool((dh[:3] == 0).all())
    # rows 3..: G is 1 at column 7 and -1 at 200, exact in 16 bits
    d = W[7].double() - W[200].double()
    assert torch.equal(dh[3:], d.to(torch.bfloat16).expand(3, H))
    s = h[3:].double().sum(0)
    assert torch.equal(dw[7], s.to(torch.bfloat16)) and torch.equal(dw[200], (-s).to(torch.bfloat16))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_other_rows_of_an_infinite_upstream_gradient(bad, dt):
    """An overflowed row's upstream gradient leaves the other rows' grad_hidden
    as they are without it (fp16: G of 2^-16 / V unscaled would be lost)."""
    M, H, V = 20, 64, 700
    say("xent infinite upstream gradient", bad, dt)
    h, W, y = grid(5, M, H, V, dt)
    gl = torch.full((M,), 2.0 ** -16, device=DEV)
    gz = torch.zeros(M, device=DEV)
    _, lse = L.xent_forward(h, W, y, 0.25)
    for into in (gl, gz):
        keep = float(into[7])
        into[7] = 0.0
        want = L.xent_backward(gl, h, W, y, lse, 0.25, grad_lse=gz)[0]
        into[7] = bad
        got = L.xent_backward(gl, h, W, y, lse, 0.25, grad_lse=gz)[0]
        into[7] = keep
        assert not bool(got[7].isfinite().all())
        rows = torch.arange(M, device=DEV) != 7
        assert bool(want[rows].isfinite().all()) and bool((want[rows] != 0).any(1).all())
        assert torch.equal(got[rows], want[rows])
