"""The losses where their inputs leave the ordinary range, whose state a call takes, and
their differentiable functions without grad mode; which rows the scale of G is chosen
from, and for which entries. Formulas and bounds: tests/loss_formulas.py."""
import math

import pytest
import torch

import lm_head_logits_amd as L
import loss_formulas as F
from gpu_util import DEV, say
from test_gpu_losses import DT, KW, OPS, call, check, make, reference

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


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [40, 300])
def test_teachers_logits_past_the_range_at_the_temperature(dt, M):
    """Entries whose quotient by the temperature leaves fp32 (a row of the type's
    lowest value, of its largest) weigh what their differences say."""
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt]
    c = make("distill", 31, M, 64, 300, "bf16", True, mask=0.0)
    c["teacher_ids"][c["teacher_ids"] < 0] = 17
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max

    def both(fill, plain):
        got = []
        for f in (fill, plain):
            s = c["teacher_logits"].to(dtype).clone()
            f(s)
            say("teacher's extremes", dt, M)
            (loss,), grads = check(dict(c, teacher_logits=s), kw=dict(temperature=0.5))
            assert bool(loss.isfinite().all()) and all(bool(t.isfinite().all()) for t in grads)
            got.append((loss, *grads))
        return got

    def ends(s):
        s[1], s[2] = low, high

    def zeros(s):
        s[1:3] = 0.0

    assert all(torch.equal(a, b) for a, b in zip(*both(ends, zeros)))

    def far(s):
        s[3, ::2], s[4, 1] = low, high

    def absent(s):  # a probability of 0, or none at all
        s[3, ::2] = -math.inf
        s[4, 0], s[4, 1], s[4, 2:] = -math.inf, 0.0, -math.inf

    a, b = both(far, absent)
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("V,others", [(1000, (999, 1001, 961, 1024)), (511, (510, 512))])
def test_a_state_belongs_to_its_vocabulary(V, others, keep):
    """Vocabularies whose states are of one size."""
    c = make("policy", 3, 20, 64, V, "bf16", False)
    reference(c, 0.5, KW["policy"])
    *_, saved = call(c, 0.5, KW["policy"], keep_logits=keep)
    for n in others:
        assert L.loss_state_bytes(20, 64, n, 0, keep) == saved.state.numel()
        with pytest.raises(ValueError, match="saved"):
            L.loss_backward(c["grad"], torch.zeros(n, 64, dtype=torch.bfloat16, device=DEV), saved)


def apply(c, h, W, b, **kw):
    kw = {**KW[c["op"]], **kw}
    if c["op"] == "distill":
        return L.distillation(h, W, c["teacher_ids"], c["teacher_logits"], 0.5, b, **kw)
    if c["op"] == "policy":
        return L.policy_loss(h, W, c["target"], c["advantage"], c["old"], c["ref"], 0.5, b, **kw)
    return L.preference_loss(h, W, c["target"], c["starts"], c["ref"], 0.5, b, **kw)


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("op", OPS)
def test_evaluation_leaves_no_state(op, off):
    """Parameters that require gradients, without grad mode: the loss alone, without
    the memory of the backward pass (here all logits, 48 MB, and the hidden rows)."""
    M, H, V = 600, 64, 20000
    c = make(op, 41, M, H, V, "bf16", True)
    reference(c, 0.5, KW[op])
    leaves = [c[k].clone().requires_grad_() for k in ("hidden", "weight", "bias")]

    def peak(fn):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out = fn()
        return out, torch.cuda.max_memory_allocated() - before

    trained, with_state = peak(lambda: apply(c, *leaves, reduction="none"))
    with off():
        (alone, without) = peak(lambda: apply(c, *leaves, reduction="none"))
    say("peak", op, with_state, without)
    assert torch.equal(alone, trained.detach()) and not alone.requires_grad
    assert with_state >= 4 * M * V and without < 2 * L.loss_forward_workspace_bytes(M, H, V, 7, False) < M * V
    # ... and with grad mode on again, inside it too
    with off(), torch.inference_mode(False), torch.enable_grad():
        apply(c, *leaves, reduction="sum").backward()
    assert leaves[0].grad is not None


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_prompts_do_not_reach_the_rounding(seed, dt):
    """Rows that are left out before those worked on, or behind them: the same
    gradients, bit for bit, since the scale under which G is rounded is chosen from the
    rows worked on."""
    n, H, V, K = 300, 64, 500, 8
    c = make("distill", seed, n, H, V, dt, False, K=K, mask=0.0)
    c["teacher_ids"][c["teacher_ids"] < 0] = 17  # no row without entries
    pad = make("distill", seed + 10, n, H, V, dt, False, K=K, mask=0.0)
    pad["teacher_ids"][:] = -100
    got = []
    for front in (0, n // 2, n):
        x = dict(c)
        for k in ("hidden", "teacher_ids", "teacher_logits", "grad"):
            x[k] = torch.cat([pad[k][:front], c[k], pad[k][front:]])
        say("prompts", front, dt, seed)
        loss, saved = call(x, 0.5, KW["distill"])
        dh, dw, _ = L.loss_backward(x["grad"], c["weight"], saved)
        got.append((loss[front:front + n], dh[front:front + n], dw))
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], g))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M", [200, 300, 3000])
@pytest.mark.parametrize("p", [0.553, 0.617, 0.68, 0.703, 0.761, 0.822, 0.87, 0.94])
def test_the_scale_suits_the_entries_that_weigh_most(p, M, dt):
    """A batch whose rows have one large entry of G each, of the same value, but for some
    with many small ones (the first rows, and some between): the factor of the scale is the
    one of the sixteen that rounds the large entry best. With W the unit matrix
    grad_hidden is G, off by that rounding and by its own: half a step."""
    V, K, high = 256, 100, 7
    c = make("distill", 1, M, V, V, dt, False, K=K, mask=0.0)
    hidden, weight = torch.zeros_like(c["hidden"]), torch.eye(V, device=DEV).to(DT[dt])
    ids = torch.arange(K, device=DEV).repeat(M, 1)
    s = torch.zeros(M, K, device=DEV)
    s[:, high] = math.log(p / (1 - p) * (K - 1))
    small = torch.arange(M, device=DEV)
    small = (small < 11) | (small % 30 == 15)
    s[small] = 0.0
    g = torch.full((M,), 1.0 / M, device=DEV)
    say("scale", p, M, dt)
    _, saved = L.distill_forward(hidden, weight, ids, s)
    got = L.loss_backward(g, weight, saved)[0][~small, high].double()
    pk = torch.softmax(s.double(), 1)[~small, high]
    x = 1.0 / V - float(pk[0])  # the entry over the largest coefficient
    tries = [2.0 ** (-j / 16) for j in range(16)]
    rounding = min(abs(float(torch.tensor(x * t).to(DT[dt])) / t - x) for t in tries)
    want = x * float(g[0])
    half = 2.0 ** math.floor(math.log2(abs(want))) * torch.finfo(DT[dt]).eps / 2
    bound = rounding * float(g[0]) + half * (1 + 1e-3)  # and what fp32 adds
    assert float((got - want).abs().max()) <= bound, (float((got - want).abs().max()) / half, bound / half)


@pytest.mark.parametrize("M,H,V,tokens", [(1, 32, 40, 1), (40, 64, 300, 1), (64, 2080, 300, 2), (200, 64, 500, 1), (256, 4096, 333, 3),
                                          (300, 64, 500, 1), (700, 2080, 500, 5), (3000, 96, 700, 2), (4600, 608, 500, 1), (5000, 32, 300, 200),
                                          (70000, 32, 300, 3)])
def test_rows_of_frequent_tokens(M, H, V, tokens):
    """grad_W's row of a token that is the target of many rows, of either sign: elements in
    which they cancel are as exact as the others. With no ratio and no KL term the entry of
    a row is -g A (1 - q). Bound: q is off by what log q is (loss_formulas), 1 - q and the
    entry by 4 u, a chain of M additions; the token's other logits' share, G rounded to
    half a step, summed and rounded; and the result's own rounding. (bf16: fp16's G has
    three bits more, and the target's entry in it.)"""
    dt = "bf16"
    c = make("policy", 11, M, H, V, dt, False, mask=0.1 if M > 1 else 0.0)
    y = c["target"]
    y[y >= 0] = y[y >= 0] % tokens  # the first ones
    kw = dict(KW["policy"], kl_coef=0.0)
    c.update(old=None, ref=None)
    loss, logp, saved = call(c, 0.5, kw)
    say("frequent tokens", M, H, V, tokens, dt)
    for keep in (True, False):
        *_, saved = call(c, 0.5, kw, keep_logits=keep)
        dh, dw, _ = L.loss_backward(c["grad"], c["weight"], saved)
        head = F.Head(c["hidden"], c["weight"], None, 0.5, 1.0)
        kept = y >= 0
        at = torch.where(kept, y, torch.zeros_like(y)).long()[:, None]
        a = torch.where(kept, c["grad"].double() * c["advantage"].double(), torch.zeros(M, dtype=torch.float64, device=DEV))
        G = a[:, None] * head.q
        G.scatter_add_(1, at, -a[:, None])
        own = torch.zeros_like(G).scatter_(1, at, G.gather(1, at))
        rest, h = G - own, c["hidden"].double()
        u, step = F.U, torch.finfo(DT[dt]).eps / 2
        q = head.q.gather(1, at)[:, 0]
        err = a.abs() * (q * 2 * head.dlogq.gather(1, at)[:, 0] + 8 * u)  # of the entry
        spread = torch.zeros_like(G).scatter_(1, at, err[:, None] + (M + 8) * u * own.gather(1, at).abs())
        want = 0.5 * (G.t() @ h)
        main = 0.5 * (rest.t() @ h)
        d = rest.abs() * step + a.abs()[:, None] * head.dq
        tol = 0.5 * (spread.t() @ h.abs() + d.t() @ h.abs() + 2e-5 * (rest.abs().t() @ h.abs()))
        tol = tol * (1 + 2 * step) + step * main.abs() + step * want.abs() + 2.0 ** -126
        bad = (dw.double() - want)[:tokens].abs() - tol[:tokens]
        assert float(bad.max()) <= 0, (keep, float(((dw.double() - want)[:tokens].abs() / tol[:tokens]).max()))


@pytest.mark.parametrize("M", [700, 4500])
def test_frequent_tokens_replayed(M):
    """A captured backward pass over other targets each time, some left out: the eager
    call's bits, whichever work-groups come first."""
    H, V = 96, 600
    c = make("policy", 3, M, H, V, "bf16", True, mask=0.2)
    c.update(old=None, ref=None)
    kw = dict(KW["policy"], kl_coef=0.0)

    def step():
        *_, saved = call(c, 0.5, kw)
        return L.loss_backward(c["grad"], c["weight"], saved)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        other = make("policy", 20 + k, M, H, V, "bf16", False, mask=0.1 * k)["target"]
        c["target"].copy_(torch.where(other < 0, other, other % (1 + 40 * k)))
        say("frequent tokens, replay", M, k)
        want = step()
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(want, step()))
        torch.cuda.synchronize()
        for t in out:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
