"""Distillation, the policy loss and the preference loss, with their gradients,
against the formulas in 64 bits (tests/loss_formulas.py, where the bounds are
derived)."""
import math

import pytest
import torch

import lm_head_logits_amd as L
import loss_formulas as F
from gpu_util import DEV, say
from test_gpu_xent import TINY16, close

pytestmark = pytest.mark.gpu
U = F.U
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
OPS = ("distill", "policy", "preference")


def make(op, seed, M, H, V, dt, bias, K=7, pairs=3, index=torch.int64, mask=0.3, std=1.0):
    """A call's inputs by name."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g)
    normal = lambda *s: torch.randn(*s, generator=g)
    c = dict(op=op, hidden=normal(M, H).mul_(std).to(DT[dt]).to(DEV), weight=normal(V, H).mul_(0.05).to(DT[dt]).to(DEV),
             bias=normal(V).mul_(0.3).to(DEV) if bias else None)
    if op == "distill":
        K = min(K, V)
        ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(M)]) if M else torch.zeros(0, K, dtype=torch.long)
        ids[rand(M) < mask] = -100
        ids[rand(M, K) < 0.1] = -1
        c.update(teacher_ids=ids.to(index).to(DEV), teacher_logits=(normal(M, K) * 2).to(DEV), grad=normal(M).to(DEV))
        return c
    y = torch.randint(0, V, (M,), generator=g)
    y[rand(M) < mask] = -100
    c.update(target=y.to(index).to(DEV))
    if op == "policy":
        c.update(advantage=normal(M).to(DEV), noise=normal(M).mul_(0.2).double().to(DEV),
                 drift=normal(M).mul_(0.5).double().to(DEV), grad=normal(M).to(DEV))
    else:
        cuts = torch.sort(torch.randint(0, M + 1, (2 * pairs + 1,), generator=g)).values
        if M > 8:
            cuts[0], cuts[-1] = 1, M - 2  # a row before the first, two behind the last
        c.update(starts=cuts.to(index).to(DEV), ref=normal(2 * pairs).to(DEV), grad=normal(pairs).to(DEV))
    return c


KW = dict(distill=dict(temperature=1.0), policy=dict(temperature=1.0, clip_low=0.2, clip_high=0.3, kl_coef=0.05),
          preference=dict(temperature=1.0, beta=0.5, margin=0.25, label_smoothing=0.1, average=False))


def old_and_ref(c, head, low, high):
    """Log-probabilities of an earlier policy, no ratio within 2^-8 of a border of
    the clip, or within twice what the log-probabilities may be off."""
    keep, _, logp, dl = F._token(head, c["target"], -100)
    gap = max(2.0 ** -8, 2 * float(dl.max()))
    assert gap < 2.0 ** -5
    lr = c["noise"]
    for border in (math.log1p(-low), math.log1p(high)):
        lr = torch.where((lr - border).abs() < gap, lr + 4 * gap, lr)
    fin = logp.nan_to_num(0, 0, 0)
    return (fin - lr).float(), (fin + c["drift"]).float()


def call(c, alpha, kw, train=True, **more):
    """The library's forward call on the inputs, and its other outputs."""
    if c["op"] == "distill":
        return L.distill_forward(c["hidden"], c["weight"], c["teacher_ids"], c["teacher_logits"], alpha, c["bias"],
                                 train=train, **kw, **more)
    if c["op"] == "policy":
        return L.policy_forward(c["hidden"], c["weight"], c["target"], c["advantage"], c.get("old"), c.get("ref"), alpha,
                                c["bias"], train=train, **kw, **more)
    return L.preference_forward(c["hidden"], c["weight"], c["target"], c["starts"], c.get("ref"), alpha, c["bias"],
                                train=train, **kw, **more)


def reference(c, alpha, kw):
    """(head, [(name, value, bound)], gradients); fills in old_logp and ref_logp."""
    head = F.Head(c["hidden"], c["weight"], c["bias"], alpha, kw["temperature"])
    if c["op"] == "distill":
        loss, bound, grads = F.distill(head, c["teacher_ids"], c["teacher_logits"], kw["temperature"],
                                       kw.get("teacher_lse"), c["grad"])
        return head, [("loss", loss, bound)], grads
    if c["op"] == "policy":
        if "old" not in c:
            c["old"], c["ref"] = old_and_ref(c, head, kw["clip_low"], kw["clip_high"])
        loss, bound, logp, dl, grads = F.policy(head, c["target"], c["advantage"], c["old"], c["ref"], kw["clip_low"],
                                                kw["clip_high"], kw["kl_coef"], grad=c["grad"])
    else:
        loss, bound, logp, dl, grads = F.preference(head, c["target"], c["starts"], c.get("ref"), kw["beta"], kw["margin"],
                                                    kw["label_smoothing"], kw["average"], grad=c["grad"])
    return head, [("loss", loss, bound), ("logp", logp, dl)], grads


def check_grads(got, grads, dt, bias):
    tiny, h16 = TINY16["f16" if dt == torch.float16 else "bf16"], torch.finfo(dt).eps / 2
    for name, t in zip(("hidden", "weight"), got):
        want, tol = grads[name]
        assert t.dtype == dt
        close(name, t, want, tol + h16 * (want.abs() + tol) * (1 + 4 * U) + 4 * U * want.abs() + tiny)
    if bias:
        close("bias", got[2], *grads["bias"])
    else:
        assert got[2] is None


def check(c, alpha=0.5, kw=None):
    kw = {**KW[c["op"]], **(kw or {})}
    head, outs, grads = reference(c, alpha, kw)
    *got, saved = call(c, alpha, kw)
    for (name, want, bound), t in zip(outs, got):
        assert t.dtype == torch.float32
        close(name, t, want, bound)
    alone = call(c, alpha, kw, train=False)
    assert alone[-1] is None
    for a, b in zip(alone, got):
        assert torch.equal(a, b)
    assert saved.keep_logits
    d = L.loss_backward(c["grad"], c["weight"], saved)
    check_grads(d, grads, c["hidden"].dtype, c["bias"] is not None)
    # the logits made again instead of kept: the same bits but for grad_bias, whose sums have another order
    *again, lean = call(c, alpha, kw, keep_logits=False)
    assert all(torch.equal(a, b) for a, b in zip(again, got)) and not lean.keep_logits
    e = L.loss_backward(c["grad"], c["weight"], lean)
    assert torch.equal(d[0], e[0]) and torch.equal(d[1], e[1])
    if c["bias"] is not None:
        close("bias", e[2], *grads["bias"])
    return got, d


# one row and one column; ends inside a 16-row block, a 128-row half, a tile; a
# partial stage, odd and even stage counts; columns past a tile, past a K-order group
SIZES = [(1, 32, 1), (1, 64, 300), (2, 96, 17), (16, 128, 256), (37, 256, 1000), (64, 160, 257), (128, 320, 511),
         (129, 64, 2049), (255, 192, 129), (257, 512, 700), (300, 288, 333), (513, 224, 1025), (31, 512, 20500)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("M,H,V", SIZES)
def test_against_the_formula(op, M, H, V, dt):
    bias, T = (M + V) % 2 == 0, 0.75 if M % 2 else 1.0
    say(f"{op} M={M} H={H} V={V} {dt} bias={bias} T={T}")
    c = make(op, M * 7 + V, M, H, V, dt, bias, index=torch.int32 if H % 64 else torch.int64)
    check(c, kw=dict(temperature=T))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("K,V", [(1, 400), (63, 700), (64, 300), (65, 999), (200, 256), (256, 5000), (257, 700),
                                 (1024, 1500), (1000, 3001)])
def test_teachers_of_every_size(K, V, dt):
    M, H = 70, 96
    say(f"distill K={K} V={V} {dt}")
    c = make("distill", K + V, M, H, V, dt, True, K=K)
    check(c, kw=dict(temperature=2.0))
    for t in (torch.bfloat16, torch.float16):
        c["teacher_logits"] = c["teacher_logits"].to(t)
        check(c)


def test_a_teacher_known_whole():
    M, H, V, K = 90, 64, 800, 20
    c = make("distill", 3, M, H, V, "bf16", True, K=K, mask=0.0)
    whole = torch.logsumexp(c["teacher_logits"].double() / 1.5, 1) + torch.rand(M, dtype=torch.float64, device=DEV)
    check(c, kw=dict(temperature=1.5, teacher_lse=whole.float()))


def test_entries_in_one_tile_and_entries_that_repeat():
    """Every entry of every row in one 256-column tile; ids that a row has several times."""
    M, H, V, K = 300, 64, 1200, 100
    c = make("distill", 5, M, H, V, "bf16", True, K=K, mask=0.0)
    say("distill one tile")
    c["teacher_ids"] = (c["teacher_ids"].clamp(0) % 256) + 512
    check(c)
    say("distill repeats")
    c["teacher_ids"] = c["teacher_ids"] % 8
    check(c)
    c["teacher_ids"].fill_(V - 1)
    check(c)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_entries_that_are_absent(index):
    M, H, V, K = 40, 64, 500, 9
    c = make("distill", 7, M, H, V, "f16", True, K=K, index=index, mask=0.0)
    ids, s = c["teacher_ids"], c["teacher_logits"]
    ids[0], ids[1, 1:], ids[2, ::2] = V, -5, 2 ** 31 - 1
    s[3] = -math.inf
    s[4, 1:] = -math.inf
    s[5] = torch.finfo(torch.float32).min  # a number: all entries alike
    s[6, 3] = torch.finfo(torch.float32).min
    if index == torch.int64:
        ids[7, 0] = 2 ** 40 + 3  # not its low 32 bits
    say("distill absent", index)
    (loss,), d = check(c)
    assert float(loss[0]) == 0.0 and float(loss[3]) == 0.0
    assert bool((d[0][0] == 0).all() and (d[0][3] == 0).all())
    ids.fill_(-1)
    (loss,), d = check(c)
    assert bool((loss == 0).all()) and all(bool((t == 0).all()) for t in d)


@pytest.mark.parametrize("op", OPS)
def test_masked_columns(op):
    """-inf biases: columns of probability 0, a whole tile of them; the type's lowest value."""
    M, H, V = 30, 64, 600
    c = make(op, 11, M, H, V, "bf16", True, K=5)
    b = c["bias"]
    b[::3] = -math.inf
    b[:256] = -math.inf
    if op == "distill":  # what the teacher names is not masked, but for one row
        c["teacher_ids"] = torch.where(c["teacher_ids"] >= 0, 257 + 3 * (c["teacher_ids"] % 100), c["teacher_ids"])
    else:
        c["target"] = torch.where(c["target"] >= 0, 257 + 3 * (c["target"] % 100), c["target"])
    say("masked", op)
    check(c)
    b[b == -math.inf] = torch.finfo(torch.float32).min
    check(c)
    # a masked token: log-probability -inf
    b[b == torch.finfo(torch.float32).min] = -math.inf
    if op == "distill":
        c["teacher_ids"][0, 0], c["teacher_logits"][0, 0] = 3, 1.0
        assert float(call(c, 0.5, KW[op])[0][0]) == math.inf
    elif op == "policy":
        c["target"][0] = 3
        loss, logp, _ = call({**c, "old": None, "ref": None}, 0.5, KW[op])
        assert float(logp[0]) == -math.inf
    else:
        s = c["starts"]
        c["target"][int(s[0])], s[1:] = 3, M
        assert float(call(c, 0.5, KW[op])[1][0]) == -math.inf


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("op", OPS)
def test_peaked_rows_and_large_logits(op, dt):
    M, H, V = 20, 32, 300
    c = make(op, 13, M, H, V, dt, False, std=30.0)
    c["weight"][5] = c["weight"][9]  # exact ties
    c["hidden"][3] = 0               # constant row: lse = log V
    say("peaked", op, dt)
    if op == "policy":  # no ratio against rows whose bound is wider than the borders' distance
        c.update(old=None, ref=None)
    check(c, alpha=8.0)


@pytest.mark.parametrize("op", OPS)
def test_more_than_one_piece_and_a_scale_of_its_own(op):
    # 16385 rows of 8192 columns a piece; more than 32768 rows: the scale has a launch of its own
    for M, H, V in ((16385, 32, 8450), (32769 + 200, 32, 40)):
        say(f"{op} M={M} V={V}")
        check(make(op, 17, M, H, V, "f16", True, pairs=40, K=5))


@pytest.mark.parametrize("M,H,V", [(3, 1 << 16, 70), (5, 32, 1 << 20)])
@pytest.mark.parametrize("op", OPS)
def test_the_contracts_maxima(op, M, H, V):
    say(f"{op} maxima M={M} H={H} V={V}")
    c = make(op, 19, M, H, V, "bf16", False, std=0.1)
    if op == "distill":
        c["teacher_ids"][:, 0] = V - 1
    else:
        c["target"][:] = V - 1
    check(c)


@pytest.mark.parametrize("op", OPS)
def test_gradient_scale_range(op):
    """Upstream gradients far from 1, rows of very different size, all zero."""
    M, H, V = 33, 64, 150
    for dt, k in (("bf16", 1e-12), ("bf16", 1e8), ("f16", 1e-3), ("f16", 30.0)):
        c = make(op, 23, M, H, V, dt, True)
        c["grad"] *= k / M
        c["grad"][1:3] *= 1e-3
        say("gradient scale", op, dt, k)
        check(c)
    saved = call(c, 0.5, KW[op])[-1]
    for t in L.loss_backward(torch.zeros_like(c["grad"]), c["weight"], saved):
        assert bool((t == 0).all())


def test_policy_without_old_or_reference():
    c = make("policy", 29, 50, 64, 300, "bf16", True)
    for old, ref, kl in ((True, False, 0.1), (False, True, 0.1), (True, True, 0.0), (False, False, 0.0)):
        head = F.Head(c["hidden"], c["weight"], c["bias"], 0.5, 1.0)
        o, r = old_and_ref(c, head, 0.2, 0.3)
        c.update(old=o if old else None, ref=r if ref else None)
        say("policy old", old, "ref", ref, "kl", kl)
        (loss, logp), _ = check(c, kw=dict(kl_coef=kl))
        if not old and not ref:  # the first step after a rollout: the policy gradient
            kept = c["target"] >= 0
            assert torch.equal(loss[kept], -c["advantage"][kept])
    # no advantage, no loss, whatever the ratio
    c.update(advantage=torch.zeros(50, device=DEV), old=torch.full((50,), -1e4, device=DEV), ref=None)
    loss, logp, saved = call(c, 0.5, KW["policy"])
    assert bool((loss == 0).all()) and all(bool((t == 0).all()) for t in L.loss_backward(c["grad"], c["weight"], saved))


@pytest.mark.parametrize("average", [False, True])
def test_preference_forms(average):
    M, H, V, P = 400, 64, 300, 6
    c = make("preference", 31, M, H, V, "bf16", True, pairs=P)
    say("preference forms", average)
    check(c, kw=dict(average=average, label_smoothing=0.0))
    c["ref"] = None
    check(c, kw=dict(average=average, beta=2.0, label_smoothing=1.0))
    # empty sequences, sequences without a target, all of one sequence
    s = torch.tensor([0, 0, 5, 5, 9, 100, 100, 100, 300, 301, 302, 303, 400], device=DEV)
    c["starts"], c["target"][5:9] = s, -100
    check(c, kw=dict(average=average))
    c["starts"] = torch.tensor([0] + [0] * P + [M] * P, device=DEV)
    check(c, kw=dict(average=average))
    # extreme margins: one side saturates
    for margin in (1e4, -1e4):
        (loss, _), d = check(c, kw=dict(average=average, margin=margin, label_smoothing=0.0))
        assert bool(torch.isfinite(loss).all()) and all(bool(torch.isfinite(t).all()) for t in d)
    c["starts"] = torch.zeros(1, dtype=torch.int64, device=DEV)
    c["grad"] = torch.zeros(0, device=DEV)
    loss, logp, saved = call(c, 0.5, KW["preference"])
    assert loss.shape == logp.shape == (0,)
    assert all(bool((t == 0).all()) for t in L.loss_backward(c["grad"], c["weight"], saved))


@pytest.mark.parametrize("op", OPS)
def test_gradients_against_differences(op):
    """Central differences of the library's own loss (summed in 64 bits) along a
    direction in each input; the remainder is bounded by halving the step: for a
    smooth loss the quotients of steps e and e / 2 differ by 3/4 of the first
    one's remainder to leading order, taken twice over here."""
    M, H, V, alpha = 8, 32, 70, 1.0
    c = make(op, 37, M, H, V, "f16", True, pairs=2, mask=0.0)
    c["hidden"] = (c["hidden"] * 4).round().div(4)
    c["weight"] = (c["weight"] * 64).round().div(64)  # sums of two grid values stay exact
    c["grad"] = torch.ones_like(c["grad"])
    kw = KW[op]
    head, _, _ = reference(c, alpha, kw)
    if op == "policy":  # far from the borders, where the loss has a corner
        _, _, logp, _ = F._token(head, c["target"], -100)
        c["old"] = (logp - torch.tensor([0.0, 0.02, -0.02, 2.0, -2.0, 0.05, 0.0, 3.0], device=DEV, dtype=torch.float64)).float()
    saved = call(c, alpha, kw)[-1]
    grads = L.loss_backward(c["grad"], c["weight"], saved)
    rng = torch.Generator().manual_seed(3)
    for name, grad in zip(("hidden", "weight", "bias"), grads):
        for _ in range(4):
            d = torch.randint(-1, 2, grad.shape, generator=rng).to(DEV)
            e = {"hidden": 0.125, "weight": 2.0 ** -6, "bias": 0.125}[name]
            quot = []
            for step in (e, e / 2):
                vals = []
                for sgn in (1, -1):
                    x = c[name].float() + sgn * step * d
                    assert torch.equal(x.to(c[name].dtype).float(), x)
                    vals.append(call({**c, name: x.to(c[name].dtype)}, alpha, kw)[0].double().sum())
                quot.append(float(vals[0] - vals[1]) / (2 * step))
            ana = float((grad.double() * d.double()).sum())
            noise = sum(float(b.sum()) for n, v, b in reference(c, alpha, kw)[1] if n == "loss") * 4 / e
            # the gradient's own 16-bit roundings, of G and of the result
            r = 2.0 ** -10 * float((grad.double().abs() * d.double().abs()).sum()) + 2.0 ** -10 * M
            tol = 2 * abs(quot[0] - quot[1]) + noise + r
            say(f"  differences {name}: {quot[1]:.6f} against {ana:.6f}, bound {tol:.2e}")
            assert abs(quot[1] - ana) <= tol


@pytest.mark.parametrize("op", OPS)
def test_rows_do_not_depend_on_the_call_and_runs_repeat(op):
    M, H, V = 300, 256, 5000
    c = make(op, 41, M, H, V, "bf16", True, pairs=4, K=30)
    reference(c, 0.5, KW[op])
    *out, saved = call(c, 0.5, KW[op])
    if op != "preference":
        for n in (1, 16, 37, 129, 256):
            part = {k: v[:n].contiguous() if torch.is_tensor(v) and v.shape[:1] == (M,) else v for k, v in c.items()}
            for a, b in zip(call(part, 0.5, KW[op]), out):
                assert torch.equal(a, b[:n]), n
    a = L.loss_backward(c["grad"], c["weight"], saved)
    for _ in range(2):
        *again, s2 = call(c, 0.5, KW[op])
        assert all(torch.equal(p, q) for p, q in zip(again, out))
        for p, q in zip(a, L.loss_backward(c["grad"], c["weight"], s2)):
            assert torch.equal(p, q)
        for p, q in zip(a, L.loss_backward(c["grad"], c["weight"], saved)):  # one state, more than once
            assert torch.equal(p, q)
    # parts asked for alone are the same bits
    assert torch.equal(L.loss_backward(c["grad"], c["weight"], saved, need_weight=False, need_bias=False)[0], a[0])
    only = L.loss_backward(c["grad"], c["weight"], saved, need_hidden=False, need_bias=False)
    assert only[0] is None and only[2] is None and torch.equal(only[1], a[1])
    assert torch.equal(L.loss_backward(c["grad"], c["weight"], saved, need_hidden=False, need_weight=False)[2], a[2])


@pytest.mark.parametrize("op", OPS)
def test_captured_and_replayed(op):
    M, H, V = 300, 128, 3000
    c = make(op, 43, M, H, V, "bf16", True, pairs=3, K=12)
    reference(c, 0.5, KW[op])

    def step():
        *out, saved = call(c, 0.5, KW[op])
        return (*out, *L.loss_backward(c["grad"], c["weight"], saved))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        say("replay", op, k)
        c["hidden"].copy_(torch.randn(M, H, device=DEV) * (k + 1))
        for name in ("target", "teacher_ids"):
            if name in c:
                c[name].copy_(torch.randint(-k * V // 2, V, c[name].shape, device=DEV))
        want = step()
        torch.cuda.synchronize()
        for t in out:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("op", OPS)
def test_two_streams_at_once(op):
    ins = [make(op, 50 + k, 290, 256, 4000, "bf16", True) for k in range(2)]
    want = []
    for c in ins:
        reference(c, 0.5, KW[op])
        *out, saved = call(c, 0.5, KW[op])
        want.append((*out, *L.loss_backward(c["grad"], c["weight"], saved)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(3):
        for k, c in enumerate(ins):
            *out, saved = call(c, 0.5, KW[op], stream=streams[k])
            got[k] = (*out, *L.loss_backward(c["grad"], c["weight"], saved, stream=streams[k]))
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        for a, b in zip(p, q):
            assert torch.equal(a, b)


@pytest.mark.parametrize("keep", [0, 1])
@pytest.mark.parametrize("M", [90, 290])
@pytest.mark.parametrize("op", OPS)
def test_nothing_outside_the_outputs_is_written(op, M, keep):
    """Exact sizes of state and workspace, guards around every output."""
    H, V, K, P, pad = 96, 333, 9, 2, 64
    c = make(op, 59, M, H, V, "bf16", True, K=K, pairs=P)
    reference(c, 0.5, KW[op])
    from lm_head_logits_amd import _lib
    lib, s = _lib.load(), torch.cuda.current_stream().cuda_stream
    K = K if op == "distill" else 0
    ns, nf, nb = (L.loss_state_bytes(M, H, V, K, keep), L.loss_forward_workspace_bytes(M, H, V, K),
                  L.loss_backward_workspace_bytes(M, H, V, K, keep, True))
    n = dict(loss=P if op == "preference" else M, logp=2 * P if op == "preference" else M)
    buf = {k: torch.full((m + 2 * pad,), 123.0, dtype=d, device=DEV) for k, m, d in
           (("loss", n["loss"], torch.float32), ("logp", n["logp"], torch.float32), ("dh", M * H, torch.bfloat16),
            ("dw", V * H, torch.bfloat16), ("db", V, torch.float32))}
    state = torch.full((ns + 512,), 77, dtype=torch.uint8, device=DEV)
    ws = torch.full((max(nf, nb) + 512,), 77, dtype=torch.uint8, device=DEV)
    at = {k: v.data_ptr() + pad * v.element_size() for k, v in buf.items()}
    head = (c["hidden"].data_ptr(), M, H, c["weight"].data_ptr(), V, 0.5, c["bias"].data_ptr(), _lib.LMHEAD_BF16, 1.25)
    mem = (state.data_ptr(), ns, keep, ws.data_ptr(), nf, s)
    if op == "distill":
        st = lib.lmhead_distill_forward(*head, c["teacher_ids"].data_ptr(), 1, c["teacher_logits"].data_ptr(), 0, K, None,
                                        at["loss"], *mem)
        del buf["logp"]
    elif op == "policy":
        st = lib.lmhead_policy_forward(*head, c["target"].data_ptr(), 1, -100, c["advantage"].data_ptr(),
                                       c["old"].data_ptr(), c["ref"].data_ptr(), 0.2, 0.2, 0.1, at["loss"], at["logp"], *mem)
    else:
        st = lib.lmhead_preference_forward(*head, c["target"].data_ptr(), 1, -100, c["starts"].data_ptr(), 1, P, None, 0.1,
                                           0.0, 0.0, 1, at["loss"], at["logp"], *mem)
    assert st == _lib.OK
    torch.cuda.synchronize()
    assert bool((ws[nf:] == 77).all()) and bool((state[ns:] == 77).all())
    st = lib.lmhead_loss_backward(*head, K, c["grad"].data_ptr(), state.data_ptr(), ns, keep, at["dh"], at["dw"],
                                  at["db"],
                                  ws.data_ptr(), nb, s)
    assert st == _lib.OK
    torch.cuda.synchronize()
    assert bool((ws[nb:][:512] == 77).all()) and bool((state[ns:] == 77).all())
    for k, v in buf.items():
        assert bool((v[:pad] == 123).all() and (v[-pad:] == 123).all()), k
        assert not bool((v[pad:-pad] == 123).any()), k


@pytest.mark.parametrize("op", OPS)
def test_no_rows(op):
    c = make(op, 61, 0, 64, 50, "bf16", True, pairs=2)
    c.update(old=None, ref=None)
    for T in (1.0, 2.0):
        *out, saved = call(c, 0.5, {**KW[op], "temperature": T})
        if op == "preference":
            z = -0.25
            want = -0.9 * math.log(1 / (1 + math.exp(-z))) - 0.1 * math.log(1 / (1 + math.exp(z)))
            assert bool((out[1] == 0).all()) and float((out[0] - want).abs().max()) <= 4 * U
        else:
            assert out[0].shape == (0,)
        dh, dw, db = L.loss_backward(c["grad"], c["weight"], saved)
        assert dh.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_refusals():
    h, W = torch.zeros(4, 64, device=DEV), torch.zeros(9, 64, device=DEV)
    y, f = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, device=DEV)
    ids, s = torch.zeros(4, 3, dtype=torch.int32, device=DEV), torch.zeros(4, 3, device=DEV)
    cuts = torch.tensor([0, 2, 4], device=DEV)
    hh, WW = h.half(), W.half()
    for a, b in ((h, W), (hh, W.bfloat16()), (hh[:, :40].contiguous(), WW[:, :40].contiguous())):
        with pytest.raises(L.NotHandled):
            L.policy_forward(a, b, y, f)
        with pytest.raises(L.NotHandled):
            L.preference_forward(a, b, y, cuts)
        with pytest.raises(L.NotHandled):
            L.distill_forward(a, b, ids, s)
    for bad in (lambda: L.policy_forward(hh, WW, y[:3], f), lambda: L.policy_forward(hh, WW, y, f[:3]),
                lambda: L.policy_forward(hh, WW, y, f, f.double()), lambda: L.policy_forward(hh, WW, y.float(), f),
                lambda: L.policy_forward(hh, WW, y, f, None, f.cpu()),
                lambda: L.preference_forward(hh, WW, y, cuts[:2]), lambda: L.preference_forward(hh, WW, y, cuts.float()),
                lambda: L.preference_forward(hh, WW, y, cuts, f[:1]), lambda: L.distill_forward(hh, WW, ids, s[:, :2]),
                lambda: L.distill_forward(hh, WW, ids[:3], s[:3]), lambda: L.distill_forward(hh, WW, ids, s.double()),
                lambda: L.distill_forward(hh, WW, ids.t().contiguous().t(), s),
                lambda: L.distill_forward(hh, WW, ids, s, teacher_lse=f[:2]),
                lambda: L.policy_loss(hh, WW, y, f, reduction="best"), lambda: L.loss_backward(f, WW, None)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: L.policy_forward(hh, WW, y, f, temperature=0.0),
                lambda: L.policy_forward(hh, WW, y, f, temperature=-1.0),
                lambda: L.policy_forward(hh, WW, y, f, temperature=math.inf),
                lambda: L.policy_forward(hh, WW, y, f, clip_low=-0.1), lambda: L.policy_forward(hh, WW, y, f, kl_coef=math.nan),
                lambda: L.preference_forward(hh, WW, y, cuts, label_smoothing=1.5),
                lambda: L.preference_forward(hh, WW, y, cuts, beta=math.nan),
                lambda: L.distill_forward(hh, WW, ids.repeat(1, 400).contiguous(), s.repeat(1, 400).contiguous()),
                lambda: L.policy_forward(hh, WW, y, f, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(L.LmHeadError):
            bad()
    loss, logp, saved = L.policy_forward(hh, WW, y, f)
    with pytest.raises(ValueError):
        L.loss_backward(f[:3], WW, saved)
    with pytest.raises(ValueError):
        L.loss_backward(f, WW, saved, need_bias=True)
    with pytest.raises(L.LmHeadError):
        L.loss_backward(f, WW, saved, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("op", OPS)
def test_differentiable(op):
    M, H, V = 290, 64, 400
    c = make(op, 67, M, H, V, "bf16", True)
    reference(c, 0.5, KW[op])
    kw = KW[op]
    loss, *_, saved = call(c, 0.5, kw)
    kept = {"distill": lambda: ((c["teacher_ids"] >= 0).any(1)).sum(), "policy": lambda: (c["target"] >= 0).sum(),
            "preference": lambda: torch.tensor(len(c["grad"]), device=DEV)}[op]()

    def apply(h, W, b, **more):
        if op == "distill":
            return L.distillation(h, W, c["teacher_ids"], c["teacher_logits"], 0.5, b, **kw, **more)
        if op == "policy":
            return L.policy_loss(h, W, c["target"], c["advantage"], c["old"], c["ref"], 0.5, b, **kw, **more)
        return L.preference_loss(h, W, c["target"], c["starts"], c["ref"], 0.5, b, **kw, **more)

    leaves = [c[k].clone().requires_grad_(True) for k in ("hidden", "weight", "bias")]
    out = apply(*leaves)
    assert torch.equal(out.detach(), loss.sum() / kept)
    out.backward()
    want = L.loss_backward(torch.ones_like(c["grad"]) / kept, c["weight"], saved)
    for t, w in zip(leaves, want):
        assert torch.equal(t.grad, w)
    # only what is asked for; "sum" and "none"; without a graph
    h2 = c["hidden"].clone().requires_grad_(True)
    apply(h2, c["weight"], c["bias"], reduction="sum").backward()
    assert torch.equal(h2.grad, L.loss_backward(torch.ones_like(c["grad"]), c["weight"], saved)[0])
    h3 = c["hidden"].clone().requires_grad_(True)
    apply(h3, c["weight"], c["bias"], reduction="none").backward(c["grad"])
    assert torch.equal(h3.grad, L.loss_backward(c["grad"], c["weight"], saved)[0])
    with torch.no_grad():
        assert torch.equal(apply(h3, c["weight"], c["bias"], reduction="none"), loss)
    if op != "distill":
        _, logp = apply(h3, c["weight"], c["bias"], return_logp=True)
        assert not logp.requires_grad


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("M", [40, 700, 4500])
def test_no_row_is_trained_on(op, M):
    """All left out, then all but one, the last."""
    c = make(op, 71, M, 64, 500, "bf16", True)
    name = "teacher_ids" if op == "distill" else "target"
    was = c[name][-1].clone().clamp(min=3)
    c[name].fill_(-100)
    if op == "preference":
        c["starts"][1:] = M
    c.update(old=None, ref=None)
    say("no row", op, M)
    for k in range(2):
        got, d = check(c)
        if k == 0:
            assert all(bool((t == 0).all()) for t in d)
            if op != "preference":
                assert all(bool((t == 0).all()) for t in got)
        c[name][-1] = was


def _step(op, c, h, W, b, kw):
    if op == "distill":
        return L.distillation(h, W, c["teacher_ids"], c["teacher_logits"], 0.5, b, **kw)
    if op == "policy":
        return L.policy_loss(h, W, c["target"], c["advantage"], c["old"], c["ref"], 0.5, b, **kw)
    return L.preference_loss(h, W, c["target"], c["starts"], c["ref"], 0.5, b, **kw)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("M", [200, 900])
def test_differentiable_captured_and_replayed(op, M):
    """The differentiable forms, with their means and their backward passes, in a
    graph; the number of rows trained on changes from replay to replay."""
    H, V, kw = 64, 700, KW[op]
    c = make(op, 73, M, H, V, "bf16", True, pairs=3)
    reference(c, 0.5, kw)
    new = lambda k: c[k].clone().requires_grad_(True)

    def grads(h, W, b):
        loss = _step(op, c, h, W, b, kw)
        return (loss.detach(), *torch.autograd.grad(loss, [h, W, b]))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            grads(new("hidden"), new("weight"), new("bias"))
    torch.cuda.current_stream().wait_stream(s)
    leaves = [new(k) for k in ("hidden", "weight", "bias")]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = grads(*leaves)
    for k in range(4):
        say("replay", op, M, k)
        c["hidden"].copy_(torch.randn(M, H, device=DEV) * (k + 1))
        leaves[0].data.copy_(c["hidden"])
        name = "teacher_ids" if op == "distill" else "target"
        c[name].copy_(torch.randint(0, V, c[name].shape, device=DEV))
        c[name][torch.rand(M, device=DEV) < 0.3 * k] = -100
        want = grads(new("hidden"), new("weight"), new("bias"))
        torch.cuda.synchronize()
        for t in out:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q)


def test_a_policy_step_with_a_tied_embedding():
    """Rollout, reference and update together: log-probabilities of the policy
    that sampled, the clipped loss, its gradient in the head's matrix with the
    embedding's added, and the candidates of the next token."""
    M, H, V = 300, 64, 2000
    c = make("policy", 79, M, H, V, "bf16", False)
    h, W = c["hidden"], c["weight"]
    zero = torch.zeros(M, device=DEV)
    _, old, none = L.policy_forward(h, W, c["target"], zero, train=False)
    xent, _ = L.xent_forward(h, W, c["target"])
    assert none is None and torch.equal(old, -xent)  # the cross entropy's own bits
    loss, logp, saved = L.policy_forward(h, W, c["target"], c["advantage"], old, old, kl_coef=0.1)
    assert torch.equal(logp, old)
    kept = c["target"] >= 0
    assert torch.equal(loss[kept], -c["advantage"][kept])  # ratio 1, no divergence
    dh, dw, _ = L.loss_backward(torch.full((M,), 1.0 / M, device=DEV), W, saved)
    want = dw.double().index_add_(0, c["target"][kept], dh[kept].double() * 2.0)
    got = L.embed_backward(dh[kept].contiguous(), c["target"][kept].contiguous(), V, 2.0, grad_weight=dw.clone())
    err = (got.double() - want).abs()
    # one more rounding of the sum, and of fp32 sums of at most M terms
    assert bool((err <= 2.0 ** -8 * want.abs() + M * 2.0 ** -24 * dh.double().abs().max() * 2 + 2.0 ** -126).all())
    values, ids, lse = L.logits_topk(L.logits(h, W), 5)
    assert float((values[:, 0] - lse).max()) <= 1e-6 and torch.equal(ids[:, 0], L.logits_rowreduce(h, W)[1])


def left_out(c):
    """The rows that a call leaves out."""
    V, M = c["weight"].shape[0], c["hidden"].shape[0]
    if c["op"] == "distill":
        return ~((c["teacher_ids"] >= 0) & (c["teacher_ids"] < V)).any(1)
    out = c["target"] == -100
    if c["op"] == "preference":
        at = torch.arange(M, device=DEV)
        out = out | (at < c["starts"][0]) | (at >= c["starts"][-1])
    return out


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [40, 64, 200, 300])
@pytest.mark.parametrize("op", OPS)
def test_what_stands_in_rows_that_are_left_out(op, M, bias, bad):
    """... does not matter, to the gradients either: hidden states of padding."""
    say(f"left out {op} M={M} bias={bias} {bad}")
    c = make(op, 40 + M, M, 96, 1300, "bf16", bias, K=70)
    if bias:
        c["bias"][5] = 120.0  # its exponential alone is none
    kw = KW[op]
    reference(c, 0.5, kw)
    spoilt = dict(c, hidden=c["hidden"].clone())
    out = left_out(c)
    assert 0 < int(out.sum()) < M
    spoilt["hidden"][out] = bad
    for keep in (True, False):
        *a, sa = call(c, 0.5, kw, keep_logits=keep)
        *b, sb = call(spoilt, 0.5, kw, keep_logits=keep)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        for x, y in zip(L.loss_backward(c["grad"], c["weight"], sa), L.loss_backward(c["grad"], c["weight"], sb)):
            assert x is y is None or (bool(torch.isfinite(y).all()) and torch.equal(x, y))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("M,V", [(200, 50001), (256, 41000), (256, 32769)])
def test_few_rows_on_a_large_vocabulary(op, M, V, bias):
    """Either side of where the rows' coefficients are found in a launch of their own."""
    say(f"{op} M={M} V={V} bias={bias}")
    check(make(op, M + V, M, 64, V, "bf16", bias, K=9))


def test_a_state_belongs_to_its_sizes():
    c = make("policy", 3, 20, 64, 1000, "bf16", False)
    reference(c, 0.5, KW["policy"])
    *_, saved = call(c, 0.5, KW["policy"])
    for V in (500, 1500):
        with pytest.raises(ValueError, match="saved"):
            L.loss_backward(c["grad"], torch.zeros(V, 64, dtype=torch.bfloat16, device=DEV), saved)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("op", OPS)
def test_differentiable_with_and_without_kept_logits(op, keep):
    c = make(op, 9, 50, 64, 700, "bf16", False)
    reference(c, 1.0, KW[op])
    fn = dict(distill=L.distillation, policy=L.policy_loss, preference=L.preference_loss)[op]
    args = dict(distill=("teacher_ids", "teacher_logits"), policy=("target", "advantage", "old", "ref"),
                preference=("target", "starts", "ref"))[op]
    got = []
    for more in (dict(), dict(keep_logits=keep)):
        h, w = c["hidden"].clone().requires_grad_(), c["weight"].clone().requires_grad_()
        fn(h, w, *[c[k] for k in args], reduction="sum", **KW[op], **more).backward()
        got.append((h.grad, w.grad))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("M", [20, 300])
def test_no_upstream_gradient_is_zeros(M):
    """The C call with grad_loss NULL."""
    from lm_head_logits_amd import _lib
    H, V = 64, 333
    c = make("policy", M, M, H, V, "bf16", True)
    reference(c, 0.5, KW["policy"])
    *_, s = call(c, 0.5, KW["policy"])
    dh, dw, db = torch.ones_like(c["hidden"]), torch.ones_like(c["weight"]), torch.ones_like(c["bias"])
    ws = torch.empty(L.loss_backward_workspace_bytes(M, H, V, 0, True, True), dtype=torch.uint8, device=DEV)
    st = _lib.load().lmhead_loss_backward(c["hidden"].data_ptr(), M, H, c["weight"].data_ptr(), V, 0.5, c["bias"].data_ptr(),
                                          _lib.LMHEAD_BF16, 1.0, 0, None, s.state.data_ptr(), s.state.numel(), 1,
                                          dh.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(),
                                          torch.cuda.current_stream().cuda_stream)
    assert st == _lib.OK and all(bool((t == 0).all()) for t in (dh, dw, db))
