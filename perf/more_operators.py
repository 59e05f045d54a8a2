"""Further operators over the vocabulary matrix W [V, H], as measured cases.

Four operators of tuning a model against a teacher, a reward or preferences:

- ``topk``: the k largest logits of each row with their tokens (equal logits:
  the lower token first), and the row's log-sum-exp at a temperature;
- ``distill``: the head's divergence from a teacher's top logits, and
  (``train``) its gradients for h, W and b;
- ``policy``: the clipped policy loss of the head's token log-probabilities
  with a KL term against a reference, and its gradients;
- ``preference``: the logistic loss of paired sequences' log ratios, and its
  gradients.

In the last three the logits are t = (alpha h W^T + b) / temperature. Rows that
are not trained on (prompts, padding) are part of the batch. ``own`` selects
what ``run`` computes: the plain form in elementary torch operations, or the
library's calls.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda", 0)
else:
    DEV = torch.device("cpu")

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORE = -100  # target of a token that is not trained on
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
KL = 0.04


def listed():
    return [
        # the alternatives shown beside one served token: latency
        dict(name="topk_token", op="topk", M=1, V=151936, K=20, dtype="f32", temperature=1.0),
        # the candidates of a decode batch, to be sampled from
        dict(name="topk_batch", op="topk", M=48, V=128256, K=50, dtype="bf16", temperature=0.7),
        # a teacher's top logits for a training batch (16-bit logits: many are equal)
        dict(name="topk_teacher", op="topk", M=4096, V=128256, K=64, dtype="bf16", temperature=1.0),
        # the smallest head the benchmark has: a unit test's or a toy model's step, bound by launches
        dict(name="distill_tiny", op="distill", M=37, H=256, V=4096, K=16, dtype="bf16", bias=False, alpha=0.25,
             temperature=2.0, whole=False, mask=0.0, train=True),
        # chat data with prompts left out, fp16, a head with a bias, the teacher's mass outside its top logits known
        dict(name="distill_train_bias", op="distill", M=1001, H=2048, V=151936, K=50, dtype="f16", bias=True, alpha=1.0,
             temperature=1.0, whole=True, mask=0.3, train=True),
        # a training micro-batch on the decode head, every token trained on
        dict(name="distill_train_large", op="distill", M=4096, H=4096, V=128256, K=64, dtype="bf16", bias=False,
             alpha=0.125, temperature=1.0, whole=False, mask=0.0, train=True),
        # a toy model's policy step
        dict(name="policy_tiny", op="policy", M=200, H=256, V=4096, dtype="bf16", bias=False, alpha=0.25, temperature=1.0,
             mask=0.4, train=True),
        # responses of odd lengths, fp16, sampled at another temperature than 1, a head with a bias
        dict(name="policy_train_bias", op="policy", M=1501, H=2048, V=151936, dtype="f16", bias=True, alpha=1.0,
             temperature=0.8, mask=0.3, train=True),
        # a micro-batch of rollouts on the decode head: prompts and padding are two fifths of it
        dict(name="policy_train_large", op="policy", M=4096, H=4096, V=128256, dtype="bf16", bias=False, alpha=0.125,
             temperature=1.0, mask=0.4, train=True),
        # evaluating a few pairs, length-normalised, without a reference: the loss alone
        dict(name="preference_score", op="preference", M=333, pairs=2, H=4096, V=128256, dtype="f16", bias=False,
             alpha=0.125, ref=False, average=True, mask=0.4, train=False),
        # a fine-tuning step's pairs, ragged
        dict(name="preference_train_bias", op="preference", M=1337, pairs=4, H=2048, V=151936, dtype="bf16", bias=True,
             alpha=1.0, ref=True, average=False, mask=0.4, train=True),
        # a micro-batch of pairs on the decode head, short answers to long prompts
        dict(name="preference_train_large", op="preference", M=4096, pairs=8, H=4096, V=128256, dtype="bf16", bias=False,
             alpha=0.125, ref=True, average=False, mask=0.55, train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "distill", "policy", "preference"])
    V = _log_int(rng, 4001, 151936)
    if op == "topk":
        return dict(op=op, M=_log_int(rng, 1, 3400), V=V, K=_log_int(rng, 1, 256),
                    dtype=rng.choice(["bf16", "f16", "f32"]), temperature=rng.choice([1.0, 0.7]))
    H = 32 * _log_int(rng, 8, 128)
    case = dict(op=op, M=_log_int(rng, 60, 4096), H=H, V=V, dtype=rng.choice(["bf16", "bf16", "f16"]),
                bias=rng.random() < 0.5, alpha=rng.choice([1.0, 0.25, 0.125]), mask=rng.choice([0.0, 0.3, 0.6]),
                train=rng.random() < 0.75)
    while case["M"] * H * V > 4096 * 4096 * 128256:
        case["M"] = max(1, case["M"] // 2)
    if op == "distill":
        case.update(K=_log_int(rng, 4, 128), temperature=rng.choice([1.0, 2.0]), whole=rng.random() < 0.5)
    elif op == "policy":
        case.update(temperature=rng.choice([1.0, 0.8]))
    else:
        case.update(pairs=max(2, min(16, case["M"] // 100)), ref=rng.random() < 0.7, average=rng.random() < 0.3)
    return case


def _tokens(g, *shape, V):
    """Token ids with a word-like distribution (density ~ 1 / rank), the ranks spread over the vocabulary."""
    u = torch.rand(*shape, generator=g, device=DEV, dtype=torch.float64)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return (rank * 7919 + 13) % V


def _cuts(g, M, S, rest):
    """Bounds [S + 1] of S sequences of uneven lengths over the first M - rest rows."""
    share = torch.rand(S, generator=g, device=DEV, dtype=torch.float64) + 0.5
    cut = torch.cumsum(share, 0) / share.sum() * (M - rest)
    return torch.cat([torch.zeros(1, device=DEV, dtype=torch.float64), cut]).round().long()


def _trained(g, M, S, mask, rest):
    """(bounds, rows trained on): a share of about `mask` of each sequence, its prompt, is not."""
    cuts = _cuts(g, M, S, rest)
    row = torch.arange(M, device=DEV)
    seq = (torch.searchsorted(cuts, row, right=True) - 1).clamp(0, S - 1)
    prompt = (cuts[1:] - cuts[:-1]) * (torch.rand(S, generator=g, device=DEV, dtype=torch.float64) * 0.4 + 0.8) * mask
    return cuts, (row - cuts[seq] >= prompt[seq]) & (row < cuts[-1]), seq


def _logp(s, rows=1024):
    """The tokens' log-probabilities as the program that made the batch had them, in 64 bits past the product."""
    out = []
    bias = 0.0 if s["bias"] is None else s["bias"]
    for r in range(0, len(s["target"]), rows):
        t = (s["hidden"][r:r + rows].float() @ s["weight"].float().t() * s["alpha"] + bias) / s["temperature"]
        y = s["target"][r:r + rows].clamp(0)[:, None]
        m = t.amax(1, keepdim=True)
        out.append((t.gather(1, y) - m)[:, 0].double() - torch.exp(t - m).sum(1, dtype=torch.float64).log())
    return torch.cat(out)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, M, V = case["op"], case["M"], case["V"]

    def normal(*shape, **kw):
        return torch.randn(*shape, generator=g, device=DEV, **kw)

    s = dict(op=op, case=dict(case))
    if op == "topk":
        # what a head gives: most logits in a bell, some tokens well above
        x = normal(M, V).mul_(2.0)
        x.scatter_add_(1, _tokens(g, M, 8, V=V), torch.rand(M, 8, generator=g, device=DEV).mul_(12.0))
        s.update(logits=x.to(DTYPES[case["dtype"]]), K=case["K"], temperature=case["temperature"])
        return s

    H, alpha, dt = case["H"], case["alpha"], DTYPES[case["dtype"]]
    W = normal(V, H).mul_(0.02).to(dt)
    lean = 1.0 / (0.0004 * H * alpha)  # of h towards a token's row, for a logit one higher
    s.update(weight=W, bias=normal(V).mul_(0.1) if case["bias"] else None, alpha=alpha,
             temperature=case.get("temperature", 1.0), train=case["train"])
    if op == "distill":
        # the teacher sees a few likely tokens; the student leans towards some of them
        y = _tokens(g, M, 4, V=V)
        push = torch.rand(M, 4, generator=g, device=DEV) * 9.0 + 3.0
        noise, teacher = normal(M, H), torch.zeros(M, H, device=DEV)
        student = torch.zeros(M, H, device=DEV)
        for j in range(4):
            row = W[y[:, j]].float() * (lean * push[:, j, None])
            teacher += row
            student += row * (torch.rand(M, 1, generator=g, device=DEV) * 0.9 + 0.1)
        s["hidden"] = (noise + student).to(dt)
        t = ((noise + teacher).to(dt) @ W.t()).float().mul_(alpha)
        t += normal(V).mul_(0.5)
        top, ids = torch.topk(t, case["K"], dim=1)
        s["teacher_lse"] = torch.logsumexp(t / s["temperature"], 1) if case["whole"] else None
        del t
        if case["mask"]:
            _, kept, _ = _trained(g, M, max(1, M // 300), case["mask"], 0)
            ids = torch.where(kept[:, None], ids, torch.full_like(ids, IGNORE))
        s.update(teacher_ids=ids.int(), teacher_logits=top)
        n = M
    else:
        y = _tokens(g, M, V=V)
        push = torch.rand(M, generator=g, device=DEV) * 9.0 + 4.0
        s["hidden"] = (normal(M, H) + W[y].float() * (lean * push[:, None])).to(dt)
        S = 2 * case["pairs"] if op == "preference" else max(1, M // 300)
        cuts, kept, seq = _trained(g, M, S, case["mask"], M // 20 if op == "preference" else 0)
        s["target"] = torch.where(kept, y, torch.full_like(y, IGNORE))
        logp = torch.where(kept, _logp(s), torch.zeros(M, device=DEV, dtype=torch.float64))
        if op == "policy":
            # the policy has moved a little since the rollout; no ratio lies on a border of the clip, where
            # two right answers differ
            moved = normal(M, dtype=torch.float64) * 0.15
            for border in (math.log1p(-CLIP_LOW), math.log1p(CLIP_HIGH)):
                near = (moved - border).abs() < 1e-3
                moved = torch.where(near, moved + 3e-3, moved)
            s.update(old_logp=(logp - moved).float(), ref_logp=(logp + normal(M, dtype=torch.float64) * 0.3).float(),
                     advantage=normal(S)[seq].contiguous())
            n = M
        else:
            n = case["pairs"]
            total = torch.zeros(S, device=DEV, dtype=torch.float64).index_add_(0, seq, logp)
            s.update(starts=cuts, beta=2.0 if case["average"] else 0.1, average=case["average"],
                     margin=0.3 if case["average"] else 0.0, smoothing=0.0 if case["average"] else 0.1,
                     ref_logp=None)
            if case["ref"]:
                drift = normal(S, dtype=torch.float64) * 6.0
                if case["average"]:
                    count = torch.zeros(S, device=DEV, dtype=torch.float64).index_add_(0, seq, kept.double())
                    total, drift = total / count.clamp(min=1.0), drift / 20.0
                s["ref_logp"] = (total - drift).float()
    if case["train"]:  # of the mean over the batch, as the loss hands it down; fp16 with loss scaling
        s["grad_loss"] = torch.full((n,), (1.0 if dt is torch.bfloat16 else 4096.0) / n, device=DEV)
    return s


def run(state):
    return _own_run(state) if own else _plain_run(state)


def _own_run(s):
    import lm_head_logits_amd as L

    if s["op"] == "topk":
        values, ids, lse = L.logits_topk(s["logits"], s["K"], s["temperature"])
        return dict(values=values, ids=ids, lse=lse)
    train = s["train"]
    if s["op"] == "distill":
        loss, saved = L.distill_forward(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logits"], s["alpha"],
                                        s["bias"], temperature=s["temperature"], teacher_lse=s["teacher_lse"],
                                        train=train)
        out = dict(loss=loss)
    elif s["op"] == "policy":
        loss, logp, saved = L.policy_forward(s["hidden"], s["weight"], s["target"], s["advantage"], s["old_logp"],
                                             s["ref_logp"], s["alpha"], s["bias"], temperature=s["temperature"],
                                             clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL, ignore_index=IGNORE,
                                             train=train)
        out = dict(loss=loss, logp=logp)
    else:
        loss, logp, saved = L.preference_forward(s["hidden"], s["weight"], s["target"], s["starts"], s["ref_logp"],
                                                 s["alpha"], s["bias"], beta=s["beta"], margin=s["margin"],
                                                 label_smoothing=s["smoothing"], average=s["average"],
                                                 ignore_index=IGNORE, train=train)
        out = dict(loss=loss, logp=logp)
    if train:
        dh, dw, db = L.loss_backward(s["grad_loss"], s["weight"], saved)
        out.update(grad_hidden=dh, grad_weight=dw, grad_bias=db)
    return out


def _plain_run(s):
    if s["op"] == "topk":
        return _plain_topk(s)
    h, W, b = s["hidden"].float(), s["weight"].float(), s["bias"]
    t = h @ W.t() * s["alpha"]
    if b is not None:
        t = t + b
    t = t / s["temperature"]
    m = t.amax(1, keepdim=True)
    logq = (t - m) - torch.log(torch.exp(t - m).sum(1, keepdim=True))
    if s["op"] == "distill":
        out, G = _plain_distill(s, logq)
    else:
        keep = s["target"] != IGNORE
        at = torch.where(keep, s["target"], torch.zeros_like(s["target"]))[:, None]
        logp = torch.where(keep, logq.gather(1, at)[:, 0], torch.zeros_like(m[:, 0]))
        out, c = _plain_policy(s, logp, keep) if s["op"] == "policy" else _plain_preference(s, logp, keep)
        if s["train"]:  # c: the loss's derivative by the token's log-probability
            G = torch.exp(logq) * -c[:, None]
            G.scatter_add_(1, at, c[:, None])
    if s["train"]:
        k = s["alpha"] / s["temperature"]
        out.update(grad_hidden=(G @ W * k).to(s["hidden"].dtype), grad_weight=(G.t() @ h * k).to(s["hidden"].dtype),
                   grad_bias=G.sum(0) / s["temperature"] if b is not None else None)
    return out


def _plain_topk(s):
    x = s["logits"].float()
    V = x.shape[1]
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits, bits)  # whole numbers in the logits' order
    key = order * 1048576 + (1048575 - torch.arange(V, device=x.device))
    ids = 1048575 - torch.topk(key, s["K"], dim=1).values % 1048576
    t = x / s["temperature"]
    m = t.amax(1, keepdim=True)
    return dict(values=s["logits"].gather(1, ids), ids=ids.int(), lse=torch.log(torch.exp(t - m).sum(1)) + m[:, 0])


def _plain_distill(s, logq):
    ids, top = s["teacher_ids"].long(), s["teacher_logits"].float() / s["temperature"]
    keep = ids >= 0
    at = torch.where(keep, ids, torch.zeros_like(ids))
    if s["teacher_lse"] is None:
        m = top.amax(1, keepdim=True)
        logp = (top - m) - torch.log(torch.where(keep, torch.exp(top - m), torch.zeros_like(top)).sum(1, keepdim=True))
    else:
        logp = top - s["teacher_lse"][:, None]
    p = torch.where(keep, torch.exp(logp), torch.zeros_like(top))
    loss = torch.where(keep, p * (logp - logq.gather(1, at)), torch.zeros_like(top)).sum(1)
    if not s["train"]:
        return dict(loss=loss), None
    g = s["grad_loss"][:, None]
    G = torch.exp(logq) * (p.sum(1, keepdim=True) * g)
    G.scatter_add_(1, at, p * -g)
    return dict(loss=loss), G


def _plain_policy(s, logp, keep):
    A = s["advantage"]
    ratio = torch.exp(logp - s["old_logp"])
    clipped = torch.clamp(ratio, 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * A
    d = s["ref_logp"] - logp
    zero = torch.zeros_like(logp)
    loss = torch.where(keep, KL * (torch.exp(d) - d - 1.0) - torch.minimum(ratio * A, clipped), zero)
    out = dict(loss=loss, logp=logp)
    if not s["train"]:
        return out, None
    c = KL * (1.0 - torch.exp(d)) - torch.where(ratio * A <= clipped, ratio * A, zero)
    return out, torch.where(keep, c * s["grad_loss"], zero)


def _plain_preference(s, logp, keep):
    starts, n = s["starts"], len(s["starts"]) // 2
    zero = torch.zeros(1, device=logp.device, dtype=torch.float64)
    run = torch.cat([zero, torch.cumsum(logp.double(), 0)])  # long sums, differences of which are wanted
    seq = run[starts[1:]] - run[starts[:-1]]
    size = torch.ones_like(seq)
    if s["average"]:
        have = torch.cat([zero, torch.cumsum(keep.double(), 0)])
        size = (have[starts[1:]] - have[starts[:-1]]).clamp(min=1.0)
        seq = seq / size
    lead = seq if s["ref_logp"] is None else seq - s["ref_logp"].double()
    z = (s["beta"] * (lead[:n] - lead[n:]) - s["margin"]).float()
    e = s["smoothing"]
    soft = torch.log(1.0 + torch.exp(-z.abs()))
    loss = (1.0 - e) * (torch.clamp(-z, min=0.0) + soft) + e * (torch.clamp(z, min=0.0) + soft)
    out = dict(loss=loss, logp=seq.float())
    if not s["train"]:
        return out, None
    dz = (e - 1.0 / (1.0 + torch.exp(z))) * s["grad_loss"] * s["beta"]
    c = torch.cat([dz, -dz]) / size.float()
    row = torch.arange(len(logp), device=logp.device)
    at = torch.searchsorted(starts, row, right=True) - 1
    inside = keep & (at >= 0) & (at < 2 * n)
    return out, torch.where(inside, c[at.clamp(0, 2 * n - 1)], torch.zeros_like(logp))


def work(case):
    M, V, op = case["M"], case["V"], case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "topk":
        return {"bytes": M * (V * e + case["K"] * (e + 4) + 4), "flops": 3 * M * V}
    H = case["H"]
    n = max(1, int(round(M * (1.0 - case["mask"]) * (0.95 if op == "preference" else 1.0))))  # rows trained on
    b = 2 * (n * H + V * H) + (4 * V if case["bias"] else 0) + (8 * M * case["K"] + 4 * M if op == "distill" else 20 * M)
    if case["train"]:
        b += 2 * (M * H + V * H) + (4 * V if case["bias"] else 0)
    return {"bytes": b, "flops": 2 * n * H * V * (3 if case["train"] else 1)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "topk":
        values, ids, lse = [], [], []
        for r in range(0, case["M"], 512):
            x = s["logits"][r:r + 512].double()
            v, i = torch.sort(x, dim=1, descending=True, stable=True)
            values.append(v[:, :case["K"]].clone())
            ids.append(i[:, :case["K"]].int())
            lse.append(torch.logsumexp(x / case["temperature"], 1))
        return dict(values=torch.cat(values), ids=torch.cat(ids), lse=torch.cat(lse))
    return _exact_loss(s, case)


def _exact_loss(s, case):
    M, H, V, op, train = case["M"], case["H"], case["V"], case["op"], case["train"]
    f64 = dict(dtype=torch.float64, device=DEV)
    Wd, T = s["weight"].double(), s["temperature"]

    def logits(r):
        t = torch.mm(s["hidden"][r:r + 512].double(), Wd.t()) * case["alpha"]
        if s["bias"] is not None:
            t += s["bias"].double()
        return t.div_(T)

    def logp_of(logq, r):  # of the rows' targets, 0 where there is none
        y = s["target"][r:r + 512]
        rows = torch.nonzero(y != IGNORE)[:, 0]
        out = torch.zeros(len(y), **f64)
        out[rows] = logq[rows, y[rows]]
        return out

    out = {}
    if op != "distill":
        logp = torch.cat([logp_of(torch.log_softmax(logits(r), 1), r) for r in range(0, M, 512)])
        kept = s["target"] != IGNORE
        leaf = logp.clone().requires_grad_(train)
        if op == "policy":
            ratio = torch.exp(leaf - s["old_logp"].double())
            A = s["advantage"].double()
            held = torch.where(A >= 0, torch.minimum(ratio, torch.full_like(ratio, 1 + CLIP_HIGH)),
                               torch.maximum(ratio, torch.full_like(ratio, 1 - CLIP_LOW)))
            d = s["ref_logp"].double() - leaf
            loss = (KL * (torch.expm1(d) - d) - held * A) * kept
            out.update(loss=loss.detach(), logp=logp)
        else:
            n = case["pairs"]
            seqs = [slice(int(a), int(b)) for a, b in zip(s["starts"][:-1], s["starts"][1:])]
            total = torch.stack([leaf[q].sum() for q in seqs])
            if case["average"]:
                total = total / torch.stack([kept[q].sum().clamp(min=1) for q in seqs])
            lead = total if s["ref_logp"] is None else total - s["ref_logp"].double()
            z = s["beta"] * (lead[:n] - lead[n:]) - s["margin"]
            sig = torch.nn.functional.logsigmoid
            loss = -(1 - s["smoothing"]) * sig(z) - s["smoothing"] * sig(-z)
            out.update(loss=loss.detach(), logp=total.detach())
        if train:
            (c,) = torch.autograd.grad((loss * s["grad_loss"].double()).sum(), leaf)
            c = c * kept  # a row left out has no log-probability to move
    dh, dw, db = torch.empty(M, H, **f64), torch.zeros(V, H, **f64) if train else None, torch.zeros(V, **f64)
    losses = []
    for r in range(0, M, 512):
        if op != "distill" and not train:
            break
        logq, hd = torch.log_softmax(logits(r), 1), s["hidden"][r:r + 512].double()
        if op == "distill":
            ids, top = s["teacher_ids"][r:r + 512].long(), s["teacher_logits"][r:r + 512].double() / T
            top = torch.where(ids >= 0, top, torch.full_like(top, -math.inf))
            whole = torch.logsumexp(top, 1) if s["teacher_lse"] is None else s["teacher_lse"][r:r + 512].double()
            p = torch.nan_to_num(torch.exp(top - whole[:, None]))
            full = torch.zeros_like(logq).scatter_add_(1, ids.clamp(0), p)  # ids of a row are distinct, or absent
            losses.append((torch.special.xlogy(full, full) - full * logq).sum(1))
            if train:
                G = (logq.exp() * full.sum(1, keepdim=True) - full) * s["grad_loss"][r:r + 512, None].double()
        else:
            G = logq.exp() * -c[r:r + 512, None]
            rows = torch.nonzero(s["target"][r:r + 512] != IGNORE)[:, 0]
            G[rows, s["target"][r:r + 512][rows]] += c[r:r + 512][rows]
        if train:
            dh[r:r + 512] = torch.mm(G, Wd) * (case["alpha"] / T)
            dw += torch.mm(G.t(), hd) * (case["alpha"] / T)
            db += G.sum(0) / T
    if losses:
        out["loss"] = torch.cat(losses)
    if train:
        out.update(grad_hidden=dh, grad_weight=dw, grad_bias=db if s["bias"] is not None else None)
    return out
