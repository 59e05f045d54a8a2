"""The training and 8-bit operators of the vocabulary matrix W [V, H], as measured cases.

Four operators:

- ``xent``: softmax cross entropy of the head's logits alpha h W^T + b against
  target tokens, and (``train``) its gradients for h, W and b;
- ``embed``: the embedding lookup, scale * W[ids];
- ``embed_grad``: the lookup's gradient for W, dense;
- ``int8``: per-token int8 quantisation of h and the product with a head held
  in int8 with a scale per vocabulary row.

``own`` selects what ``run`` computes: the plain form in elementary torch
operations, or the library's calls.
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


def listed():
    return [
        # the smallest head the benchmark has: a unit test's or a toy model's step, bound by launches
        dict(name="xent_train_tiny", op="xent", M=37, H=256, V=4096, dtype="bf16", bias=False, alpha=0.25, train=True),
        # scoring a prompt (perplexity, reward): the loss alone, fp16, an odd number of tokens
        dict(name="xent_score_f16", op="xent", M=333, H=4096, V=128256, dtype="f16", bias=False, alpha=0.125, train=False),
        # a fine-tuning step's head with a bias, ragged rows
        dict(name="xent_train_bias", op="xent", M=1001, H=2048, V=151936, dtype="bf16", bias=True, alpha=1.0, train=True),
        # a training micro-batch of 4096 tokens on the decode head
        dict(name="xent_train_large", op="xent", M=4096, H=4096, V=128256, dtype="bf16", bias=False, alpha=0.125, train=True),
        # the tokens of one decode step: latency
        dict(name="embed_decode", op="embed", M=64, H=4096, V=128256, dtype="bf16", scale=1.0),
        # a training micro-batch, scaled by sqrt(H)
        dict(name="embed_train", op="embed", M=8192, H=4096, V=128256, dtype="bf16", scale=64.0),
        # its gradient; tokens as frequent as words are
        dict(name="embed_grad", op="embed_grad", M=8192, H=4096, V=128256, dtype="bf16", scale=64.0, pad=0.0),
        # a padded batch: half of the positions hold one token, an odd count, fp16
        dict(name="embed_grad_padded", op="embed_grad", M=30011, H=2048, V=151936, dtype="f16", scale=1.0, pad=0.5),
        # decode of one sequence, and of a batch
        dict(name="int8_one", op="int8", M=1, H=4096, V=128256, out="bf16", bias=False),
        dict(name="int8_batch", op="int8", M=48, H=4096, V=128256, out="f32", bias=True),
        # speculative verification rows
        dict(name="int8_verify", op="int8", M=130, H=2048, V=151936, out="bf16", bias=False),
        # prefill with logits for every token
        dict(name="int8_prefill", op="int8", M=2048, H=4096, V=151936, out="bf16", bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "xent", "embed", "embed_grad", "int8", "int8"])
    H = 32 * _log_int(rng, 8, 128)
    V = _log_int(rng, 4001, 151936)
    case = dict(op=op, H=H, V=V)
    if op == "xent":
        case.update(M=_log_int(rng, 1, 4096), dtype=rng.choice(["bf16", "bf16", "f16"]), bias=rng.random() < 0.5,
                    alpha=rng.choice([1.0, 0.25, 0.125]), train=rng.random() < 0.7)
        while case["M"] * H * case["V"] > 4096 * 4096 * 128256:
            case["M"] = max(1, case["M"] // 2)
    elif op == "int8":
        case.update(M=_log_int(rng, 1, 2048), out=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    else:
        case.update(M=_log_int(rng, 1, 30011), dtype=rng.choice(["bf16", "f16"]), scale=rng.choice([1.0, 64.0]))
        if op == "embed_grad":
            case.update(pad=rng.choice([0.0, 0.0, 0.5]))
    return case


def _tokens(g, M, V):
    """Token ids with a word-like distribution (density ~ 1 / rank), the ranks spread over the vocabulary."""
    u = torch.rand(M, generator=g, device=DEV, dtype=torch.float64)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return (rank * 7919 + 13) % V


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    M, H, V, op = case["M"], case["H"], case["V"], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = dict(op=op, case=dict(case))
    if op == "xent":
        dt = DTYPES[case["dtype"]]
        W = normal(V, H).mul_(0.02).to(dt)
        y = _tokens(g, M, V)
        # a model that has learned something: its hidden state leans towards the target's row
        h = normal(M, H) + W[y].float() * (6.0 / (0.0004 * H * case["alpha"]))
        y[torch.rand(M, generator=g, device=DEV) < 0.05] = IGNORE
        s.update(hidden=h.to(dt), weight=W, target=y, alpha=case["alpha"],
                 bias=normal(V).mul_(0.1) if case["bias"] else None, train=case["train"])
        if case["train"]:  # of the mean over the batch, as the loss above the head hands it down; fp16 with loss scaling
            s["grad_loss"] = torch.full((M,), (1.0 if dt is torch.bfloat16 else 4096.0) / M, device=DEV)
    elif op == "int8":
        s.update(hidden=normal(M, H).to(torch.bfloat16),
                 weight_q=torch.randint(-127, 128, (V, H), generator=g, device=DEV, dtype=torch.int8),
                 weight_scale=torch.rand(V, generator=g, device=DEV).mul_(2e-4).add_(4e-4),
                 bias=normal(V).mul_(0.1) if case["bias"] else None, out=DTYPES[case["out"]])
    else:
        dt = DTYPES[case["dtype"]]
        ids = _tokens(g, M, V)
        if op == "embed":
            s.update(ids=ids, weight=normal(V, H).mul_(0.02).to(dt), scale=case["scale"])
        else:
            if case["pad"]:
                ids[torch.rand(M, generator=g, device=DEV) < case["pad"]] = 1
            s.update(ids=ids, grad_out=normal(M, H).mul_(1e-2).to(dt), V=V, scale=case["scale"])
    return s


def run(state):
    return _own_run(state) if own else _plain_run(state)


def _own_run(s):
    import lm_head_logits_amd as L

    if s["op"] == "xent":
        loss, lse = L.xent_forward(s["hidden"], s["weight"], s["target"], s["alpha"], s["bias"], ignore_index=IGNORE)
        if not s["train"]:
            return dict(loss=loss, lse=lse)
        dh, dw, db = L.xent_backward(s["grad_loss"], s["hidden"], s["weight"], s["target"], lse, s["alpha"], s["bias"],
                                     ignore_index=IGNORE)
        return dict(loss=loss, lse=lse, grad_hidden=dh, grad_weight=dw, grad_bias=db)
    if s["op"] == "embed":
        return dict(out=L.embed(s["ids"], s["weight"], s["scale"]))
    if s["op"] == "embed_grad":
        return dict(grad_weight=L.embed_backward(s["grad_out"], s["ids"], s["V"], s["scale"]))
    q, scale = L.quantize_int8(s["hidden"])
    return dict(logits=L.logits_int8(q, scale, s["weight_q"], s["weight_scale"], bias=s["bias"], out_dtype=s["out"]),
                codes=q, scale=scale)


def _plain_run(s):
    if s["op"] == "xent":
        return _plain_xent(s)
    if s["op"] == "embed":
        return dict(out=(s["weight"][s["ids"]].float() * s["scale"]).to(s["weight"].dtype))
    if s["op"] == "embed_grad":
        gw = torch.zeros(s["V"], s["grad_out"].shape[1], device=s["ids"].device)
        gw.index_add_(0, s["ids"], s["grad_out"].float())
        return dict(grad_weight=(gw * s["scale"]).to(s["grad_out"].dtype))
    x = s["hidden"].float()
    amax = x.abs().amax(1)
    scale = amax / torch.full_like(amax, 127.0)  # a tensor: a true division, not a product with 1/127
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = torch.round(x / scale[:, None]).clamp(-127, 127)
    t = (q @ s["weight_q"].float().t()) * scale[:, None] * s["weight_scale"]
    if s["bias"] is not None:
        t = t + s["bias"]
    return dict(logits=t.to(s["out"]), codes=q.to(torch.int8), scale=scale)


def _plain_xent(s):
    h, W, y, dt = s["hidden"].float(), s["weight"].float(), s["target"], s["hidden"].dtype
    t = h @ W.t() * s["alpha"]
    if s["bias"] is not None:
        t = t + s["bias"]
    keep = y != IGNORE
    at = torch.where(keep, y, torch.zeros_like(y))[:, None]
    m = t.amax(1, keepdim=True)
    lse = torch.log(torch.exp(t - m).sum(1)) + m[:, 0]
    loss = torch.where(keep, lse - t.gather(1, at)[:, 0], torch.zeros_like(lse))
    if not s["train"]:
        return dict(loss=loss, lse=lse)
    g = torch.where(keep, s["grad_loss"], torch.zeros_like(s["grad_loss"]))[:, None]
    G = torch.exp(t - lse[:, None]) * g
    G.scatter_add_(1, at, -g)
    return dict(loss=loss, lse=lse, grad_hidden=(G @ W * s["alpha"]).to(dt), grad_weight=(G.t() @ h * s["alpha"]).to(dt),
                grad_bias=G.sum(0) if s["bias"] is not None else None)


def work(case):
    M, H, V, op = case["M"], case["H"], case["V"], case["op"]
    if op == "xent":
        n = 3 if case["train"] else 1  # the product, and one for each of the two gradients
        b = 2 * (M * H + V * H) + 8 * M + 8 * M + (4 * V if case["bias"] else 0)
        if case["train"]:
            b += 2 * (M * H + V * H) + 4 * M + (4 * V if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * H * V * n}
    if op == "embed":
        return {"bytes": M * (8 + 4 * H), "flops": M * H}
    if op == "embed_grad":
        return {"bytes": M * (8 + 2 * H) + 2 * V * H, "flops": M * H}
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": 2 * M * H + M * H + 4 * M + V * H + 4 * V + M * V * out + (4 * V if case["bias"] else 0),
            "flops": 2 * M * H * V}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "xent":
        return _exact_xent(s, case)
    if case["op"] == "embed":
        return dict(out=torch.index_select(s["weight"], 0, s["ids"]).double().mul_(case["scale"]))
    if case["op"] == "embed_grad":
        d = s["grad_out"].double() * case["scale"]
        return dict(grad_weight=torch.zeros(case["V"], case["H"], dtype=torch.float64, device=DEV)
                    .index_put_((s["ids"],), d, accumulate=True))
    # the scale and the codes are what they are defined as in 32 bits; the product from there on in 64
    x = s["hidden"].double()
    scale = (x.abs().max(1).values / 127.0).float()
    scale[scale == 0] = 1.0
    q = (x / scale.double()[:, None]).float().round().double()
    out = torch.empty(case["M"], case["V"], dtype=torch.float64, device=DEV)
    for v in range(0, case["V"], 16384):  # exact: every sum is a whole number below 2^53
        w = s["weight_q"][v:v + 16384].double() * s["weight_scale"][v:v + 16384].double()[:, None]
        out[:, v:v + 16384] = (q * scale.double()[:, None]) @ w.t()
    if s["bias"] is not None:
        out += s["bias"].double()
    return dict(logits=out, codes=None, scale=scale.double())


def _exact_xent(s, case):
    M, H, V = case["M"], case["H"], case["V"]
    f64 = dict(dtype=torch.float64, device=DEV)
    Wd, train = s["weight"].double(), case["train"]
    loss, lse = torch.empty(M, **f64), torch.empty(M, **f64)
    dh, dw = torch.empty(M, H, **f64), torch.zeros(V, H, **f64) if train else None
    db = torch.zeros(V, **f64)
    for r in range(0, M, 1024):
        h, y = s["hidden"][r:r + 1024].double(), s["target"][r:r + 1024]
        t = torch.mm(h, Wd.t()).mul_(case["alpha"])
        if s["bias"] is not None:
            t += s["bias"].double()
        logp = torch.log_softmax(t, 1)
        lse[r:r + 1024] = torch.logsumexp(t, 1)
        rows = torch.nonzero(y != IGNORE)[:, 0]
        one = torch.zeros_like(t)
        one[rows, y[rows]] = 1.0
        loss[r:r + 1024] = -(logp * one).sum(1)
        if train:
            g = torch.zeros(len(y), 1, **f64)
            g[rows, 0] = s["grad_loss"][r:r + 1024].double()[rows]
            d = (logp.exp() - one) * g
            dh[r:r + 1024] = torch.mm(d, Wd) * case["alpha"]
            dw += torch.mm(d.t(), h) * case["alpha"]
            db += d.sum(0)
    if not train:
        return dict(loss=loss, lse=lse)
    return dict(loss=loss, lse=lse, grad_hidden=dh, grad_weight=dw, grad_bias=db if s["bias"] is not None else None)
