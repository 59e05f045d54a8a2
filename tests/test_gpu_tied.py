"""A training step of a model whose embedding and head are one matrix, as the
operators are used together: lookup, (a stand-in for the model) an elementwise
map, cross entropy, and the matrix's gradient from both ends."""
import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_tied_step(dt):
    B, S, V, H, scale, alpha = 3, 33, 1000, 64, 8.0, 0.5
    say("tied step", dt)
    g = torch.Generator(device=DEV).manual_seed(1)
    W = (torch.randn(V, H, generator=g, device=DEV) * 0.1).to(dt)
    ids = torch.randint(0, V, (B, S), generator=g, device=DEV)
    ids[:, 25:] = 0  # padding
    tgt = torch.roll(ids, -1, 1)
    tgt[:, 24:] = -100
    k = (torch.rand(H, generator=g, device=DEV) + 0.5).to(dt)
    up = 1.0 if dt == torch.bfloat16 else 256.0  # loss scaling

    Wl = W.clone().requires_grad_(True)
    x = L.embedding(ids, Wl, scale, padding_idx=0)
    loss = L.cross_entropy((x * k).view(-1, H), Wl, tgt.view(-1), alpha)
    (loss * up).backward()

    # the same from the calls, the head's gradient first and the embedding's added
    e = L.embed(ids, W, scale)
    h = (e * k).view(-1, H)
    l, lse = L.xent_forward(h, W, tgt.view(-1), alpha)
    n = (tgt != -100).sum()
    dh, dw, _ = L.xent_backward(torch.full((B * S,), up, device=DEV) / n, h, W, tgt.view(-1), lse, alpha)
    L.embed_backward(dh.view(B, S, H) * k, ids, V, scale, padding_idx=0, grad_weight=dw)
    assert float(l.sum() / n) == float(loss)

    # 64 bits, with the 16-bit values the step itself has (the products x * k)
    W64 = W.double().requires_grad_(True)
    keep = (tgt.view(-1) != -100)
    logits = alpha * h.double() @ W64.t()
    ref = torch.nn.functional.cross_entropy(logits[keep], tgt.view(-1)[keep])
    (ref * up).backward()
    head = W64.grad.clone()
    p = torch.softmax(logits.detach(), 1)
    p[keep, tgt.view(-1)[keep]] -= 1
    p[~keep] = 0
    dhid = up / float(n) * alpha * p @ W.double()
    de = (dhid.view(B, S, H) * k.double())
    live = ids != 0
    emb = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_put_((ids[live],), de[live] * scale, accumulate=True)
    want = head + emb
    # per element: 16-bit roundings of G in the head's sum and in dh's (h16 of
    # the sums of magnitudes, twice for dh: G and dh itself, once more for
    # dh * k), fp32 sums (2e-5), the head's gradient and the sum rounded
    h16 = torch.finfo(dt).eps / 2
    G = up / float(n) * p.abs()
    mag_head = alpha * G.t() @ h.double().abs()
    mde = alpha * (G @ W.double().abs()).view(B, S, H) * k.double().abs() * scale
    mag_emb = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_put_((ids[live],), mde[live], accumulate=True)
    tol = (h16 + 3e-5) * mag_head + (3 * h16 + 5e-5) * mag_emb * 1.01 + h16 * (head.abs() + want.abs()) * 1.02
    if dt == torch.float16:
        # subnormal results: dh and dh * k (each position's, times scale), the head's rows, the sum
        cnt = torch.zeros(V, 1, dtype=torch.float64, device=DEV).index_put_(
            (ids[live],), torch.ones(int(live.sum()), 1, dtype=torch.float64, device=DEV), accumulate=True)
        tol = tol + 2.0 ** -25 * (2 + cnt * scale * 2.5)
    for got in (Wl.grad, dw):
        err = (got.double() - want).abs()
        say(f"  worst {float((err / tol.clamp_min(1e-300)).max()):.3f} of the bound")
        assert bool((err <= tol).all())
    # a row that neither end touches stays zero in the embedding's part and
    # carries only the head's softmax
    assert bool((dw[0].double() - head[0]).abs().le(tol[0]).all())


def test_vocabulary_shards():
    """Two shards of the matrix: lookups of ids - v0 add up to the whole one;
    each shard's log-sum-exps join to the whole one's, and only the shard that
    holds a target has a loss for it."""
    V, H, v0 = 600, 64, 256
    g = torch.Generator(device=DEV).manual_seed(5)
    W = torch.randn(V, H, generator=g, device=DEV).mul_(0.1).bfloat16()
    ids = torch.randint(0, V, (70,), generator=g, device=DEV)
    parts = [(W[:v0].contiguous(), ids), (W[v0:].contiguous(), ids - v0)]
    assert torch.equal(sum(L.embed(i, w, 2.0) for w, i in parts), L.embed(ids, W, 2.0))
    go = torch.randn(70, H, generator=g, device=DEV).bfloat16()
    both = torch.cat([L.embed_backward(go, i, w.shape[0], 2.0) for w, i in parts])
    assert torch.equal(both, L.embed_backward(go, ids, V, 2.0))
    h = torch.randn(70, H, generator=g, device=DEV).bfloat16()
    loss, lse = L.xent_forward(h, W, ids)
    ls = [L.xent_forward(h, w, i) for w, i in parts]
    joined = torch.logaddexp(ls[0][1].double(), ls[1][1].double())
    # each side within the bound of an fp32 log-sum-exp of these sizes: logits
    # within 2e-5 of sum |h w| <= 2e-5 * 64 * 4 * 0.4, exponentials 1e-5
    assert bool(((joined - lse.double()).abs() <= 2 * (2e-5 * 64 * 4 * 0.4 + 1e-5)).all())
    own = torch.stack([((i >= 0) & (i < w.shape[0])) for w, i in parts])
    assert bool((own.sum(0) == 1).all())
    for k in range(2):
        assert bool((ls[k][0][~own[k]] == 0).all())
