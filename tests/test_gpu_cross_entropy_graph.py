"""cross_entropy and its backward pass captured and replayed: the sums over the
rows' losses are part of the graph."""
import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


# one work-group's sum; rows whose sum a library reduction splits over work-groups
@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("M", [300, 5000, 70000, 1 << 18, 1000003])
def test_captured_and_replayed(M, reduction):
    H, V = 32, 40
    say(f"cross_entropy graph M={M} {reduction}")
    g = torch.Generator(device=DEV).manual_seed(M)

    def inputs(k):
        h = torch.randn(M, H, generator=g, device=DEV).mul_(k + 1).bfloat16()
        y = torch.randint(0, V, (M,), generator=g, device=DEV)
        y[torch.rand(M, generator=g, device=DEV) < 0.1 * k] = -100
        return h, y

    W0 = torch.randn(V, H, generator=g, device=DEV).mul_(0.3).bfloat16()

    def step(h, W, y):
        loss = L.cross_entropy(h, W, y, 0.5, reduction=reduction)
        return (loss.detach(), *torch.autograd.grad(loss, [h, W]))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h, y = inputs(0)
    with torch.cuda.stream(s):
        for _ in range(2):
            step(h.clone().requires_grad_(), W0.clone().requires_grad_(), y)
    torch.cuda.current_stream().wait_stream(s)
    hs, Ws = h.clone().requires_grad_(), W0.clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(hs, Ws, y)
    for k in range(4):
        say("  replay", k)
        h2, y2 = inputs(k)
        hs.data.copy_(h2), y.copy_(y2)
        want = step(h2.requires_grad_(), W0.clone().requires_grad_(), y2)
        torch.cuda.synchronize()
        for t in out:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), (M, k, float((a.double() - b.double()).abs().max()))


@pytest.mark.parametrize("M", [65536, 65537, 70000, 1 << 18, 1000003])
def test_totals(M):
    """The reductions against the rows' losses in 64 bits: sums of 1024 values
    and of at most 2^16 in any order, one division."""
    H, V = 32, 40
    g = torch.Generator(device=DEV).manual_seed(M)
    h = torch.randn(M, H, generator=g, device=DEV).bfloat16()
    W = torch.randn(V, H, generator=g, device=DEV).mul_(0.3).bfloat16()
    y = torch.randint(-1, V + 1, (M,), generator=g, device=DEV)
    rows = L.cross_entropy(h, W, y, reduction="none").double()
    n = int(((y >= 0) & (y < V)).sum())
    for reduction, want in (("sum", rows.sum()), ("mean", rows.sum() / n)):
        got = L.cross_entropy(h, W, y, reduction=reduction)
        assert abs(float(got) - float(want)) <= 2.0 ** -24 * (1024 + (1 << 16)) * float(want)
    # integers, so the count is exact: the mean is the sum over n, rounded once
    total = L.cross_entropy(h, W, y, reduction="sum")
    assert torch.equal(L.cross_entropy(h, W, y), total / torch.tensor(n, device=DEV))
