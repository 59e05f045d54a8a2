"""The embedding lookup and its gradient by sorted tokens.

The lookup is one product rounded once, so it is compared bit for bit. A
gradient row is an fp32 sum of n rows (n u of the sum of magnitudes, u =
2^-24), scaled (u) and rounded to 16 bits (half a step)."""
import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def table(seed, V, H, dt):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(V, H, generator=g, device=DEV).to(DT[dt])


def tokens(seed, M, V, how, index=torch.int64):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if how == "one":
        ids = torch.full((M,), V - 1, device=DEV)
    elif how == "distinct":
        ids = torch.randperm(V, generator=g, device=DEV)[:M]
    elif how == "padded":
        ids = torch.randint(0, V, (M,), generator=g, device=DEV)
        ids[torch.rand(M, generator=g, device=DEV) < 0.6] = V // 2
    elif how == "outside":
        ids = torch.randint(-V, 2 * V, (M,), generator=g, device=DEV)
    else:
        ids = torch.randint(0, V, (M,), generator=g, device=DEV)
    return ids.to(index)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [1.0, 45.254833995939045, 0.1])
@pytest.mark.parametrize("M,V,H,how", [(1, 1, 32, "any"), (3, 50, 64, "outside"), (64, 1000, 4096, "any"),
                                       (129, 7, 96, "outside"), (1000, 333, 288, "any")])
def test_lookup(M, V, H, how, scale, dt):
    say(f"embed M={M} V={V} H={H} {how} scale={scale} {dt}")
    W, ids = table(M, V, H, dt), tokens(M + 1, M, V, how)
    inside = (ids >= 0) & (ids < V)
    rows = W[torch.where(inside, ids, torch.zeros_like(ids))]
    # the product of a 24-bit scale and an 11-bit value is exact in 64 bits;
    # fp32, then 16 bits, as the kernel's contract has it
    want = (rows.double() * torch.tensor(scale, dtype=torch.float32).double()).float().to(W.dtype)
    want[~inside] = 0
    for index in (torch.int64, torch.int32):
        got = L.embed(ids.to(index), W, scale)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)) or torch.equal(got, want)


def test_lookup_shapes_out_and_stream():
    W = table(1, 40, 64, "bf16")
    ids = tokens(2, 12, 40, "any").view(2, 3, 2)
    got = L.embed(ids, W, 2.0)
    assert got.shape == (2, 3, 2, 64) and torch.equal(got, W[ids] * 2)
    out = torch.empty_like(got)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert L.embed(ids, W, 2.0, out, stream=s) is out
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    assert L.embed(torch.tensor(3, device=DEV), W).shape == (64,)
    assert L.embed(ids[:0], W).shape == (0, 3, 2, 64)
    with pytest.raises(ValueError):
        L.embed(ids.transpose(0, 1), W)
    with pytest.raises(ValueError):
        L.embed(ids, W, out=out[:1])
    with pytest.raises(L.NotHandled):
        L.embed(ids, W.float())


def check_grad(go, ids, V, scale, padding=None, base=None):
    inside = (ids >= 0) & (ids < V)
    if padding is not None:
        inside &= ids != padding
    at, x = ids[inside].long(), go.reshape(-1, go.shape[-1])[inside.reshape(-1)].double()
    sc = float(torch.tensor(scale, dtype=torch.float32))
    H = go.shape[-1]
    z = lambda: torch.zeros(V, H, dtype=torch.float64, device=DEV)
    want = z().index_put_((at,), x * sc, accumulate=True)
    mag = z().index_put_((at,), x.abs() * abs(sc), accumulate=True)
    n = torch.zeros(V, dtype=torch.float64, device=DEV).index_put_((at,), torch.ones_like(at).double(), accumulate=True)
    tol = (n[:, None] + 2) * U * mag
    if base is not None:
        want = want + base.double()
        tol = tol + 2 * U * (mag + base.double().abs())
    h16 = torch.finfo(go.dtype).eps / 2
    tol = tol + h16 * (want.abs() + tol) + (2.0 ** -25 if go.dtype == torch.float16 else 0.0)
    got = L.embed_backward(go, ids, V, scale, padding_idx=padding, grad_weight=None if base is None else base.clone())
    err = (got.double() - want).abs()
    say(f"  worst {float((err / tol.clamp_min(1e-300)).max()):.3f} of the bound")
    assert bool((err <= tol).all())
    untouched = n == 0
    assert torch.equal(got[untouched], torch.zeros_like(got[untouched]) if base is None else base[untouched])
    return got


# both sorts (up to and past 16384 positions), one and several passes of the
# second, tiles that end inside an id, an id over many tiles, all positions one
# id, no id twice, ids without a gradient at the end of the order
GRADS = [(1, 1, 32, "any"), (7, 100, 64, "any"), (8, 3, 96, "any"), (9, 1, 32, "one"), (65, 40, 2080, "padded"),
         (1000, 5000, 288, "distinct"), (1000, 300, 64, "outside"), (4100, 4096, 4096, "padded"),
         (8193, 77, 32, "any"), (16384, 500, 64, "padded"), (16385, 500, 64, "padded"), (16385, 1 << 20, 32, "any"),
         (20000, 300, 32, "outside"), (40001, 513, 160, "padded"), (300000, 9, 32, "one"), (270001, 70000, 32, "any")]


@pytest.mark.parametrize("M,V,H,how", GRADS)
def test_gradient(M, V, H, how):
    dt = "f16" if M % 2 else "bf16"
    say(f"embed grad M={M} V={V} H={H} {how} {dt}")
    go = table(M + 3, M, H, dt) * (0.01 if dt == "f16" else 1.0)
    ids = tokens(M + 4, M, V, how, torch.int32 if V % 2 else torch.int64)
    got = check_grad(go, ids, V, 1.5)
    for _ in range(2):  # the same bits every run
        assert torch.equal(got, L.embed_backward(go, ids, V, 1.5))


@pytest.mark.parametrize("M", [300, 17000])
def test_gradient_added_and_padding(M):
    V, H = 120, 64
    go, ids, base = table(1, M, H, "bf16"), tokens(2, M, V, "outside"), table(3, V, H, "bf16")
    ids[::2] = 5
    say("embed grad added", M)
    check_grad(go, ids, V, 0.5, base=base)
    check_grad(go, ids, V, 0.5, padding=5, base=base)
    got = check_grad(go, ids, V, 0.5, padding=5)
    assert bool((got[5] == 0).all())
    # counted from the end, as torch has it
    assert torch.equal(L.embed_backward(go, ids, V, 0.5, padding_idx=5 - V), got)
    for bad in (V, -V - 1):
        with pytest.raises(ValueError):
            L.embed_backward(go, ids, V, padding_idx=bad)
    # every position without a gradient
    ids.fill_(5)
    assert bool((L.embed_backward(go, ids, V, padding_idx=5) == 0).all())
    assert torch.equal(L.embed_backward(go, ids, V, padding_idx=5, grad_weight=base.clone()), base)


def test_order_of_summation():
    """One id's rows are summed in ascending position within a tile: the fp32
    sum of 1, 2^25, -2^25 is 0 in that order and 1 in others."""
    H = 32
    go = torch.zeros(3, H, dtype=torch.bfloat16, device=DEV)
    go[0], go[1], go[2] = 1.0, 2.0 ** 25, -2.0 ** 25
    ids = torch.zeros(3, dtype=torch.int64, device=DEV)
    assert bool((L.embed_backward(go, ids, 2)[0] == 0).all())
    go[0], go[1], go[2] = 2.0 ** 25, -2.0 ** 25, 1.0
    assert bool((L.embed_backward(go, ids, 2)[0] == 1).all())


def test_no_positions_and_refusals():
    go, ids = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV)
    assert bool((L.embed_backward(go, ids, 1000) == 0).all())
    base = table(1, 10, 64, "bf16")
    assert torch.equal(L.embed_backward(go, ids, 10, grad_weight=base.clone()), base)
    go, ids = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        L.embed_backward(go, ids[:3], 10)
    with pytest.raises(ValueError):
        L.embed_backward(go, ids, 10, grad_weight=base.half())
    with pytest.raises(ValueError):
        L.embed_backward(go.t().contiguous().t(), ids, 10)
    with pytest.raises(L.NotHandled):
        L.embed_backward(go.float(), ids, 10)
    with pytest.raises(L.NotHandled):
        L.embed_backward(go[:, :48].contiguous(), ids, 10)
    with pytest.raises(L.LmHeadError):
        L.embed_backward(go, ids, 10, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("M", [500, 20000])
def test_nothing_outside_the_outputs_is_written(M):
    V, H, pad = 77, 96, 256
    need = L.embed_backward_workspace_bytes(M, H)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    from lm_head_logits_amd import _lib
    buf = torch.full((V * H + 2 * pad,), 5.0, dtype=torch.bfloat16, device=DEV)
    go, ids = table(1, M, H, "bf16"), tokens(2, M, V, "padded")
    st = _lib.load().lmhead_embed_backward(ids.data_ptr(), 1, M, go.data_ptr(), V, H, _lib.LMHEAD_BF16, 1.0, -1, 0,
                                           buf.data_ptr() + 2 * pad, ws.data_ptr(), need,
                                           torch.cuda.current_stream().cuda_stream)
    assert st == _lib.OK
    torch.cuda.synchronize()
    assert bool((ws[need:] == 77).all()) and bool((buf[:pad] == 5).all()) and bool((buf[-pad:] == 5).all())
    assert torch.equal(buf[pad:-pad].view(V, H), L.embed_backward(go, ids, V))


@pytest.mark.parametrize("M", [700, 18000])
def test_captured_and_replayed(M):
    V, H = 2000, 64
    go, ids = table(1, M, H, "bf16"), tokens(2, M, V, "padded")
    W = table(3, V, H, "bf16")
    L.embed_backward(go, ids, V)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, gw = L.embed(ids, W, 3.0), L.embed_backward(go, ids, V, 3.0)
    for k in range(3):
        say("embed replay", M, k)
        ids.copy_(tokens(10 + k, M, V, "outside"))
        go.copy_(table(20 + k, M, H, "bf16"))
        want = L.embed(ids, W, 3.0), L.embed_backward(go, ids, V, 3.0)
        torch.cuda.synchronize()
        out.fill_(1), gw.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(gw, want[1])


def test_differentiable():
    W = table(1, 100, 64, "bf16").requires_grad_(True)
    ids = tokens(2, 60, 100, "padded").view(6, 10)
    out = L.embedding(ids, W, 8.0, padding_idx=50)
    assert torch.equal(out, L.embed(ids, W.detach(), 8.0))
    out.sum().backward()  # an expanded gradient, stride 0
    want = L.embed_backward(torch.ones(6, 10, 64, dtype=torch.bfloat16, device=DEV), ids, 100, 8.0, padding_idx=50)
    assert torch.equal(W.grad, want) and bool((W.grad[50] == 0).all())
