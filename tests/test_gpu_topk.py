"""logits_topk: values and ids exactly, in the order (logit descending, column
ascending); the log-sum-exp against 64 bits.

Bound of lse: each exponential's argument (x - largest) log2(e) / T is off by 3
roundings of itself (only arguments above -126 ln 2 give anything: 3 * 88 u of the
sum), exp2 by 2 u, the sums of up to V values in chains of at most V / (256 * 4)
+ 64 additions and folds by that many u, the log and the last sum by 2 u of their
results: u (300 + V / 1024 + 64) + 4 u |lse|."""
import math

import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def want(x, k):
    """By whole-number keys: a logit's place in the order of its type, then the column."""
    f = x.float() + 0.0
    bits = f.view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits, bits)
    order = torch.where(f.isnan(), torch.full_like(order, 2 ** 31), order)
    col = torch.arange(x.shape[1], device=x.device)
    key = order * 2 ** 20 + (2 ** 20 - 1 - col)
    ids = torch.sort(key, dim=1, descending=True).indices[:, :k]
    return x.gather(1, ids), ids.int()


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def check(x, k, T=1.0):
    values, ids, lse = L.logits_topk(x, k, T)
    v, i = want(x, k)
    assert values.dtype == x.dtype and ids.dtype == torch.int32 and lse.dtype == torch.float32
    assert torch.equal(ids, i), (x.shape, k, int((ids != i).sum()))
    assert torch.equal(bits(values), bits(v))
    e = torch.logsumexp(x.double() / T, 1)
    e = torch.where(e.float().isinf(), e.float().double(), e)  # past fp32's largest number: infinite
    odd = ((x == math.inf) | x.isnan()).any(1)
    assert bool(lse[odd].isnan().all())
    e, l = e[~odd], lse[~odd].double()
    tol = U * (364 + x.shape[1] / 1024) + 4 * U * e.abs()
    assert bool(((l == e) | ((l - e).abs() <= tol)).all()), float((l - e).abs().max())
    return values, ids, lse


def logits(seed, M, V, dt, scale=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(M, V, generator=g, device=DEV).mul_(scale).to(DT[dt])


# one column; less than a piece, than a work-group's tile, than its first
# stretch; ends inside each; one segment and several; many rows
SIZES = [(1, 1, 1), (3, 5, 5), (1, 7, 3), (2, 130, 64), (1, 1000, 20), (5, 2049, 65), (700, 1023, 17), (1, 151936, 20),
         (48, 128256, 50), (600, 50257, 8), (7, 32000, 256), (2, 1 << 20, 100), (1030, 4096, 1), (1, 8193, 1024)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,V,k", SIZES)
def test_exactly(M, V, k, dt):
    say(f"topk M={M} V={V} k={k} {dt}")
    check(logits(M + V + k, M, V, dt), k, 0.7 if M % 2 else 1.0)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 255, 256, 257, 1023, 1024])
def test_every_count(k, dt):
    for M, V in ((3, 1024), (2, 30011), (530, 5003)):
        say(f"topk k={k} {dt} M={M} V={V}")
        check(logits(k, M, V, dt), k)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M", [1, 515])
def test_rows_in_order_and_ties(M, dt):
    """Ascending rows (every logit passes the bound so far), descending ones,
    constant ones, two values, zeros of both signs."""
    V = 20011
    up = torch.linspace(-300, 300, V, device=DEV)
    for name, row in (("up", up), ("down", up.flip(0)), ("same", torch.full((V,), 1.5, device=DEV)),
                      ("two", (torch.arange(V, device=DEV) % 997 == 5).float()),
                      ("zeros", torch.where(torch.arange(V, device=DEV) % 3 == 0, -0.0, 0.0)),
                      ("peak", torch.where(torch.arange(V, device=DEV) == V - 1, 9.0, -9.0))):
        for k in (1, 64, 300, 1024):
            say(f"topk {name} M={M} {dt} k={k}")
            check(row.to(DT[dt]).repeat(M, 1), k)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M", [2, 513])
def test_infinities_and_nan(M, dt):
    V = 9001
    low = torch.finfo(DT[dt]).min
    for k in (1, 40, 200):
        x = logits(3, M, V, dt)
        x[0, 10:] = -math.inf  # fewer than k numbers
        x[-1] = -math.inf
        say(f"topk -inf {dt} k={k}")
        check(x, k)
        x[0, 20:3000] = low
        check(x, k)
        x[-1].fill_(low)
        check(x, k, 0.5)
        x = logits(4, M, V, dt)
        x[0, 77], x[0, 5000], x[-1, 8999] = math.inf, math.nan, math.nan
        say(f"topk nan {dt} k={k}")
        check(x, k)
        x[0] = math.nan
        check(x, k)
    neg = torch.tensor([-1 if dt == "f32" else -1], dtype=torch.int32 if dt == "f32" else torch.int16, device=DEV)
    x = logits(5, M, V, dt)
    x[:, 3:4] = neg.view(DT[dt])  # a NaN with its sign bit set
    check(x, 5)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M", [3, 700])
def test_strides_and_alignment(M, dt):
    """Rows of a padded head, any start within 16 bytes; the padding is not looked at."""
    for V, pad, off in ((1000, 24, 0), (1000, 1, 0), (5003, 7, 3), (999, 3, 1), (8190, 2, 5), (17, 3, 2)):
        say(f"topk stride {dt} V={V} pad={pad} off={off}")
        buf = torch.full((M * (V + pad) + off + 8,), 1e4, device=DEV).to(DT[dt])
        x = buf[off:off + M * (V + pad)].view(M, V + pad)[:, :V]
        x.copy_(logits(V, M, V, dt))
        check(x, min(V, 33))
    # the first and the last row at the ends of an allocation
    x = logits(9, M, 1025, dt)
    check(x, 10)


def test_nothing_outside_the_outputs_is_written():
    from lm_head_logits_amd import _lib
    M, V, K, pad = 5, 40000, 37, 32
    x = logits(1, M, V, "bf16")
    v, i = want(x, K)
    need = L.logits_topk_workspace_bytes(M, V, K)
    assert need > 0 and L.logits_topk_workspace_bytes(4096, V, K) == 0
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device=DEV)
    values = torch.full((M * K + 2 * pad,), 5.0, dtype=x.dtype, device=DEV)
    ids = torch.full((M * K + 2 * pad,), 5, dtype=torch.int32, device=DEV)
    lse = torch.full((M + 2 * pad,), 5.0, device=DEV)
    st = _lib.load().lmhead_logits_topk(x.data_ptr(), M, V, V, _lib.LMHEAD_BF16, K, 1.0, values.data_ptr() + 2 * pad,
                                        ids.data_ptr() + 4 * pad, lse.data_ptr() + 4 * pad, ws.data_ptr(), need,
                                        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert bool((ws[need:] == 77).all())
    for t in (values, ids, lse):
        assert bool((t[:pad] == 5).all() and (t[-pad:] == 5).all())
    assert torch.equal(ids[pad:-pad].view(M, K), i) and torch.equal(values[pad:-pad].view(M, K), v)


def test_runs_repeat_and_replay():
    for M in (2, 600):
        x = logits(11, M, 50257, "bf16")
        # the second: every logit passes the bound so far, so the keys of no tile fit
        for y in (x, torch.sort(x.float(), 1).values.bfloat16(), torch.sort(logits(12, M, 50257, "f32"), 1).values):
            first = L.logits_topk(y, 40)
            for _ in range(5):
                for a, b in zip(first, L.logits_topk(y, 40)):
                    assert torch.equal(a, b)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.logits_topk(x, 40)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = L.logits_topk(x, 40)
        for k in range(3):
            say("topk replay", M, k)
            x.copy_(logits(20 + k, M, 50257, "bf16"))
            w = L.logits_topk(x, 40)
            torch.cuda.synchronize()
            for t in out:
                t.fill_(3)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, w):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    xs = [logits(30 + k, 3, 100003, "f32") for k in range(2)]
    ws = [L.logits_topk(x, 50) for x in xs]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            got[k] = L.logits_topk(xs[k], 50, stream=streams[k])
    torch.cuda.synchronize()
    for a, b in zip(got, ws):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    x = logits(1, 4, 100, "f32")
    for bad in (lambda: L.logits_topk(x, 0), lambda: L.logits_topk(x, 101), lambda: L.logits_topk(x[0], 3),
                lambda: L.logits_topk(x.double(), 3), lambda: L.logits_topk(x.t(), 3), lambda: L.logits_topk(x.cpu(), 3),
                lambda: L.logits_topk(x[:1].expand(4, 100), 3)):
        with pytest.raises(ValueError):
            bad()
    big = logits(1, 2, 5000, "f32")
    for bad in (lambda: L.logits_topk(big, 1025), lambda: L.logits_topk(x, 3, 0.0), lambda: L.logits_topk(x, 3, -1.0),
                lambda: L.logits_topk(x, 3, math.nan), lambda: L.logits_topk(x, 3, math.inf),
                lambda: L.logits_topk(logits(1, 1, 100000, "f32"), 9, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(L.LmHeadError):
            bad()
    v, i, l = L.logits_topk(x[:0], 3)
    assert v.shape == i.shape == (0, 3) and l.shape == (0,)


def test_a_teacher_and_its_student():
    """The operators together: a teacher's head, its top logits, a student's step towards them."""
    M, H, V, K, T = 300, 64, 5000, 32, 1.5
    g = torch.Generator(device=DEV).manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    Wt, ht = n(V, H).mul_(0.2).bfloat16(), n(M, H).bfloat16()
    Ws, hs = n(V, H).mul_(0.2).bfloat16().requires_grad_(), n(M, H).bfloat16().requires_grad_()
    top, ids, lse = L.logits_topk(L.logits(ht, Wt, out_dtype=torch.bfloat16), K, T)
    ids[::4] = -100  # prompts
    for whole in (None, lse):
        loss = L.distillation(hs, Ws, ids, top, temperature=T, teacher_lse=whole)
        gh, gw = torch.autograd.grad(loss * T * T, [hs, Ws])
        l2, saved = L.distill_forward(hs.detach(), Ws.detach(), ids, top, temperature=T, teacher_lse=whole)
        kept = (ids[:, 0] >= 0).sum()
        assert float(loss) == float(l2.sum() / kept)
        want = L.loss_backward((torch.ones(M, device=DEV) * (T * T)) / kept, Ws.detach(), saved)
        assert torch.equal(gh, want[0]) and torch.equal(gw, want[1]) and bool((gh[::4] == 0).all())
