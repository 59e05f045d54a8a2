"""The int8 quantiser and the int8 head, bit for bit: the integer sum is exact
and every later step is one binary32 operation, which numpy repeats."""
import numpy as np
import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def quant_ref(x):
    """From the definition, numpy float32 on the host."""
    xf = x.float().cpu().numpy()
    amax = np.abs(xf).max(axis=1)
    s = (amax / np.float32(127)).astype(np.float32)
    s[s == 0] = 1
    q = np.clip(np.rint((xf / s[:, None]).astype(np.float32)), -127, 127)
    return q.astype(np.int8), s


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R,H", [(1, 32), (5, 64), (33, 2048), (7, 4096), (3, 8192), (2, 8224), (2, 1 << 16), (1000, 96)])
def test_quantiser(R, H, dt):
    say(f"quantize_int8 R={R} H={H} {dt}")
    g = torch.Generator().manual_seed(R + H)
    x = torch.randn(R, H, generator=g)
    x[0] *= 1e-4
    x[R // 2] *= 100
    if R > 2:
        x[1] = 0
        x[2] = torch.arange(H) % 255 - 127   # codes on the grid and ...
        x[2, 1::2] += 0.5                    # ... halves between (as far as 16 bits hold them)
    x = x.to(DT[dt]).to(DEV)
    q, s = L.quantize_int8(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def test_quantiser_smallest_values():
    # bf16 subnormals over 127 underflow to a scale of 0: then 1, and codes 0
    x = torch.zeros(2, 32, dtype=torch.bfloat16, device=DEV)
    x.view(torch.int16)[0, 3] = 1
    x.view(torch.int16)[1, 5] = 0x0080  # the smallest normal value
    q, s = L.quantize_int8(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def logits_ref(hq, hs, wq, ws, alpha, bias):
    acc = (hq.double() @ wq.double().t()).cpu().numpy()  # exact: below 2^53
    f = np.float32
    t = acc.astype(f) * hs.cpu().numpy()[:, None]
    t = t.astype(f) * ws.cpu().numpy()[None, :]
    t = f(alpha) * t.astype(f)
    if bias is not None:
        t = t.astype(f) + bias.cpu().numpy()[None, :]
    return torch.from_numpy(t.astype(f))


def make(seed, M, H, V, bias, lo=-127):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randint(lo, 128, s, generator=g, device=DEV, dtype=torch.int8)
    u = lambda n: torch.rand(n, generator=g, device=DEV) * 1e-2 + 1e-3
    return r(M, H), u(M), r(V, H), u(V), (torch.randn(V, generator=g, device=DEV) if bias else None)


# one row and one column; every row-block count of the streaming kernel; its
# launch shapes (few, more, many column blocks per CU); partial chunks (H % 128)
# and K orders that do not start at 0; both sides of 64 rows; ragged tiles and
# vocabularies of every alignment of a row of logits
SIZES = [(1, 32, 1), (1, 128, 16), (3, 96, 50), (16, 160, 333), (17, 256, 20000), (33, 64, 20001), (48, 288, 17003),
         (64, 512, 33000), (5, 512, 70002), (64, 64, 70004), (65, 32, 9), (65, 160, 777), (128, 128, 1024),
         (129, 320, 260), (300, 96, 1001), (513, 64, 514)]


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,H,V", SIZES)
def test_product(M, H, V, out):
    bias, alpha = V % 2 == 0, 1.0 if M % 2 else 0.3
    say(f"logits_int8 M={M} H={H} V={V} {out} bias={bias}")
    hq, hs, wq, ws, b = make(M + V, M, H, V, bias)
    got = L.logits_int8(hq, hs, wq, ws, alpha, b, DT[out]).cpu()
    want = logits_ref(hq, hs, wq, ws, alpha, b).to(DT[out])
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [2, 70])
def test_largest_sums(M):
    # H = 2^16 of (-128)^2: 2^30, an exact int32
    H, V = 1 << 16, 40
    hq = torch.full((M, H), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((V, H), -128, dtype=torch.int8, device=DEV)
    wq[1] = 127
    one = lambda n: torch.ones(n, device=DEV)
    got = L.logits_int8(hq, one(M), wq, one(V), out_dtype=torch.float32)
    assert bool((got[:, 0] == 2.0 ** 30).all()) and bool((got[:, 1] == -128.0 * 127 * H).all())


@pytest.mark.parametrize("M", [3, 70])
def test_largest_vocabulary(M):
    V, H = 1 << 20, 64
    hq, hs, wq, ws, b = make(3, M, H, V, True)
    say("logits_int8 V = 2^20", M)
    got = L.logits_int8(hq, hs, wq, ws, 1.0, b, torch.bfloat16)
    at = torch.tensor([0, 1, 15, 16, 10239, 10240, 300000, V - 257, V - 2, V - 1], device=DEV)
    want = logits_ref(hq, hs, wq[at], ws[at], 1.0, b[at]).to(torch.bfloat16)
    assert torch.equal(got[:, at].cpu(), want)


def test_rows_do_not_depend_on_the_call():
    hq, hs, wq, ws, b = make(7, 300, 256, 5000, True)
    full = L.logits_int8(hq, hs, wq, ws, 1.0, b, torch.float32)
    for n in (1, 15, 16, 17, 48, 64, 65, 128, 129, 257):
        assert torch.equal(L.logits_int8(hq[:n].contiguous(), hs[:n].contiguous(), wq, ws, 1.0, b, torch.float32),
                           full[:n]), n


@pytest.mark.parametrize("M", [20, 90])
def test_nothing_outside_the_output_is_written(M):
    for V in (333, 336):
        hq, hs, wq, ws, b = make(9, M, 96, V, True)
        for dt in DT.values():
            buf = torch.full((M * V + 64,), 5.0, dtype=dt, device=DEV)
            out = buf[32:-32].view(M, V)
            assert L.logits_int8(hq, hs, wq, ws, 1.0, b, dt, out) is out
            assert bool((buf[:32] == 5).all() and (buf[-32:] == 5).all())
            assert torch.equal(out, L.logits_int8(hq, hs, wq, ws, 1.0, b, dt))


def test_refusals():
    hq, hs, wq, ws, b = make(11, 4, 64, 50, True)
    for bad in (dict(hidden=hq.float()), dict(weight=wq[:, :32].contiguous()), dict(hidden_scale=hs[:3]),
                dict(weight_scale=ws.double()), dict(bias=b[:9]), dict(hidden=hq.t().contiguous().t()),
                dict(out_dtype=torch.int32)):
        kw = dict(hidden=hq, hidden_scale=hs, weight=wq, weight_scale=ws, bias=b)
        kw.update(bad)
        with pytest.raises(ValueError):
            L.logits_int8(**kw)
    with pytest.raises(L.NotHandled):
        L.logits_int8(hq[:, :40].contiguous(), hs, wq[:, :40].contiguous(), ws)
    with pytest.raises(L.NotHandled):
        L.quantize_int8(torch.zeros(4, 64, device=DEV))
    with pytest.raises(ValueError):
        L.quantize_int8(torch.zeros(4, 64, device=DEV).half().t())
    assert L.logits_int8(hq[:0], hs[:0], wq, ws).shape == (0, 50)
    q, s = L.quantize_int8(torch.zeros(0, 64, device=DEV, dtype=torch.bfloat16))
    assert q.shape == (0, 64) and s.shape == (0,)


def test_a_bf16_head_in_8_bits():
    """Quantise the head once and a batch's hidden rows per call, as a server
    does: the logits are off by what the codes' half steps allow, |dx| <= s / 2
    (1 + 2^-22) on either side."""
    M, H, V = 24, 512, 3000
    g = torch.Generator(device=DEV).manual_seed(3)
    h = torch.randn(M, H, generator=g, device=DEV).bfloat16()
    W = (torch.randn(V, H, generator=g, device=DEV) * 0.02).bfloat16()
    wq, ws = L.quantize_int8(W)
    hq, hs = L.quantize_int8(h)
    got = L.logits_int8(hq, hs, wq, ws, out_dtype=torch.float32)
    hd, Wd = h.double(), W.double()
    eh, ew = hs.double()[:, None] / 2 * (1 + 2.0 ** -22), ws.double()[None] / 2 * (1 + 2.0 ** -22)
    bound = eh * Wd.abs().sum(1)[None] + ew * hd.abs().sum(1)[:, None] + H * eh * ew
    bound = bound + 4 * 2.0 ** -24 * (hd.abs() @ Wd.abs().t() + bound)
    assert bool(((got.double() - hd @ Wd.t()).abs() <= bound).all())


def test_captured_and_replayed():
    M, H, V = 20, 128, 3000
    h = torch.randn(M, H, device=DEV).bfloat16()
    _, _, wq, ws, b = make(13, M, H, V, True)
    h2 = torch.randn(100, H, device=DEV).bfloat16()

    def step():
        out = []
        for x in (h, h2):
            q, s = L.quantize_int8(x)
            out += [q, s, L.logits_int8(q, s, wq, ws, 1.0, b)]
        return out
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for k in range(3):
        say("int8 replay", k)
        h.copy_(torch.randn(M, H, device=DEV) * (k + 1))
        h2.copy_(torch.randn(100, H, device=DEV))
        want = step()
        torch.cuda.synchronize()
        for t in got:
            t.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)
