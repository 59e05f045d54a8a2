"""Softmax cross entropy of the head and its gradients against the formula in
64 bits.

Bounds, elementwise. u = 2^-24; h16 = half a step of the inputs' type (2^-8
bf16, 2^-11 fp16, relative).
  T[m]    how far a logit may be off: the projection's bound, 2e-5 alpha A with
          A = sum |h w| (its fp32 accumulation), and two roundings of the epilogue
  E[m]    relative error of a sum of exponentials: each exponential's argument
          is off by T and by a rounding of itself (|x| u, twice: the difference
          and its product with log2 e), each fold adds a few u
  lse     T + E + 2 u |lse|           (log's derivative is 1 / sum; log itself)
  loss    that, T once more and a rounding
  G       |G| h16 for its rounding to 16 bits; a p (T + E + |x| u + T_lse) for p's
          error; fp16 G is scaled to 2^14 / largest, so below 2^-14 its step is
          2^-24: 2^-25 / 2^14 of the largest coefficient. fp32's smallest normal
          number is 2^-126, and an exponential or a product below it may come out
          as 0: p is off by up to 2^-126, G, kept scaled so that the largest
          coefficient c is 1 or more, by c 2^-126 more, and each of the products
          of the sums for grad_hidden and grad_W by c alpha 2^-126 in the result
  grads   the products' terms carry G's error; their fp32 sums 2e-5 of the sum of
          magnitudes, as the projection's; the result is rounded to 16 bits
"""
import math

import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
TINY16 = {"bf16": 2.0 ** -126, "f16": 2.0 ** -25}  # results below the normal range: 0, or half a step


def make(seed, M, H, V, dt, bias, std=1.0, target="random", index=torch.int64):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(M, H, generator=g).mul_(std).to(DT[dt]).to(DEV)
    W = torch.randn(V, H, generator=g).mul_(0.05).to(DT[dt]).to(DEV)
    b = torch.randn(V, generator=g).mul_(0.3).to(DEV) if bias else None
    y = torch.randint(0, V, (M,), generator=g)
    if target == "ignored":
        y[::3] = -100
    y = y.to(index).to(DEV)
    gl = (torch.rand(M, generator=g) + 0.5).div_(max(M, 1)).to(DEV)
    gz = torch.randn(M, generator=g).div_(max(M, 1)).to(DEV)
    return h, W, b, y, gl, gz


def reference(h, W, b, y, gl, gz, alpha, ignore=-100):
    """Everything in float64, from the formula; with the pieces the bounds need."""
    hd, Wd, V = h.double(), W.double(), W.shape[0]
    t = hd @ Wd.t() * alpha
    A = hd.abs() @ Wd.abs().t() * abs(alpha)
    if b is not None:
        t = t + b.double()
    finite = torch.where(t.isinf(), torch.zeros_like(t), t)
    T = (2e-5 * A + 2 * U * finite.abs()).amax(1)
    mx = t.amax(1)
    mz = torch.where(mx.isinf(), torch.zeros_like(mx), mx)
    s = torch.exp(t - mz[:, None]).sum(1)
    lse = torch.log(s) + mz
    keep = (y != ignore) & (y >= 0) & (y < V)
    at = torch.where(keep, y.long(), torch.zeros_like(y.long()))[:, None]
    ty = t.gather(1, at)[:, 0]
    loss = torch.where(keep, torch.where(ty.isinf(), torch.full_like(ty, math.inf), lse - ty), torch.zeros_like(ty))
    x = torch.where(t.isinf(), torch.zeros_like(t), (t - mz[:, None])).abs()
    tiles = (V + 255) // 256
    E = 2 * U * x.amax(1) + (22 + 3 * (tiles // 16 + 18)) * U + T
    out = dict(t=t, T=T, E=E, lse=lse, loss=loss, keep=keep)
    if gl is None:
        return out
    p = torch.where(lse[:, None].isinf(), torch.zeros_like(t), torch.exp(t - torch.where(lse.isinf(), 0 * lse, lse)[:, None]))
    gk = torch.where(keep, gl.double(), torch.zeros_like(lse))
    a = gk + (gz.double() if gz is not None else 0.0)
    G = p * a[:, None]
    G.scatter_add_(1, at, -gk[:, None])
    h16 = torch.finfo(h.dtype).eps / 2
    perr = (2 * T + 2 * E + 4 * U * lse.abs().nan_to_num(0, 0, 0))[:, None] + 4 * U * (1 + x + finite.abs())
    c = float(torch.maximum(a.abs(), gk.abs()).amax())
    dG32 = a.abs()[:, None] * p * perr + 2 * U * G.abs() + 2 * c * 2.0 ** -126
    dG = dG32 + h16 * (G.abs() + dG32)
    if h.dtype == torch.float16:
        dG = dG + c * 2.0 ** -38
    Gm = G.abs() + dG
    dh, dw = alpha * (G @ Wd), alpha * (G.t() @ hd)
    al = abs(alpha)
    out.update(dh=dh, dw=dw, db=G.sum(0),
               dh_tol=al * (dG @ Wd.abs() + 2e-5 * (Gm @ Wd.abs()) + c * V * 2.0 ** -126),
               dw_tol=al * (dG.t() @ hd.abs() + 2e-5 * (Gm.t() @ hd.abs()) + c * len(y) * 2.0 ** -126),
               db_tol=dG32.sum(0) + (len(y) + 8) * U * Gm.sum(0), h16=h16)
    return out


def close(name, got, want, tol):
    err = (got.double() - want).abs()
    same = got.double() == want  # infinities
    ok = same | (err <= tol)
    worst = float(torch.where(same, torch.zeros_like(err), err / tol.clamp_min(1e-300)).max()) if err.numel() else 0.0
    say(f"  {name}: worst {worst:.3f} of the bound")
    assert bool(ok.all()), (name, worst, int((~ok).sum()))


def check(h, W, b, y, gl, gz, alpha, ignore=-100):
    r = reference(h, W, b, y, gl, gz, alpha, ignore)
    loss, lse = L.xent_forward(h, W, y, alpha, b, ignore_index=ignore)
    tl = r["T"] + r["E"] + 2 * U * r["lse"].abs().nan_to_num(0, 0, 0)
    close("lse", lse, r["lse"], tl)
    close("loss", loss, r["loss"], tl + r["T"] + 2 * U * r["loss"].abs().nan_to_num(0, 0, 0))
    assert bool((loss[~r["keep"]] == 0).all())
    if gl is None:
        return loss, lse
    dh, dw, db = L.xent_backward(gl, h, W, y, lse, alpha, b, grad_lse=gz, ignore_index=ignore)
    tiny = TINY16["f16" if h.dtype == torch.float16 else "bf16"]
    for name, got in (("dh", dh), ("dw", dw)):
        assert got.dtype == h.dtype
        t = r[name + "_tol"]
        close(name, got, r[name], t + r["h16"] * (r[name].abs() + t) * (1 + 4 * U) + 4 * U * r[name].abs() + tiny)
    if b is not None:
        close("db", db, r["db"], r["db_tol"])
    else:
        assert db is None
    return loss, lse, dh, dw, db


# one row and one column; ends inside a 16-row block, a 128-row half, a tile;
# H of one K-step, a partial stage, several stages with a partial one, odd and
# even stage counts; columns past a tile, past a K-order group
SIZES = [(1, 32, 1), (1, 64, 300), (2, 96, 17), (16, 128, 256), (37, 256, 1000), (64, 160, 257), (128, 320, 511),
         (129, 64, 2049), (255, 192, 129), (257, 512, 700), (300, 288, 333), (513, 224, 1025), (31, 512, 20500)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,H,V", SIZES)
def test_against_the_formula(M, H, V, dt):
    bias, target = (M + V) % 2 == 0, "ignored" if M % 2 else "random"
    say(f"xent M={M} H={H} V={V} {dt} bias={bias} {target}")
    h, W, b, y, gl, gz = make(M * 7 + V, M, H, V, dt, bias, target=target)
    check(h, W, b, y, gl, gz if M % 3 else None, 0.5)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_more_than_one_piece(dt, monkeypatch):
    # 16385 rows of 8192 columns a piece: V = 8450 is two pieces, the second ragged
    M, H, V = 16385, 32, 8450
    say(f"xent pieces M={M} H={H} V={V} {dt}")
    h, W, b, y, gl, gz = make(5, M, H, V, dt, True, target="ignored")
    check(h, W, b, y, gl, gz, 1.0)


def test_scale_found_by_a_launch_of_its_own():
    M, H, V = 32769 + 200, 32, 40
    say(f"xent many rows M={M}")
    h, W, b, y, gl, gz = make(6, M, H, V, "f16", True)
    check(h, W, b, y, gl, None, 1.0)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_targets_left_out(index):
    M, H, V = 40, 64, 90
    h, W, b, y, gl, gz = make(9, M, H, V, "bf16", False, index=index)
    y[0], y[1], y[2], y[3], y[4] = -100, -1, V, 2 ** 31 - 1, 7
    say("xent left-out targets", index)
    loss, lse, dh, dw, db = check(h, W, b, y, gl, None, 1.0, ignore=7)
    # -100 is no column either way; a row left out passes nothing on
    for m in (0, 1, 2, 3, 4):
        assert float(loss[m]) == 0.0 and bool((dh[m] == 0).all())
    if index == torch.int64:
        y[5] = 2 ** 40 + 3  # not its low 32 bits
        check(h, W, b, y, gl, None, 1.0, ignore=7)
    y.fill_(7)
    loss, lse, dh, dw, db = check(h, W, b, y, gl, None, 1.0, ignore=7)
    assert bool((loss == 0).all()) and bool((dh == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("V", [200, 600])
def test_masked_columns(V):
    """-inf biases: columns of probability 0, whole tiles of them, a target there, every column."""
    M, H = 30, 64
    h, W, b, y, gl, gz = make(11, M, H, V, "bf16", True)
    b[::3] = -math.inf
    if V > 300:
        b[:256] = -math.inf
    y[0], y[1] = 0, V - 1
    b[V - 1] = 0.25
    say("xent masked", V)
    loss, *_ = check(h, W, b, y, gl, None, 1.0)
    assert float(loss[0]) == math.inf
    b.fill_(torch.finfo(torch.float32).min)  # the type's lowest value is a number
    b[3] = 1.0
    y.fill_(3)
    check(h, W, b, y, gl, None, 1.0)
    b.fill_(-math.inf)
    y[2] = -100
    loss, lse = L.xent_forward(h, W, y, 1.0, b)
    assert bool((lse == -math.inf).all()) and float(loss[2]) == 0.0 and bool((loss[3:] == math.inf).all())
    dh, dw, db = L.xent_backward(gl, h, W, y, lse, 1.0, b)
    assert not bool(dh.isnan().any() | dw.isnan().any() | db.isnan().any())
    want = torch.zeros(V, device=DEV).index_add_(0, y[y >= 0].long(), -gl[y >= 0])
    assert torch.allclose(db, want, rtol=1e-5, atol=0)  # at most 30 terms: 30 u


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_peaked_rows_and_large_logits(dt):
    """A row of near certainty, ties, and logits of thousands (no overflow)."""
    M, H, V = 20, 32, 300
    h, W, b, y, gl, gz = make(13, M, H, V, dt, False, std=40.0)
    W[5] = W[9]  # exact ties
    h[3] = 0     # constant row: lse = log V
    say("xent peaked", dt)
    loss, lse, *_ = check(h, W, b, y, gl, gz, 8.0)
    assert bool((loss >= 0).all())
    assert abs(float(lse[3]) - math.log(V)) <= 40 * U * math.log(V) + 40 * U


def test_gradient_scale_range():
    """Upstream gradients far from 1, rows of very different size, all zero."""
    M, H, V = 33, 64, 150
    for dt, k in (("bf16", 1e-12), ("bf16", 1e8), ("f16", 1e-3), ("f16", 30.0)):
        h, W, b, y, gl, gz = make(17, M, H, V, dt, True)
        gl = gl * k
        gl[4:9] *= 1e-3
        say("xent gradient scale", dt, k)
        check(h, W, b, y, gl, None, 1.0)
    h, W, b, y, gl, gz = make(17, M, H, V, "f16", True)
    _, lse = L.xent_forward(h, W, y, 1.0, b)
    for out in L.xent_backward(torch.zeros_like(gl), h, W, y, lse, 1.0, b):
        assert bool((out == 0).all())


def test_gradients_against_differences():
    """Central differences of the library's own loss along a direction in each
    input. L is the sum of the rows' losses (fp32, summed at 64 bits); along a
    direction that moves logit v of row m by z[m, v], the difference quotient
    with step e is off by e^2 / 6 max |L'''| <= e^2 / 6 sum_m (2 max_v |z|)^3
    (a third cumulant is at most the cube of the range) and by the losses'
    rounding, M 8 u (|lse| + |t|) / e."""
    M, H, V, alpha = 8, 32, 70, 1.0
    h, W, b, y, gl, gz = make(19, M, H, V, "f16", True)
    h = (h * 4).round().div(4).to(torch.float16)
    W = (W * 64).round().div(64).to(torch.float16)  # sums of two grid values stay exact
    gl = torch.ones(M, device=DEV)
    _, lse = L.xent_forward(h, W, y, alpha, b)
    dh, dw, db = L.xent_backward(gl, h, W, y, lse, alpha, b)
    rng = torch.Generator().manual_seed(3)
    for name, grad in (("h", dh), ("W", dw), ("b", db)):
        for _ in range(4):
            d = torch.randint(-1, 2, grad.shape, generator=rng).to(DEV)
            e = {"h": 0.25, "W": 2.0 ** -6, "b": 0.125}[name]
            z = {"h": lambda: alpha * d.double() @ W.double().t(), "W": lambda: alpha * h.double() @ d.double().t(),
                 "b": lambda: d.double()[None].expand(M, V)}[name]()
            vals = []
            for sgn in (1, -1):
                hh, WW, bb = h, W, b
                step = (sgn * e * d)
                if name == "h": hh = (h.float() + step).to(torch.float16)
                if name == "W": WW = (W.float() + step).to(torch.float16)
                if name == "b": bb = b + step
                vals.append(L.xent_forward(hh, WW, y, alpha, bb)[0].double().sum())
            num = float(vals[0] - vals[1]) / (2 * e)
            ana = float((grad.double() * d.double()).sum())
            tol = e * e / 6 * float(((2 * z.abs().amax(1)) ** 3).sum()) + M * 8 * U * (float(lse.abs().max()) + 10) / e
            # the gradient's own 16-bit roundings, of G and of the result
            tol += 2 * 2.0 ** -11 * float((grad.double().abs() * d.double().abs()).sum())
            tol += 2.0 ** -11 * 2 * float(z.abs().amax(1).sum())
            say(f"  differences {name}: {num:.6f} against {ana:.6f}, bound {tol:.2e}")
            assert abs(num - ana) <= tol


def test_rows_do_not_depend_on_the_call_and_runs_repeat():
    M, H, V = 300, 256, 5000
    h, W, b, y, gl, gz = make(23, M, H, V, "bf16", True)
    loss, lse = L.xent_forward(h, W, y, 1.0, b)
    for n in (1, 16, 37, 129, 256):
        l2, s2 = L.xent_forward(h[:n].contiguous(), W, y[:n].contiguous(), 1.0, b)
        assert torch.equal(l2, loss[:n]) and torch.equal(s2, lse[:n]), n
    a = L.xent_backward(gl, h, W, y, lse, 1.0, b)
    for _ in range(2):
        for p, q in zip(a, L.xent_backward(gl, h, W, y, lse, 1.0, b)):
            assert torch.equal(p, q)
    # parts asked for alone are the same bits
    assert torch.equal(L.xent_backward(gl, h, W, y, lse, 1.0, b, need_weight=False, need_bias=False)[0], a[0])
    only = L.xent_backward(gl, h, W, y, lse, 1.0, b, need_hidden=False, need_bias=False)
    assert only[0] is None and only[2] is None and torch.equal(only[1], a[1])
    assert torch.equal(L.xent_backward(gl, h, W, y, lse, 1.0, b, need_hidden=False, need_weight=False)[2], a[2])


def test_nothing_outside_the_outputs_is_written():
    M, H, V, pad = 45, 96, 333, 64
    h, W, b, y, gl, gz = make(29, M, H, V, "bf16", True)
    from lm_head_logits_amd import _lib
    lib, s = _lib.load(), torch.cuda.current_stream().cuda_stream
    nf, nb = L.xent_forward_workspace_bytes(M, V), L.xent_backward_workspace_bytes(M, H, V, True)
    buf = {k: torch.full((n + 2 * pad,), 123.0, dtype=d, device=DEV) for k, n, d in
           (("loss", M, torch.float32), ("lse", M, torch.float32), ("dh", M * H, torch.bfloat16),
            ("dw", V * H, torch.bfloat16), ("db", V, torch.float32))}
    ws = torch.full((max(nf, nb) + 512,), 77, dtype=torch.uint8, device=DEV)
    at = {k: v.data_ptr() + pad * v.element_size() for k, v in buf.items()}
    st = lib.lmhead_xent_forward(h.data_ptr(), M, H, W.data_ptr(), V, 1.0, b.data_ptr(), _lib.LMHEAD_BF16,
                                 y.data_ptr(), 1, -100, at["loss"], at["lse"], ws.data_ptr(), nf, s)
    assert st == _lib.OK
    torch.cuda.synchronize()
    assert bool((ws[nf:] == 77).all())
    st = lib.lmhead_xent_backward(h.data_ptr(), M, H, W.data_ptr(), V, 1.0, b.data_ptr(), _lib.LMHEAD_BF16,
                                  y.data_ptr(), 1, -100, at["lse"], gl.data_ptr(), None, at["dh"], at["dw"], at["db"],
                                  ws.data_ptr(), nb, s)
    assert st == _lib.OK
    torch.cuda.synchronize()
    assert bool((ws[nb:][:512] == 77).all())
    for k, v in buf.items():
        assert bool((v[:pad] == 123).all() and (v[-pad:] == 123).all()), k
        assert not bool((v[pad:-pad] == 123).all()), k


def test_no_rows():
    W = torch.ones(50, 64, dtype=torch.bfloat16, device=DEV)
    h = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    y, f, b = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV), torch.ones(50, device=DEV)
    loss, lse = L.xent_forward(h, W, y)
    assert loss.shape == lse.shape == (0,)
    dh, dw, db = L.xent_backward(f, h, W, y, f, 1.0, b)
    assert dh.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_other_types_are_not_handled():
    h, W = torch.zeros(4, 64, device=DEV), torch.zeros(9, 64, device=DEV)
    y = torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(L.NotHandled):
        L.xent_forward(h, W, y)
    with pytest.raises(L.NotHandled):
        L.xent_forward(h.half(), W.bfloat16(), y)
    with pytest.raises(L.NotHandled):
        L.xent_forward(h[:, :40].contiguous().half(), W[:, :40].contiguous().half(), y)
    with pytest.raises(ValueError):
        L.xent_forward(h.half().t().contiguous().t(), W.half(), y)
    with pytest.raises(ValueError):
        L.xent_forward(h.half(), W.half(), y[:3])
    with pytest.raises(ValueError):
        L.xent_forward(h.half(), W.half(), y.float())
    with pytest.raises(ValueError):
        L.xent_backward(torch.zeros(4, device=DEV), h.half(), W.half(), y, torch.zeros(4, device=DEV), need_bias=True)
    with pytest.raises(L.LmHeadError):
        L.xent_forward(h.half(), W.half(), y, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_captured_and_replayed():
    M, H, V = 70, 128, 3000
    h, W, b, y, gl, gz = make(31, M, H, V, "bf16", True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            loss, lse = L.xent_forward(h, W, y, 1.0, b)
            L.xent_backward(gl, h, W, y, lse, 1.0, b)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, lse = L.xent_forward(h, W, y, 1.0, b)
        dh, dw, db = L.xent_backward(gl, h, W, y, lse, 1.0, b)
    for k in range(3):
        say("xent replay", k)
        h.copy_(torch.randn(M, H, device=DEV) * (k + 1))
        y.copy_(torch.randint(0, V, (M,), device=DEV))
        l2, s2 = L.xent_forward(h, W, y, 1.0, b)
        want = (l2, s2, *L.xent_backward(gl, h, W, y, s2, 1.0, b))
        torch.cuda.synchronize()
        for t in (loss, lse, dh, dw, db):
            t.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip((loss, lse, dh, dw, db), want):
            assert torch.equal(p, q)


def test_two_streams_at_once():
    ins = [make(40 + k, 150, 256, 4000, "bf16", True) for k in range(2)]
    want = []
    for h, W, b, y, gl, gz in ins:
        loss, lse = L.xent_forward(h, W, y, 1.0, b)
        want.append((loss, lse, *L.xent_backward(gl, h, W, y, lse, 1.0, b)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(3):
        for k, (h, W, b, y, gl, gz) in enumerate(ins):
            loss, lse = L.xent_forward(h, W, y, 1.0, b, stream=streams[k])
            got[k] = (loss, lse, *L.xent_backward(gl, h, W, y, lse, 1.0, b, stream=streams[k]))
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        for a, c in zip(p, q):
            assert torch.equal(a, c)


# at most 64 rows, where the weight's gradient walks down the vocabulary: one
# block of columns and several a work-group, ends inside a 16-row store, a
# block, a wave's 64 columns of H, a slab of 256
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,H,V", [(1, 32, 1), (1, 4128, 5000), (2, 64, 129), (17, 96, 12001), (33, 288, 70005),
                                   (63, 2048, 15193), (64, 320, 128), (64, 224, 100003), (65, 288, 8200)])
def test_weight_gradient_of_few_rows(M, H, V, dt):
    say(f"xent few rows M={M} H={H} V={V} {dt}")
    h, W, b, y, gl, gz = make(M + H + V, M, H, V, dt, False, target="ignored")
    _, lse, dh, dw, _ = check(h, W, b, y, gl, gz, 0.5)
    guard = torch.full((V + 2, H), 7.0, dtype=h.dtype, device=DEV)
    _, alone, _ = L.xent_backward(gl, h, W, y, lse, 0.5, grad_lse=gz, need_hidden=False)
    assert torch.equal(alone, dw)
    ws = torch.empty(L.xent_backward_workspace_bytes(M, H, V), dtype=torch.uint8, device=DEV)
    st = L._lib.load().lmhead_xent_backward(
        h.data_ptr(), M, H, W.data_ptr(), V, 0.5, None, {"bf16": 1, "f16": 2}[dt], y.data_ptr(), 1, -100,
        lse.data_ptr(), gl.data_ptr(), gz.data_ptr(), None, guard[1:].data_ptr(), None, ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(guard[1:V + 1], dw) and bool((guard[0] == 7).all()) and bool((guard[V + 1] == 7).all())


@pytest.mark.parametrize("M,H,V", [(3, 1 << 16, 70), (5, 32, 1 << 20)])
def test_the_contracts_maxima(M, H, V):
    say(f"xent maxima M={M} H={H} V={V}")
    h, W, b, y, gl, gz = make(47, M, H, V, "bf16", False, std=0.1)
    y[0] = V - 1
    check(h, W, b, y, gl, None, 0.5)


def test_differentiable():
    M, H, V = 50, 64, 400
    h, W, b, y, gl, gz = make(53, M, H, V, "bf16", True, target="ignored")
    for t in (h, W, b):
        t.requires_grad_(True)
    loss, lse = L.cross_entropy(h, W, y, 0.5, b, reduction="mean", return_lse=True)
    (loss + 0.01 * lse.square().mean()).backward()
    keep = y != -100
    with torch.no_grad():
        l2, s2 = L.xent_forward(h, W, y, 0.5, b)
        # the upstream gradients autograd hands down, in its own arithmetic
        s3 = s2.clone().requires_grad_(True)
    (0.01 * s3.square().mean()).backward()
    g = torch.ones(M, device=DEV) / keep.sum()
    want = L.xent_backward(g, h.detach(), W.detach(), y, s2, 0.5, b.detach(), grad_lse=s3.grad)
    assert float(loss) == float(l2.sum() / keep.sum())
    for t, w in zip((h, W, b), want):
        assert torch.equal(t.grad, w)
    # only what is asked for; the same from "sum" scaled by hand; from "none"
    h2 = h.detach().requires_grad_(True)
    L.cross_entropy(h2, W.detach(), y, 0.5, b.detach(), reduction="sum").backward()
    w2 = L.xent_backward(torch.ones(M, device=DEV), h2.detach(), W.detach(), y, s2, 0.5, b.detach())
    assert torch.equal(h2.grad, w2[0])
    h3 = h.detach().requires_grad_(True)
    L.cross_entropy(h3, W.detach(), y, 0.5, b.detach(), reduction="none").backward(gl)
    assert torch.equal(h3.grad, L.xent_backward(gl, h3.detach(), W.detach(), y, s2, 0.5, b.detach())[0])
    # only the log-sum-exp
    h4 = h.detach().requires_grad_(True)
    L.cross_entropy(h4, W.detach(), y, 0.5, b.detach(), return_lse=True)[1].sum().backward()
    w4 = L.xent_backward(torch.zeros(M, device=DEV), h4.detach(), W.detach(), y, s2, 0.5, b.detach(),
                         grad_lse=torch.ones(M, device=DEV))
    assert torch.equal(h4.grad, w4[0])
