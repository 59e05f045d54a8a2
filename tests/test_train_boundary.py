"""The training and int8 entry points without a GPU: bad arguments are refused
on the host, with nothing launched."""
import pytest
import torch

import lm_head_logits_amd as L
from lm_head_logits_amd import _lib

FAKE = 1 << 20  # aligned, non-null, never dereferenced on these paths
OK, NH, INV, ALIGN = _lib.OK, _lib.NOT_HANDLED, _lib.ERR_INVALID, _lib.ERR_ALIGN
BF16, F16, F32 = _lib.LMHEAD_BF16, _lib.LMHEAD_F16, _lib.LMHEAD_F32
MAX = (1 << 63) - 1


def fwd(hidden=FAKE, M=4, H=64, W=FAKE, V=100, alpha=1.0, bias=None, dt=BF16, target=FAKE, ti=1, ignore=-100,
        loss=FAKE, lse=FAKE, ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_xent_forward(hidden, M, H, W, V, alpha, bias, dt, target, ti, ignore, loss, lse, ws,
                                           wsb, None)


def bwd(hidden=FAKE, M=4, H=64, W=FAKE, V=100, alpha=1.0, bias=None, dt=BF16, target=FAKE, ti=1, ignore=-100,
        lse=FAKE, gl=FAKE, glse=None, dh=FAKE, dw=FAKE, db=None, ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_xent_backward(hidden, M, H, W, V, alpha, bias, dt, target, ti, ignore, lse, gl, glse,
                                            dh, dw, db, ws, wsb, None)


def emb(ids=FAKE, ti=1, M=4, W=FAKE, V=100, H=64, dt=BF16, scale=1.0, out=FAKE):
    return _lib.load().lmhead_embed(ids, ti, M, W, V, H, dt, scale, out, None)


def embb(ids=FAKE, ti=1, M=4, go=FAKE, V=100, H=64, dt=BF16, scale=1.0, pad=-1, acc=0, gw=FAKE, ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_embed_backward(ids, ti, M, go, V, H, dt, scale, pad, acc, gw, ws, wsb, None)


def quant(x=FAKE, R=4, H=64, dt=BF16, q=FAKE, s=FAKE):
    return _lib.load().lmhead_quantize_int8(x, R, H, dt, q, s, None)


def int8(h=FAKE, hs=FAKE, M=4, H=64, W=FAKE, ws=FAKE, V=100, alpha=1.0, bias=None, dt=BF16, out=FAKE):
    return _lib.load().lmhead_logits_int8(h, hs, M, H, W, ws, V, alpha, bias, dt, out, None)


SHAPES = [(dict(M=-1), INV), (dict(H=0), INV), (dict(V=0), INV), (dict(H=48), NH), (dict(H=(1 << 16) + 32), INV),
          (dict(V=(1 << 20) + 1), INV), (dict(M=(1 << 24) + 1), INV)]


@pytest.mark.parametrize("call", [fwd, bwd, emb, embb, int8])
@pytest.mark.parametrize("kw,want", SHAPES)
def test_shapes_outside_the_contract(call, kw, want):
    assert call(**kw) == want


def test_quantize_shapes():
    assert quant(R=-1) == INV and quant(H=0) == INV and quant(H=40) == NH and quant(R=(1 << 24) + 1) == INV
    assert quant(R=0, x=None, q=None, s=None) == OK


@pytest.mark.parametrize("call", [fwd, bwd, emb, embb, quant])
def test_types(call):
    assert call(dt=F32) == NH
    assert call(dt=7) == INV
    if call is not quant:
        assert call(ti=2) == INV and call(ti=-1) == INV
    assert int8(dt=9) == INV


@pytest.mark.parametrize("call,names", [
    (fwd, ("hidden", "W", "target", "loss", "lse", "ws")),
    (bwd, ("hidden", "W", "target", "lse", "gl", "ws")),
    (emb, ("ids", "W", "out")), (embb, ("ids", "go", "gw", "ws")),
    (quant, ("x", "q", "s")), (int8, ("h", "hs", "W", "ws", "out"))])
def test_null_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == INV, n


@pytest.mark.parametrize("call,names", [
    (fwd, dict(hidden=8, W=8, target=4, loss=2, lse=2, bias=2, ws=8)),
    (bwd, dict(hidden=8, W=8, target=4, lse=2, gl=2, glse=2, dh=8, dw=8, db=2, ws=16)),
    (emb, dict(ids=4, W=8, out=8)), (embb, dict(ids=4, go=8, gw=8, ws=16)),
    (quant, dict(x=8, q=8, s=2)), (int8, dict(h=8, hs=2, W=8, ws=2, bias=2, out=8))])
def test_alignment(call, names):
    for n, off in names.items():
        assert call(**{n: FAKE + off}) == ALIGN, n


def test_int32_indices_need_four_bytes():
    # past the pointer checks these would launch: a misaligned int32 address is what is refused
    for call, n in ((fwd, "target"), (bwd, "target"), (emb, "ids"), (embb, "ids")):
        assert call(ti=0, **{n: FAKE + 2}) == ALIGN


def test_workspaces():
    lib = _lib.load()
    for M, H, V in ((1, 32, 1), (333, 4096, 128256), (4096, 4096, 128256), (1 << 17, 2048, 151936)):
        f, b = L.xent_forward_workspace_bytes(M, V), L.xent_backward_workspace_bytes(M, H, V)
        assert f >= 8 * M * ((V + 255) // 256) and b > 0
        assert L.xent_backward_workspace_bytes(M, H, V, True) >= b
        assert fwd(M=M, H=H, V=V, wsb=f - 1) == INV and bwd(M=M, H=H, V=V, wsb=b - 1) == INV
        # a piece of the logits' gradient and fp32 sums of grad_hidden, not all of [M, V]
        assert b <= max(256 << 20, 2 * 8192 * M) + 4 * 64 * max(M, 256) * H + 16 * M + (1 << 20)
        e = L.embed_backward_workspace_bytes(M, H)
        assert e > 8 * M and embb(M=M, H=H, wsb=e - 1) == INV
    assert lib.lmhead_xent_forward_workspace_bytes(-1, 5) == 0
    assert lib.lmhead_xent_backward_workspace_bytes(4, 48, 5, 0) == 0
    assert lib.lmhead_embed_backward_workspace_bytes(4, 48) == 0


def test_nothing_to_do():
    assert fwd(M=0, hidden=None, W=None, target=None, loss=None, lse=None, ws=None, wsb=0) == OK
    assert bwd(dh=None, dw=None, db=None, hidden=None) == OK
    assert bwd(M=0, hidden=None, W=None, target=None, lse=None, gl=None, dw=None, ws=None, wsb=0) == OK
    assert emb(M=0, ids=None, W=None, out=None) == OK
    assert embb(M=0, acc=1, ids=None, go=None, ws=None, wsb=0) == OK
    assert int8(M=0, h=None, hs=None, W=None, ws=None, out=None) == OK


def test_python_refuses_host_tensors_and_wrong_metadata():
    h, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16)
    y, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    for call in (lambda: L.xent_forward(h, W, y), lambda: L.xent_backward(f, h, W, y, f),
                 lambda: L.cross_entropy(h, W, y), lambda: L.embed(y, W), lambda: L.embedding(y, W),
                 lambda: L.embed_backward(h, y, 9), lambda: L.quantize_int8(h),
                 lambda: L.logits_int8(h.to(torch.int8), f, W.to(torch.int8), torch.zeros(9))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="reduction"):
        L.cross_entropy(h, W, y, reduction="median")
