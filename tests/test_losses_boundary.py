"""The losses' and the top logits' entry points without a GPU: bad arguments
are refused on the host, with nothing launched; sizes of states and workspaces."""
import math

import pytest
import torch

import lm_head_logits_amd as L
from lm_head_logits_amd import _lib

FAKE = 1 << 20  # aligned, non-null, never dereferenced on these paths
OK, NH, INV, ALIGN = _lib.OK, _lib.NOT_HANDLED, _lib.ERR_INVALID, _lib.ERR_ALIGN
BF16, F16, F32 = _lib.LMHEAD_BF16, _lib.LMHEAD_F16, _lib.LMHEAD_F32
MAX = (1 << 63) - 1


def distill(hidden=FAKE, M=4, H=64, W=FAKE, V=100, alpha=1.0, bias=None, dt=BF16, T=1.0, ids=FAKE, ti=1, logits=FAKE, ldt=F32,
            K=8, tlse=None, loss=FAKE, state=FAKE, sb=MAX, keep=0, ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_distill_forward(hidden, M, H, W, V, alpha, bias, dt, T, ids, ti, logits, ldt, K, tlse, loss,
                                              state, sb, keep, ws, wsb, None)


def policy(hidden=FAKE, M=4, H=64, W=FAKE, V=100, alpha=1.0, bias=None, dt=BF16, T=1.0, target=FAKE, ti=1, ignore=-100,
           adv=FAKE, old=None, ref=None, low=0.2, high=0.2, kl=0.0, loss=FAKE, logp=FAKE, state=FAKE, sb=MAX, keep=0,
           ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_policy_forward(hidden, M, H, W, V, alpha, bias, dt, T, target, ti, ignore, adv, old, ref, low,
                                             high, kl, loss, logp, state, sb, keep, ws, wsb, None)


def preference(hidden=FAKE, M=4, H=64, W=FAKE, V=100, alpha=1.0, bias=None, dt=BF16, T=1.0, target=FAKE, ti=1, ignore=-100,
               starts=FAKE, si=1, pairs=2, ref=None, beta=0.1, margin=0.0, smooth=0.0, average=0, loss=FAKE, logp=FAKE,
               state=FAKE, sb=MAX, keep=0, ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_preference_forward(hidden, M, H, W, V, alpha, bias, dt, T, target, ti, ignore, starts, si, pairs,
                                                 ref, beta, margin, smooth, average, loss, logp, state, sb, keep, ws, wsb,
                                                 None)


def backward(hidden=FAKE, M=4, H=64, W=FAKE, V=100, alpha=1.0, bias=None, dt=BF16, T=1.0, K=0, g=FAKE, state=FAKE, sb=MAX,
             keep=0, dh=FAKE, dw=FAKE, db=None, ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_loss_backward(hidden, M, H, W, V, alpha, bias, dt, T, K, g, state, sb, keep, dh, dw, db, ws, wsb,
                                            None)


def topk(x=FAKE, M=4, V=100, ld=None, dt=BF16, K=8, T=1.0, values=FAKE, ids=FAKE, lse=FAKE, ws=FAKE, wsb=MAX):
    return _lib.load().lmhead_logits_topk(x, M, V, V if ld is None else ld, dt, K, T, values, ids, lse, ws, wsb, None)


CALLS = [distill, policy, preference, backward]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(H=0), INV), (dict(V=0), INV), (dict(H=48), NH), (dict(H=(1 << 16) + 32), INV),
    (dict(V=(1 << 20) + 1), INV), (dict(M=(1 << 24) + 1), INV), (dict(M=1 << 23, V=1 << 20), INV), (dict(dt=F32), NH),
    (dict(dt=7), INV), (dict(T=0.0), INV), (dict(T=-1.0), INV), (dict(T=math.inf), INV), (dict(T=math.nan), INV)])
def test_shapes_types_and_temperatures(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw", [dict(M=-1), dict(V=0), dict(V=(1 << 20) + 1), dict(M=(1 << 24) + 1), dict(dt=7), dict(K=0),
                                dict(K=101), dict(V=2000, K=1025), dict(ld=99), dict(T=0.0), dict(T=math.nan),
                                dict(T=math.inf), dict(ld=1 << 60)])
def test_topk_arguments(kw):
    assert topk(**kw) == INV


def test_other_arguments():
    assert distill(K=0) == INV and distill(K=1025) == INV and distill(ldt=5) == INV and distill(ti=2) == INV
    assert policy(low=-0.1) == INV and policy(high=-0.1) == INV and policy(low=math.nan) == INV and policy(kl=math.nan) == INV
    assert policy(ti=9) == INV and preference(ti=9) == INV and preference(si=-1) == INV
    assert preference(pairs=-1) == INV and preference(pairs=1 << 24) == INV
    for bad in (-0.1, 1.1, math.nan):
        assert preference(smooth=bad) == INV
    assert preference(beta=math.nan) == INV and preference(margin=math.nan) == INV
    assert backward(K=1025) == INV and backward(K=-1) == INV


@pytest.mark.parametrize("call,names", [
    (distill, ("hidden", "W", "ids", "logits", "loss", "ws")), (policy, ("hidden", "W", "target", "adv", "loss", "logp", "ws")),
    (preference, ("hidden", "W", "target", "starts", "loss", "logp", "ws")), (backward, ("hidden", "W", "state", "ws")),
    (topk, ("x", "values", "ids", "lse"))])
def test_null_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == INV, n
    if call in (distill, policy, preference):  # logits can be kept only in a state
        assert call(state=None, keep=1) == INV
    if call is topk:
        assert topk(V=200000, M=1, ws=None) == INV


@pytest.mark.parametrize("call,names", [
    (distill, dict(hidden=8, W=8, ids=4, logits=2, tlse=2, loss=2, bias=2, state=64, ws=64)),
    (policy, dict(hidden=8, W=8, target=4, adv=2, old=2, ref=2, loss=2, logp=2, bias=2, state=64, ws=64)),
    (preference, dict(hidden=8, W=8, target=4, starts=4, ref=2, loss=2, logp=2, bias=2, state=64, ws=64)),
    (backward, dict(hidden=8, W=8, g=2, dh=8, dw=8, db=2, bias=2, state=64, ws=64)),
    (topk, dict(x=1, values=1, ids=2, lse=2, ws=8))])
def test_alignment(call, names):
    for n, off in names.items():
        assert call(**{n: FAKE + off}) == ALIGN, n
    for n in ("ids", "target", "starts"):
        if n in names and call is not topk:
            kw = dict(si=0) if n == "starts" else dict(ti=0)
            assert call(**{n: FAKE + 2}, **kw) == ALIGN, n
    if call is distill:
        assert distill(ldt=BF16, logits=FAKE + 1) == ALIGN
    if call is topk:
        assert topk(dt=F32, x=FAKE + 2) == ALIGN and topk(dt=F32, values=FAKE + 2) == ALIGN


def test_sizes():
    lib = _lib.load()
    for M, H, V in ((1, 32, 1), (256, 64, 500), (257, 64, 500), (4096, 4096, 128256), (1 << 17, 2048, 151936)):
        for K in (0, 1, 64, 1024):
            call = distill if K else policy
            kw = dict(M=M, H=H, V=V, **(dict(K=K) if K else {}))
            for keep in (0, 1):
                s, b = L.loss_state_bytes(M, H, V, K, keep), L.loss_backward_workspace_bytes(M, H, V, K, keep)
                f = L.loss_forward_workspace_bytes(M, H, V, K)
                assert call(**kw, keep=keep, sb=s - 1) == INV and call(**kw, keep=keep, wsb=f - 1) == INV
                assert call(**kw, state=None, wsb=L.loss_forward_workspace_bytes(M, H, V, K, False) - 1) == INV
                assert backward(M=M, H=H, V=V, K=K, keep=keep, sb=s - 1) == INV
                assert backward(M=M, H=H, V=V, K=K, keep=keep, wsb=b - 1) == INV
                assert L.loss_backward_workspace_bytes(M, H, V, K, keep, True) >= b
                # all logits only where they are kept
                if keep:
                    assert s >= 4 * M * V
                else:
                    assert s <= M * (2 * H + 12 * K + 32) + 4 * V + 8192
            assert preference(M=M, H=H, V=V, sb=L.loss_state_bytes(M, H, V) - 1) == INV
    assert lib.lmhead_loss_state_bytes(4, 48, 5, 0, 0) == 0 and lib.lmhead_loss_state_bytes(0, 64, 5, 0, 0) == 0
    assert lib.lmhead_loss_state_bytes(4, 64, 5, 1025, 0) == 0 and lib.lmhead_loss_state_bytes(4, 64, 5, -1, 0) == 0
    assert lib.lmhead_loss_forward_workspace_bytes(-1, 64, 5, 0, 0) == 0
    assert lib.lmhead_loss_backward_workspace_bytes(4, 64, 0, 0, 0, 0) == 0
    for M, V, K in ((1, 151936, 20), (48, 128256, 50), (3, 1 << 20, 1024)):
        n = L.logits_topk_workspace_bytes(M, V, K)
        assert n >= 8 * M * 2 * K and topk(M=M, V=V, K=K, wsb=n - 1) == INV
    assert L.logits_topk_workspace_bytes(4096, 128256, 64) == 0 and L.logits_topk_workspace_bytes(1, 100, 101) == 0


def test_nothing_to_do():
    none = dict(hidden=None, W=None, loss=None, state=None, ws=None, sb=0, wsb=0)
    assert distill(M=0, ids=None, logits=None, **none) == OK
    assert policy(M=0, target=None, adv=None, logp=None, **none) == OK
    assert preference(M=0, pairs=0, target=None, starts=None, logp=None, **none) == OK
    assert backward(dh=None, dw=None, db=None, hidden=None) == OK
    assert backward(M=0, hidden=None, W=None, g=None, state=None, sb=0, dw=None, ws=None, wsb=0) == OK
    assert topk(M=0, x=None, values=None, ids=None, lse=None, ws=None, wsb=0) == OK


def test_python_refuses_host_tensors_and_wrong_metadata():
    h, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16)
    y, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    ids, s, cuts = torch.zeros(4, 3, dtype=torch.int64), torch.zeros(4, 3), torch.tensor([0, 2, 4])
    for call in (lambda: L.distill_forward(h, W, ids, s), lambda: L.distillation(h, W, ids, s),
                 lambda: L.policy_forward(h, W, y, f), lambda: L.policy_loss(h, W, y, f),
                 lambda: L.preference_forward(h, W, y, cuts), lambda: L.preference_loss(h, W, y, cuts),
                 lambda: L.loss_backward(f, W, L.LossState(f, h, None, 1.0, 1.0, 0, 4, False)), lambda: L.logits_topk(s, 2),
                 lambda: L.loss_backward(f, W, None)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: L.distillation(h, W, ids, s, reduction="median"),
                 lambda: L.policy_loss(h, W, y, f, reduction="median"),
                 lambda: L.preference_loss(h, W, y, cuts, reduction="median")):
        with pytest.raises(ValueError, match="reduction"):
            call()
