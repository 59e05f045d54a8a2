"""The differentiable losses and their memory without a GPU: when a backward pass is
prepared, which arguments may ask for a gradient, what is asked of the allocator."""
import pytest
import torch

import lm_head_logits_amd as L
from lm_head_logits_amd import losses

M, H, V, K = 4, 64, 9, 3
Y, F = torch.zeros(M, dtype=torch.int64), torch.zeros(M)
IDS, S, CUTS = torch.zeros(M, K, dtype=torch.int64), torch.zeros(M, K), torch.tensor([0, 2, 4])


def head(grad=True):
    return [torch.zeros(*s, dtype=t, requires_grad=grad)
            for s, t in (((M, H), torch.bfloat16), ((V, H), torch.bfloat16), ((V,), torch.float32))]


CALLS = {"distill": lambda h, w, b, **kw: L.distillation(h, w, IDS, S, bias=b, reduction="none", **kw),
         "policy": lambda h, w, b, **kw: L.policy_loss(h, w, Y, F, bias=b, reduction="none", **kw),
         "preference": lambda h, w, b, **kw: L.preference_loss(h, w, Y, CUTS, bias=b, reduction="none", **kw)}


@pytest.mark.parametrize("op", list(CALLS))
def test_a_backward_pass_is_prepared_where_one_can_follow(op, monkeypatch):
    seen = []

    def forward(*args, train=True, **kw):
        seen.append(train)
        saved = losses.LossState(torch.zeros(0), args[0], None, 1.0, 1.0, 0, M, False) if train else None
        return (*[torch.zeros(M) for _ in range(1 if op == "distill" else 2)], saved)

    monkeypatch.setattr(losses, {"distill": "distill_forward", "policy": "policy_forward",
                                 "preference": "preference_forward"}[op], forward)
    call = CALLS[op]
    h, w, b = head()
    call(h, w, b)
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            call(h, w, b)
    call(*head(False))
    for k in range(3):  # any of the three
        x = head(False)
        x[k].requires_grad_()
        assert call(*x).requires_grad
    with torch.no_grad(), torch.enable_grad():
        call(h, w, b)
    assert seen == [True, False, False, False, True, True, True, True]


@pytest.mark.parametrize("call,names", [
    (lambda **kw: L.distillation(*head()[:2], **{"teacher_ids": IDS, "teacher_logits": S, **kw}), ("teacher_logits", "teacher_lse")),
    (lambda **kw: L.policy_loss(*head()[:2], **{"target": Y, "advantage": F, **kw}), ("advantage", "old_logp", "ref_logp")),
    (lambda **kw: L.preference_loss(*head()[:2], Y, CUTS, **kw), ("ref_logp",))])
def test_no_gradient_is_dropped_in_silence(call, names):
    for name in names:
        x = (S if name == "teacher_logits" else F).clone().requires_grad_()
        with pytest.raises(ValueError, match=f"{name}.*detach"):
            call(**{name: x})
        for fine in (lambda: call(**{name: x.detach()}), torch.no_grad()(lambda: call(**{name: x}))):
            with pytest.raises(ValueError, match="device tensor"):  # host tensors: the next check
                fine()


def test_logits_are_kept_where_there_is_room(monkeypatch):
    """Without room for the logits the state is one without them; an allocation that
    the caller asked for, or the lean one, fails as it does."""
    lean, full = (L.loss_state_bytes(M, H, 5000, 0, k) for k in (False, True))
    real = torch.empty
    limit = [1 << 40]

    def empty(n, *args, **kw):
        if isinstance(n, int) and n > limit[0]:
            raise torch.OutOfMemoryError("no room")
        return real(n, *args, **kw)

    monkeypatch.setattr(torch, "empty", empty)
    memory = lambda keep: losses._Memory(M, H, 5000, 0, True, keep, real(16, dtype=torch.uint8), torch.device("cpu"))
    monkeypatch.setattr(losses, "_workspace", lambda *a: a[0])
    assert memory(None).keep and memory(None).state.numel() == full and not memory(False).keep
    limit[0] = full - 1
    m = memory(None)
    assert not m.keep and m.state.numel() == lean and m.args()[2] == 0
    with pytest.raises(torch.OutOfMemoryError):
        memory(True)
    limit[0] = lean - 1
    for keep in (None, False):
        with pytest.raises(torch.OutOfMemoryError):
            memory(keep)


@pytest.mark.parametrize("M,H,V", [(65536, 4096, 128256), (1 << 17, 2048, 151936), (8192, 4096, 128256), (8192, 8192, 32000)])
def test_backward_workspace_of_many_rows(M, H, V):
    """The cross entropy's, whose sums of grad_hidden are not split for that many rows,
    and room for the splits of fewer: a split more is taken below 1024 tiles of sums
    only, so that fewer than 2048 are written. A piece may have an eighth more columns."""
    tiles = -(-M // 256) * -(-H // 256)
    room = L.xent_backward_workspace_bytes(M, H, V) + 2 * M * (V // 8 + 256) + max(0, 2048 - tiles) * 4 * 256 * 256 + 4096
    assert L.loss_backward_workspace_bytes(M, H, V) <= room


@pytest.mark.parametrize("M,H,V,pieces", [(1337, 4096, 200000, 391), (1337, 2048, 200000, 391), (1000, 2048, 151936, 320),
                                          (4096, 2048, 151936, 128), (4096, 4096, 128256, 126)])
def test_pieces_stay_in_the_memory_side_cache(M, H, V, pieces):
    """G of a piece: whole rounds of work-groups' worth of columns up to 256 MiB, else
    the cross entropy's pieces. With a bias a row tile's sums take 4 bytes a column more."""
    col = L.loss_backward_workspace_bytes(M, H, V, grad_bias=True) - L.loss_backward_workspace_bytes(M, H, V)
    assert col == 4 * -(-M // 256) * pieces * 256 and 2 * M * pieces * 256 <= 256 << 20
