"""Further losses of the head's logits, which need not be whole in memory: the
divergence from a teacher's top logits (lmhead_distill_forward), the clipped
policy loss with a KL term (lmhead_policy_forward) and the logistic loss of
preferred pairs (lmhead_preference_forward), each with its gradients
(lmhead_loss_backward). And the rows' top logits (lmhead_logits_topk), which a
teacher hands down and a token is sampled from.

``logits_topk``, ``distill_forward``, ``policy_forward``, ``preference_forward``
and ``loss_backward`` are the C calls with torch tensors; ``distillation``,
``policy_loss`` and ``preference_loss`` are the same as differentiable
functions.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from ._binding import _DTYPES, _alloc_on, _check, _device_ctx, _need, _same_device, _stream_handle
from .training import _f32_arg, _head_args, _index_arg, _ptr, _Total, _total, _workspace


class LossState(NamedTuple):
    """What a forward call leaves for loss_backward."""
    state: torch.Tensor   # bytes, the library's own layout
    hidden: torch.Tensor
    bias: torch.Tensor | None
    alpha: float
    temperature: float
    K: int                # the teacher's logits a row; 0 for the losses of targets
    elements: int         # of the loss, and so of its upstream gradient
    keep_logits: bool     # the logits are in the state
    V: int = 0            # rows of the weight (sizes of states are rounded up: others may have the same)


# Up to this many bytes of fp32 logits a forward call for training keeps them for
# the backward pass by default: a quarter of the pass's products saved (4096 rows,
# H = 4096, V = 128256: 12.6 -> 10.0 ms) for a small share of the card's 288 GB.
KEEP_BYTES = 16 << 30


def loss_state_bytes(M: int, H: int, V: int, K: int = 0, keep_logits: bool = False) -> int:
    return int(_lib.load().lmhead_loss_state_bytes(M, H, V, K, int(keep_logits)))


def loss_forward_workspace_bytes(M: int, H: int, V: int, K: int = 0, train: bool = True) -> int:
    return int(_lib.load().lmhead_loss_forward_workspace_bytes(M, H, V, K, int(train)))


def loss_backward_workspace_bytes(M: int, H: int, V: int, K: int = 0, keep_logits: bool = False,
                                  grad_bias: bool = False) -> int:
    return int(_lib.load().lmhead_loss_backward_workspace_bytes(M, H, V, K, int(keep_logits), int(grad_bias)))


class _Memory:
    """State and workspace of a forward call."""

    def __init__(self, M, H, V, K, train, keep_logits, workspace, dev):
        self.keep = train and (4 * M * V <= KEEP_BYTES if keep_logits is None else bool(keep_logits))
        self.state = None
        if train:
            try:
                self.state = torch.empty(loss_state_bytes(M, H, V, K, self.keep), dtype=torch.uint8, device=dev)
            except torch.OutOfMemoryError:
                if keep_logits is not None or not self.keep:
                    raise
                self.keep = False  # kept by default only, and there is no room for them
                self.state = torch.empty(loss_state_bytes(M, H, V, K, False), dtype=torch.uint8, device=dev)
        self.workspace = _workspace(workspace, loss_forward_workspace_bytes(M, H, V, K, train), dev)

    def args(self):
        st, ws = self.state, self.workspace
        return (st.data_ptr() if st is not None and st.numel() else None, st.numel() if st is not None else 0,
                int(self.keep), ws.data_ptr(), ws.numel() * ws.element_size())

    def saved(self, hidden, weight, bias, alpha, temperature, K, elements):
        if self.state is None:
            return None
        return LossState(self.state, hidden, bias, float(alpha), float(temperature), K, elements, self.keep,
                         weight.shape[0])


def logits_topk_workspace_bytes(M: int, V: int, k: int) -> int:
    return int(_lib.load().lmhead_logits_topk_workspace_bytes(M, V, k))


def logits_topk(logits: torch.Tensor, k: int, temperature: float = 1.0, *, workspace: torch.Tensor | None = None,
                stream=None):
    """The k largest logits of each row of logits [M, V] (float32, bfloat16 or
    float16; rows may be further apart than V, as in a slice of padded columns)
    in descending order, equal ones by ascending column (lmhead_logits_topk):
    returns (values [M, k] of the logits' type, ids int32 [M, k], lse fp32 [M]),
    lse being the log-sum-exp of the whole row of logits / temperature, so that
    values.float() / temperature - lse are the candidates' log-probabilities. It
    gives no gradient to logits."""
    _need(logits.is_cuda and logits.dtype in _DTYPES and logits.dim() == 2,
          "logits must be a device tensor [M, V], float32, bfloat16 or float16")
    M, V = logits.shape
    _need(V == 1 or logits.stride(1) == 1, "a row's logits must be next to each other")
    ld = logits.stride(0) if M > 1 else V
    _need(ld >= V, "rows must not overlap")
    _need(1 <= k <= V, "k must be 1 .. V")
    dev = logits.device
    with _alloc_on(stream):
        values = torch.empty((M, k), dtype=logits.dtype, device=dev)
        ids = torch.empty((M, k), dtype=torch.int32, device=dev)
        lse = torch.empty(M, dtype=torch.float32, device=dev)
        workspace = _workspace(workspace, logits_topk_workspace_bytes(M, V, k), dev)
    _same_device(logits, workspace)
    with _device_ctx(dev):
        st = _lib.load().lmhead_logits_topk(
            logits.data_ptr(), M, V, ld, _DTYPES[logits.dtype], k, float(temperature), values.data_ptr(), ids.data_ptr(),
            lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream_handle(dev, stream))
    _check(st, "lmhead_logits_topk")
    return values, ids, lse


def _optional_f32(t, M, name):
    if t is not None:
        _f32_arg(t, M, name)


def distill_forward(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                    alpha: float = 1.0, bias=None, *, temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                    train: bool = True, keep_logits: bool | None = None, workspace: torch.Tensor | None = None,
                    stream=None):
    """Divergence of the head's distribution at `temperature` from a teacher's,
    given by its top logits (lmhead_distill_forward): returns (loss fp32 [M],
    saved). teacher_ids [M, K] (int32 or int64) and teacher_logits [M, K]
    (float32, bfloat16 or float16) in any order, as logits_topk gives them;
    entries whose id is no row of weight, or whose logit is -inf, are absent, and
    a row without entries has loss 0. The teacher's probabilities are normalised
    over the entries, or, with teacher_lse (fp32 [M], the log-sum-exp of its
    logits / temperature over its whole vocabulary), are those of its whole
    distribution. saved is what loss_backward takes (None where train is
    false); keep_logits: it holds the logits too, fp32 [M, V], which saves making
    them again there (None: up to 16 GB of them, where they can be allocated)."""
    M, H, V, code = _head_args(hidden, weight, bias)
    _need(teacher_ids.dim() == 2 and teacher_ids.shape[0] == M and teacher_ids.shape[1] >= 1,
          "teacher_ids must be [M, K]")
    K = teacher_ids.shape[1]
    itype = _index_arg(teacher_ids, (M, K), "teacher_ids")
    if not (teacher_logits.is_cuda and teacher_logits.dtype in _DTYPES and teacher_logits.shape == (M, K)
            and teacher_logits.is_contiguous()):
        raise ValueError("teacher_logits must be a contiguous device tensor [M, K], float32, bfloat16 or float16")
    _optional_f32(teacher_lse, M, "teacher_lse")
    dev = hidden.device
    with _alloc_on(stream):
        loss = torch.empty(M, dtype=torch.float32, device=dev)
        mem = _Memory(M, H, V, K, train, keep_logits, workspace, dev)
    _same_device(hidden, weight, bias, teacher_ids, teacher_logits, teacher_lse, mem.workspace)
    with _device_ctx(dev):
        st = _lib.load().lmhead_distill_forward(
            hidden.data_ptr(), M, H, weight.data_ptr(), V, float(alpha), _ptr(bias), code, float(temperature),
            teacher_ids.data_ptr(), itype, teacher_logits.data_ptr(), _DTYPES[teacher_logits.dtype], K,
            _ptr(teacher_lse), loss.data_ptr(), *mem.args(), _stream_handle(dev, stream))
    _check(st, "lmhead_distill_forward")
    return loss, mem.saved(hidden, weight, bias, alpha, temperature, K, M)


def policy_forward(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, advantage: torch.Tensor,
                   old_logp: torch.Tensor | None = None, ref_logp: torch.Tensor | None = None, alpha: float = 1.0,
                   bias=None, *, temperature: float = 1.0, clip_low: float = 0.2, clip_high: float = 0.2,
                   kl_coef: float = 0.0, ignore_index: int = -100, train: bool = True,
                   keep_logits: bool | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Clipped policy loss of the tokens target [M] with a KL term
    (lmhead_policy_forward): returns (loss fp32 [M], logp fp32 [M], saved), logp
    being the tokens' log-probabilities. advantage, old_logp (None: logp itself,
    the first step after a rollout) and ref_logp (None: no KL term) are fp32 [M].
    Rows whose target is ignore_index or no row of weight have loss and logp 0.
    saved and keep_logits are distill_forward's."""
    M, H, V, code = _head_args(hidden, weight, bias)
    itype = _index_arg(target, (M,), "target")
    _f32_arg(advantage, M, "advantage")
    _optional_f32(old_logp, M, "old_logp")
    _optional_f32(ref_logp, M, "ref_logp")
    dev = hidden.device
    with _alloc_on(stream):
        loss = torch.empty(M, dtype=torch.float32, device=dev)
        logp = torch.empty(M, dtype=torch.float32, device=dev)
        mem = _Memory(M, H, V, 0, train, keep_logits, workspace, dev)
    _same_device(hidden, weight, bias, target, advantage, old_logp, ref_logp, mem.workspace)
    with _device_ctx(dev):
        st = _lib.load().lmhead_policy_forward(
            hidden.data_ptr(), M, H, weight.data_ptr(), V, float(alpha), _ptr(bias), code, float(temperature),
            target.data_ptr(), itype, int(ignore_index), advantage.data_ptr(), _ptr(old_logp), _ptr(ref_logp),
            float(clip_low), float(clip_high), float(kl_coef), loss.data_ptr(), logp.data_ptr(),
            *mem.args(), _stream_handle(dev, stream))
    _check(st, "lmhead_policy_forward")
    return loss, logp, mem.saved(hidden, weight, bias, alpha, temperature, 0, M)


def preference_forward(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, starts: torch.Tensor,
                       ref_logp: torch.Tensor | None = None, alpha: float = 1.0, bias=None, *, beta: float = 0.1,
                       margin: float = 0.0, label_smoothing: float = 0.0, average: bool = False,
                       temperature: float = 1.0, ignore_index: int = -100, train: bool = True,
                       keep_logits: bool | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Logistic loss of P preferred pairs of sequences
    (lmhead_preference_forward): returns (loss fp32 [P], logp fp32 [2 P], saved).
    Sequence s is rows starts[s] .. starts[s + 1] - 1 of the batch (starts: int32
    or int64 [2 P + 1], ascending); sequences 0 .. P - 1 are the preferred ones,
    P .. 2 P - 1 the others. logp is the sum (average: the mean) of the log-
    probabilities of a sequence's targets, without those left out; ref_logp
    (None: zeros), fp32 [2 P], is a reference model's, as this function returns it.
    saved and keep_logits are distill_forward's."""
    M, H, V, code = _head_args(hidden, weight, bias)
    itype = _index_arg(target, (M,), "target")
    _need(starts.dim() == 1 and starts.shape[0] % 2 == 1, "starts must be [2 P + 1]")
    stype = _index_arg(starts, starts.shape, "starts")
    P = starts.shape[0] // 2
    if ref_logp is not None and not (ref_logp.is_cuda and ref_logp.dtype == torch.float32 and ref_logp.shape == (2 * P,)
                                     and ref_logp.is_contiguous()):
        raise ValueError("ref_logp must be a contiguous fp32 device tensor [2 P]")
    dev = hidden.device
    with _alloc_on(stream):
        loss = torch.empty(P, dtype=torch.float32, device=dev)
        logp = torch.empty(2 * P, dtype=torch.float32, device=dev)
        mem = _Memory(M, H, V, 0, train, keep_logits, workspace, dev)
    _same_device(hidden, weight, bias, target, starts, ref_logp, mem.workspace)
    with _device_ctx(dev):
        st = _lib.load().lmhead_preference_forward(
            hidden.data_ptr(), M, H, weight.data_ptr(), V, float(alpha), _ptr(bias), code, float(temperature),
            target.data_ptr(), itype, int(ignore_index), starts.data_ptr(), stype, P, _ptr(ref_logp), float(beta),
            float(margin), float(label_smoothing), int(average), loss.data_ptr(), logp.data_ptr(),
            *mem.args(), _stream_handle(dev, stream))
    _check(st, "lmhead_preference_forward")
    return loss, logp, mem.saved(hidden, weight, bias, alpha, temperature, 0, P)


def loss_backward(grad_loss: torch.Tensor, weight: torch.Tensor, saved: LossState, *, need_hidden: bool = True,
                  need_weight: bool = True, need_bias: bool | None = None, workspace: torch.Tensor | None = None,
                  stream=None):
    """Gradients of distill_forward, policy_forward or preference_forward
    (lmhead_loss_backward): returns (grad_hidden, grad_weight, grad_bias), of the
    inputs' types, None where not needed (need_bias: by default when there is a
    bias). grad_loss is fp32, of the loss's shape; saved is what the forward call
    returned, weight what it was given."""
    _need(isinstance(saved, LossState), "saved must be what a forward call with train=True returned")
    hidden, bias = saved.hidden, saved.bias
    M, H, V, code = _head_args(hidden, weight, bias)
    if not (grad_loss.is_cuda and grad_loss.dtype == torch.float32 and grad_loss.shape == (saved.elements,)
            and grad_loss.is_contiguous()):
        raise ValueError(f"grad_loss must be a contiguous fp32 device tensor [{saved.elements}]")
    if need_bias is None:
        need_bias = bias is not None
    _need(not need_bias or bias is not None, "there is no bias to differentiate")
    _need(saved.V == V and saved.state.numel() == loss_state_bytes(M, H, V, saved.K, saved.keep_logits),
          "saved is of a head of another size than weight")
    dev = hidden.device
    with _alloc_on(stream):
        dh = torch.empty_like(hidden) if need_hidden else None
        dw = torch.empty_like(weight) if need_weight else None
        db = torch.empty_like(bias) if need_bias else None
        workspace = _workspace(workspace, loss_backward_workspace_bytes(M, H, V, saved.K, saved.keep_logits, need_bias), dev)
    _same_device(hidden, weight, bias, grad_loss, saved.state, workspace)
    with _device_ctx(dev):
        st = _lib.load().lmhead_loss_backward(
            hidden.data_ptr(), M, H, weight.data_ptr(), V, saved.alpha, _ptr(bias), code, saved.temperature, saved.K,
            grad_loss.data_ptr(), saved.state.data_ptr(), saved.state.numel(), int(saved.keep_logits), _ptr(dh), _ptr(dw),
            _ptr(db),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_handle(dev, stream))
    _check(st, "lmhead_loss_backward")
    return dh, dw, db


class _HeadLoss(torch.autograd.Function):
    """forward(hidden, weight, bias, train, call): call(hidden, weight, bias, train)
    is one of the forward calls above with its other arguments bound."""

    @staticmethod
    def forward(ctx, hidden, weight, bias, train, call):
        *out, saved = call(hidden, weight, bias, train)
        if saved is not None:
            ctx.save_for_backward(hidden, weight, bias, saved.state)
            ctx.rest = saved[3:]
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(*out[1:])
        return tuple(out)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, *_):
        if grad_loss is None:
            return None, None, None, None, None
        hidden, weight, bias, state = ctx.saved_tensors
        dh, dw, db = loss_backward(grad_loss.contiguous(), weight, LossState(state, hidden, bias, *ctx.rest),
                                   need_hidden=ctx.needs_input_grad[0], need_weight=ctx.needs_input_grad[1],
                                   need_bias=ctx.needs_input_grad[2])
        return dh, dw, db, None, None


def _apply(hidden, weight, bias, call):
    """A backward pass is prepared where one can follow: in forward itself grad mode is
    off, and needs_input_grad is true of a parameter without grad mode too."""
    train = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (hidden, weight, bias))
    return _HeadLoss.apply(hidden, weight, bias, train, call)


def _reduce(loss, reduction, kept):
    """kept(): which elements the mean is over."""
    if reduction == "mean":
        return _Total.apply(loss) / _total(kept())
    return _Total.apply(loss) if reduction == "sum" else loss


def _check_reduction(reduction):
    _need(reduction in ("none", "sum", "mean"), "reduction must be none, sum or mean")


def _check_constants(**tensors):
    """What the losses are not differentiated by must not ask for it: the gradient would be missing in silence."""
    for name, t in tensors.items():
        _need(t is None or not t.requires_grad or not torch.is_grad_enabled(),
              f"there is no gradient for {name}: detach it")


def distillation(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                 alpha: float = 1.0, bias=None, *, temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                 keep_logits: bool | None = None, reduction: str = "mean") -> torch.Tensor:
    """Differentiable distill_forward. reduction: "none" (fp32 [M]), "sum", or
    "mean" over the rows that have entries (NaN when there are none). Losses at a
    temperature T are usually weighted by T * T; that is left to the caller.
    keep_logits as there, here and in the functions below: False saves fp32 [M, V]
    between the passes, the gradients stay as they are. Here and there gradients are
    those of hidden, weight and bias: without grad mode, or where none of them requires
    one, only the loss is computed, and any other tensor that requires one is refused
    (ValueError)."""
    _check_reduction(reduction)
    _check_constants(teacher_logits=teacher_logits, teacher_lse=teacher_lse)

    def call(h, w, b, train):
        return distill_forward(h, w, teacher_ids, teacher_logits, alpha, b, temperature=temperature,
                               teacher_lse=teacher_lse, train=train, keep_logits=keep_logits)

    (loss,) = _apply(hidden, weight, bias, call)
    return _reduce(loss, reduction, lambda: ((teacher_ids >= 0) & (teacher_ids < weight.shape[0])
                                             & (teacher_logits != -torch.inf)).any(1))


def policy_loss(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, advantage: torch.Tensor,
                old_logp: torch.Tensor | None = None, ref_logp: torch.Tensor | None = None, alpha: float = 1.0, bias=None,
                *, temperature: float = 1.0, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                ignore_index: int = -100, keep_logits: bool | None = None, reduction: str = "mean",
                return_logp: bool = False):
    """Differentiable policy_forward. reduction: "none" (fp32 [M]), "sum", or
    "mean" over the rows that are not left out. With return_logp also the tokens'
    log-probabilities [M], without a gradient (for the ratio's and the KL's
    statistics)."""
    _check_reduction(reduction)
    _check_constants(advantage=advantage, old_logp=old_logp, ref_logp=ref_logp)

    def call(h, w, b, train):
        return policy_forward(h, w, target, advantage, old_logp, ref_logp, alpha, b, temperature=temperature,
                              clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef, ignore_index=ignore_index,
                              train=train, keep_logits=keep_logits)

    loss, logp = _apply(hidden, weight, bias, call)
    loss = _reduce(loss, reduction, lambda: (target != ignore_index) & (target >= 0) & (target < weight.shape[0]))
    return (loss, logp) if return_logp else loss


def preference_loss(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, starts: torch.Tensor,
                    ref_logp: torch.Tensor | None = None, alpha: float = 1.0, bias=None, *, beta: float = 0.1,
                    margin: float = 0.0, label_smoothing: float = 0.0, average: bool = False, temperature: float = 1.0,
                    ignore_index: int = -100, keep_logits: bool | None = None, reduction: str = "mean",
                    return_logp: bool = False):
    """Differentiable preference_forward. reduction: "none" (fp32 [P]), "sum",
    or "mean" over the pairs. With return_logp also the sequences'
    log-probabilities [2 P], without a gradient (for the implicit rewards)."""
    _check_reduction(reduction)
    _check_constants(ref_logp=ref_logp)

    def call(h, w, b, train):
        return preference_forward(h, w, target, starts, ref_logp, alpha, b, beta=beta, margin=margin,
                                  label_smoothing=label_smoothing, average=average, temperature=temperature,
                                  ignore_index=ignore_index, train=train, keep_logits=keep_logits)

    loss, logp = _apply(hidden, weight, bias, call)
    loss = _reduce(loss, reduction, lambda: torch.ones_like(loss))
    return (loss, logp) if return_logp else loss
