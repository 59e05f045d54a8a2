"""The losses of losses.hip and their gradients in float64, from the formulas,
with bounds on what the kernels may be off (test helper).

u = 2^-24. Of a row: T bounds a logit's error, E a sum of exponentials' relative
error, as tests/test_gpu_xent.py derives them (T twice over here: alpha and the bias
are divided by the temperature and rounded once more).
  log q    (t - largest) - log s: the errors of t and of the largest (T each), of
           the sum (E), and three roundings of values up to |t - largest| + |log s|
  exp, expm1, log of the device library: 2 u of the result each
  c        from the derivative of its formula, term by term below
  G = a q - S (a: the coefficient of q, S: what the target or the entries take off):
           a's and S's errors, q's (2 T + 2 E + 4 u |lse| and the argument's
           roundings), then the rounding to 16 bits
  grads    as in tests/test_gpu_xent.py
"""
import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


class Head:
    """t, lse and log q of a head, and their bounds."""

    def __init__(self, h, W, b, alpha, T):
        self.h, self.W, self.b, self.k = h.double(), W.double(), b, alpha / T
        self.T_, self.type = T, h.dtype
        t = self.h @ self.W.t() * self.k
        A = self.h.abs() @ self.W.abs().t() * abs(self.k)
        if b is not None:
            t = t + b.double() / T
        # a column more than 1000 below the row's largest (masked by the type's lowest
        # value) has e^-1000 = 0 in fp32 and in the sums here, whatever its own error:
        # it is left out of the row's bounds, and an exponential that is not 0 has an
        # argument above -104
        finite = torch.where(t.isinf() | (t < t.amax(1, keepdim=True) - 1000), torch.zeros_like(t), t)
        size = A + torch.where(finite == 0, finite, (b.double().abs().nan_to_num(0, 0, 0) / T)[None]) if b is not None else A
        self.t = t
        self.T = (2e-5 * A + 2 * U * finite.abs() + 4 * U * size).amax(1)
        self.mx = t.amax(1)
        self.mz = torch.where(self.mx.isinf(), torch.zeros_like(self.mx), self.mx)
        s = torch.exp(t - self.mz[:, None]).sum(1)
        self.ls = torch.log(s)
        self.lse = self.ls + self.mz
        self.x = torch.where(t.isinf(), torch.zeros_like(t), t - self.mz[:, None]).abs()
        tiles = (W.shape[0] + 255) // 256
        self.E = 2 * U * self.x.clamp(max=104).amax(1) + (22 + 3 * (tiles // 16 + 18)) * U + self.T
        self.logq = torch.where(t == -math.inf, t, t - self.lse[:, None])
        self.q = torch.where(self.lse[:, None].isinf(), torch.zeros_like(t),
                             torch.exp(t - torch.where(self.lse.isinf(), 0 * self.lse, self.lse)[:, None]))
        self.dlogq = (2 * self.T + self.E)[:, None] + 4 * U * (self.x + self.ls.abs().nan_to_num(0, 0, 0)[:, None])
        # where q is not 0 (above)
        self.dq = self.q * ((2 * self.T + 2 * self.E + 4 * U * self.lse.abs().nan_to_num(0, 0, 0))[:, None]
                            + 4 * U * (1 + self.x.clamp(max=104) + finite.abs())) + TINY

    def gradients(self, a, S, da, dS, largest):
        """{name: (value, bound before its own rounding)} of G = a q - S; da, dS:
        the errors of a [M] and S [M, V]; largest: the largest |coefficient|."""
        a, da = a[:, None], da[:, None]
        G = a * self.q - S
        d32 = a.abs() * self.dq + da * (self.q + self.dq) + dS + 3 * U * (a.abs() * self.q + S.abs()) + 2 * largest * TINY
        h16 = torch.finfo(self.type).eps / 2
        d = d32 + h16 * (G.abs() + d32)
        if self.type == torch.float16:
            d = d + largest * 2.0 ** -38
        Gm, k = G.abs() + d, abs(self.k)
        M, V = G.shape
        out = dict(hidden=(self.k * (G @ self.W), k * (d @ self.W.abs() + 2e-5 * (Gm @ self.W.abs()) + largest * V * TINY)),
                   weight=(self.k * (G.t() @ self.h),
                           k * (d.t() @ self.h.abs() + 2e-5 * (Gm.t() @ self.h.abs()) + largest * M * TINY)))
        # the entries' share is kept in whole numbers of 2^-30 (or finer) of the largest coefficient
        n = (S != 0).sum(0)
        out["bias"] = (G.sum(0) / self.T_, ((d32.sum(0) + (M + 12) * U * ((a * self.q).abs() + S.abs()).sum(0)
                                             + n * largest * 2.0 ** -31) / self.T_ + 2 * U * G.sum(0).abs()))
        return out


def distill(head, ids, logits, T, teacher_lse=None, grad=None):
    """(loss, bound, gradients or None)"""
    M, V = head.t.shape
    s = logits.double() / T
    there = (ids >= 0) & (ids < V) & (logits != -math.inf)
    s = torch.where(there, s, torch.full_like(s, -math.inf))
    at = torch.where(there, ids.long(), torch.zeros_like(ids.long()))
    n = torch.logsumexp(s, 1) if teacher_lse is None else teacher_lse.double()
    n = torch.where(there.any(1), n, torch.zeros_like(n))
    lp = s - n[:, None]
    p = torch.exp(lp)
    lq = head.logq.gather(1, at)
    term = torch.where(there & (p > 0), p * (lp - lq), torch.zeros_like(p))
    loss = term.sum(1)
    fine = torch.where(there, s, torch.zeros_like(s)).abs().amax(1, keepdim=True)
    # log p: s / T and n rounded, two differences, the log; p: exp of that
    dlp = U * (8 * fine + 6 * n.abs()[:, None] + 12) + (2e-7 if teacher_lse is None else 0.0) * U
    K = ids.shape[1]
    if teacher_lse is None:
        dlp = dlp + (K + 8) * U
    dp = p * (dlp + 3 * U) + TINY
    zero = torch.zeros_like(p)
    fin = lambda v: torch.where(there & (p > 0), v.nan_to_num(0, 0, 0), zero)
    bound = (fin(dp * (lp - lq).abs()) + fin(p * (dlp + head.dlogq.gather(1, at)))
             + (K / 32 + 80) * U * fin(p * (lp.abs() + lq.abs()))).sum(1) + TINY
    if grad is None:
        return loss, bound, None
    P = p.sum(1)
    dP = dp.sum(1) + (K + 8) * U * P
    if teacher_lse is None:
        P, dP = there.any(1).double(), torch.zeros_like(P)
    g = grad.double()
    S = torch.zeros_like(head.t).scatter_add_(1, at, p * g[:, None])
    dS = torch.zeros_like(head.t).scatter_add_(1, at, torch.where(there, dp * g.abs()[:, None], zero)) + (K + 2) * U * S.abs()
    largest = float(torch.maximum(g.abs() * P, g.abs()).amax())
    return loss, bound, head.gradients(g * P, S, g.abs() * dP + 2 * U * (g * P).abs(), dS, largest)


def _token(head, y, ignore):
    V = head.t.shape[1]
    keep = (y != ignore) & (y >= 0) & (y < V)
    at = torch.where(keep, y.long(), torch.zeros_like(y.long()))[:, None]
    zero = torch.zeros_like(head.lse)
    return keep, at, torch.where(keep, head.logq.gather(1, at)[:, 0], zero), torch.where(keep, head.dlogq.gather(1, at)[:, 0], zero)


def _token_gradients(head, keep, at, c, dc):
    c, dc = torch.where(keep, c, torch.zeros_like(c)), torch.where(keep, dc, torch.zeros_like(c))
    S = torch.zeros_like(head.t).scatter_add_(1, at, -c[:, None])
    dS = torch.zeros_like(head.t).scatter_add_(1, at, dc[:, None])
    return head.gradients(-c, S, dc, dS, float(c.abs().amax()))


def policy(head, y, A, old, ref, low, high, kl, ignore=-100, grad=None):
    """(loss, bound, logp, bound, gradients or None, ratio)"""
    keep, at, logp, dl = _token(head, y, ignore)
    A = A.double()
    lr = logp - old.double() if old is not None else torch.zeros_like(logp)
    r = torch.exp(lr)
    dr = r * (dl + 3 * U * (lr.abs() + 1)) if old is not None else torch.zeros_like(r)
    held = r.clamp(1 - low, 1 + high)
    free = r * A <= held * A
    pg = -torch.where(free, r * A, held * A)
    loss, bound = pg, A.abs() * torch.where(free, dr, torch.full_like(dr, 4 * U)) + 3 * U * pg.abs()
    c = torch.where(free, -r * A, torch.zeros_like(r))
    dc = torch.where(free, A.abs() * dr, torch.zeros_like(r)) + 2 * U * c.abs()
    # a ratio on a border may be taken for either side
    near = torch.minimum((r - (1 - low)).abs(), (r - (1 + high)).abs()) <= dr + 2 * U
    assert not bool((near & keep & (A != 0)).any()), "the inputs lie on a border"
    if ref is not None and kl:
        d = ref.double() - logp
        dd = dl + U * d.abs()
        e = torch.expm1(d)
        loss = loss + kl * (e - d)
        bound = bound + kl * (torch.expm1(dd) * torch.exp(d) + dd + 4 * U * (e.abs() + d.abs())) + 4 * U * loss.abs()
        c = c - kl * e
        dc = dc + kl * (torch.expm1(dd) * torch.exp(d) + 4 * U * e.abs()) + 2 * U * c.abs()
    zero = torch.zeros_like(loss)
    loss, bound = torch.where(keep, loss, zero), torch.where(keep, bound, zero)
    if grad is None:
        return loss, bound, logp, dl, None
    g = grad.double()
    return loss, bound, logp, dl, _token_gradients(head, keep, at, c * g, dc * g.abs() + 2 * U * (c * g).abs())


def preference(head, y, starts, ref, beta, margin, smoothing, average, ignore=-100, grad=None):
    """(loss, bound, logp, bound, gradients or None)"""
    keep, at, logp, dl = _token(head, y, ignore)
    s = starts.tolist()
    P = len(s) // 2
    n = [max(1, int(keep[a:b].sum())) if average else 1 for a, b in zip(s, s[1:])]
    S = torch.stack([logp[a:b].sum() / k for a, b, k in zip(s, s[1:], n)] + [logp.new_zeros(())])[:2 * P]
    dS = torch.stack([dl[a:b].sum() / k for a, b, k in zip(s, s[1:], n)] + [logp.new_zeros(())])[:2 * P] + 1e-12 * (1 + S.abs())
    lead = S - (ref.double() if ref is not None else 0.0)
    b32 = lambda v: float(torch.tensor(v, dtype=torch.float32))
    z = b32(beta) * (lead[:P] - lead[P:]) - b32(margin)
    dz = b32(beta) * (dS[:P] + dS[P:])
    e = b32(smoothing)
    sig = torch.nn.functional.logsigmoid
    loss = -(1 - e) * sig(z) - e * sig(-z)
    bound = dz + 2 * U * loss + 1e-12
    if grad is None:
        return loss, bound, S, dS + U * S.abs(), None
    w = e - torch.sigmoid(-z)
    c = torch.zeros_like(logp)
    dc = torch.zeros_like(logp)
    g = grad.double()
    for i, (a, b) in enumerate(zip(s, s[1:])):
        p, sign = i % P, 1.0 if i < P else -1.0
        c[a:b] = sign * w[p] * b32(beta) / n[i] * g[p]
        dc[a:b] = (dz[p] * b32(beta) / n[i] + U * (w[p] * b32(beta) / n[i]).abs() + TINY) * g[p].abs() + 2 * U * c[a:b].abs()
    return loss, bound, S, dS + U * S.abs(), _token_gradients(head, keep, at, c, dc)
