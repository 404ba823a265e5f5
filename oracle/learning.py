"""Plain 64-bit forms of the operators that a drafter learns with
(``include/sel.h``): cross entropy through an output head with its gradient, and
the divergence from a teacher's top logits with its gradient. Inputs are torch
tensors of any device whose values are taken as they are; written from the
definitions, with no code of the kernels."""
from __future__ import annotations

import math

import torch

INF = float("inf")


def _in_vocabulary(ids, V):
    """ids as int64, -1 for those that name no column."""
    ids = ids.to(torch.int64)
    return torch.where((ids >= 0) & (ids < V), ids, -1)


def head_loss(x, w, targets):
    """(loss, lse) of hidden rows x [n, H] through w [V, H]. The loss of a row is
    ln(1 + sum over the other ids of exp(z - z_target)), 0 where the target names
    no id."""
    z = x.double() @ w.double().T
    t = _in_vocabulary(targets, w.shape[0])
    lse = torch.logsumexp(z, dim=1)
    rows = torch.arange(len(t), device=z.device)
    at = z[rows, t.clamp(min=0)]
    others = z.clone()
    others[rows, t.clamp(min=0)] = -INF
    d = torch.logsumexp(others, dim=1) - at
    loss = torch.where(d > 30, d + torch.exp(-d), torch.log1p(torch.exp(d)))
    return torch.where(t >= 0, loss, 0.0), lse


def head_loss_grad(x, w, targets, lse, grad):
    """(hidden gradient, weight gradient) of sum of grad * loss; rows whose target
    names no id or whose grad is 0 count for nothing."""
    x64, w64 = x.double(), w.double()
    t = _in_vocabulary(targets, w.shape[0])
    live = torch.nonzero((t >= 0) & (grad != 0))[:, 0]
    p = torch.exp(x64[live] @ w64.T - lse[live].double()[:, None])
    p[torch.arange(len(live), device=p.device), t[live]] -= 1.0
    p = p * grad[live].double()[:, None]
    dx = torch.zeros_like(x64)
    dx[live] = p @ w64
    return dx, p.T @ x64[live]


def distill(x, vals, ids, teacher_lse, temperature, grad=None):
    """loss [n] of logits rows x [n, V] against a teacher's lists, and with `grad`
    [n] also the gradient of sum of grad * loss as to x."""
    n, V = x.shape
    T = torch.tensor(temperature, dtype=torch.float32).double().item()  # the value that a call hands over
    lq = torch.log_softmax(x.double() / T, dim=1)
    q = lq.exp()
    at = _in_vocabulary(ids, V)
    loss = torch.zeros(n, dtype=torch.float64, device=x.device)
    out = torch.zeros((n, V), dtype=torch.float64, device=x.device)
    for r in range(n):
        e = torch.nonzero(at[r] >= 0)[:, 0]
        i, v = at[r, e], vals[r, e].double() / T
        if not len(i) or (v == -INF).all():
            continue
        g = 1.0 if grad is None else grad[r].double()
        L = torch.logsumexp(v, dim=0) if teacher_lse is None else teacher_lse[r].double()
        lp = v - L
        p = lp.exp()
        if len(i.unique()) < len(i) or not torch.isfinite(L) or (v == INF).any() or torch.isnan(lq[r]).any():
            loss[r] = float("nan")
            out[r] = float("nan")
        else:
            some = p > 0
            loss[r] = (p[some] * (lp[some] - lq[r, i[some]])).sum()
            listed = torch.zeros(V, dtype=torch.bool, device=x.device)
            listed[i] = True
            left = torch.zeros((), dtype=torch.float64, device=x.device)
            if teacher_lse is not None and len(i) < V:
                left = (1.0 - p.sum()).clamp(min=0.0)
                # an r no larger than the rounding of a 32-bit lse, with nothing left for it
                nothing = -126 * math.log(2.0)
                if left <= 2.0 ** -21 * max(1.0, abs(L.item())):
                    if (lp < nothing).any() or torch.logsumexp(lq[r, ~listed], dim=0) < nothing:
                        left = torch.zeros_like(left)
            m = p.sum() + left
            d = m * q[r]
            d[i] -= p
            if left > 0:
                # in logarithms, and each id's share of s from the logits: s may lie below
                # every 64-bit number
                ln_s = torch.logsumexp(lq[r, ~listed], dim=0)
                loss[r] += left * (torch.log(left) - ln_s)
                share = torch.softmax(x[r, ~listed].double() / T, dim=0)
                d[~listed] = d[~listed] - left * share if ln_s > -INF else 0.0
            out[r] = g / T * d
        if grad is not None and g == 0:
            out[r] = 0.0
    return loss if grad is None else (loss, out)
