"""Distillation from a teacher's top logits in float64 (torch on the CPU), from
the definition alone: the loss as a function of the logits, and its gradient
with the teacher's masses as they are, whatever they add up to."""
import math

import torch

F64 = torch.float64
NAN = math.nan


def masses(V, l, idx, tau, lse):
    """Per row: (tokens, p, log p) of the entries that are there, or None for a
    row without teacher weight."""
    at = [j for j, v in enumerate(idx.tolist()) if 0 <= v < V]
    v, x = idx[at].long(), l[at].to(F64) / tau
    if lse is not None:
        logp = torch.where(x < math.inf, x, NAN) - float(lse)
        return v, logp.exp(), logp
    if not len(at) or bool((x == -math.inf).all()):
        return None
    logp = x - torch.logsumexp(x, 0) if bool((x < math.inf).all()) else x * NAN
    return v, logp.exp(), logp


def distill_row(z, l, idx, tau, lse=None):
    """(loss, gradient [V], size [V]) of a row of weight 1; size is the sum of
    the magnitudes that a gradient element is the difference of, the teacher's
    rest counted as 2^-6 larger (it is 1 less a sum, so a relative error e of
    that sum is one of up to e / rest in it)."""
    V, x = z.shape[0], z.to(F64) / tau
    rows = masses(V, l, idx, tau, lse)
    if rows is None:
        return 0.0, torch.zeros(V, dtype=F64), torch.zeros(V, dtype=F64)
    v, p, logp = rows
    bad = bool(torch.isnan(x).any() or (x == math.inf).any() or (x == -math.inf).all())
    if bad or bool(torch.isnan(p).any()):
        return NAN, torch.full((V,), NAN, dtype=F64), torch.full((V,), NAN, dtype=F64)
    logz = torch.logsumexp(x, 0)
    used = p > 0
    kl = float((p[used] * (logp[used] - (x[v[used]] - logz))).sum())
    mass = float(p.sum())
    take = torch.zeros(V, dtype=F64).index_add_(0, v, p)
    slack = torch.zeros(V, dtype=F64)
    if lse is not None:
        free = torch.ones(V, dtype=torch.bool)
        free[v] = False
        pr = max(0.0, 1.0 - mass)
        if bool((x[free] > -math.inf).any()):
            logr = torch.logsumexp(x[free], 0)  # log of the unlisted part of the sum
            kl += pr * (math.log(pr) - float(logr - logz)) if pr > 0 else 0.0
            mass += pr
            take[free] += pr * (x[free] - logr).exp()
            slack[free] = 2.0 ** -6 * (x[free] - logr).exp()
    q = (x - logz).exp()
    return tau * tau * kl, tau * (mass * q - take), tau * (mass * q + take + slack)


def distill(Z, l, idx, tau, lse=None, weight=None, dloss=None):
    """(loss [T], dZ [T, V], size [T, V])."""
    T = Z.shape[0]
    out = [distill_row(Z[t], l[t], idx[t], tau, None if lse is None else lse[t])
           for t in range(T)]
    w = torch.ones(T, dtype=F64) if weight is None else weight.to(F64)
    g = w if dloss is None else w * dloss.to(F64)
    loss = torch.tensor([o[0] for o in out], dtype=F64) * w
    dZ, size = (torch.stack([o[i] for o in out]) * g[:, None] for i in (1, 2))
    for t in (w == 0).nonzero()[:, 0]:
        loss[t] = 0.0
    for t in (g == 0).nonzero()[:, 0]:
        dZ[t] = size[t] = 0.0
    return loss, dZ, size.abs()
