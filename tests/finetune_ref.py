"""Plain float64 references of the fine-tuning operators (torch on the CPU),
written from their formulas and sharing nothing with the HIP path."""
import math

import torch

F64 = torch.float64
GROUP = 128
C, B = math.sqrt(2.0 / math.pi), 0.044715


def dense(S, A):
    """W_hat [m, n] of signs [K, m, n] and scales [K, m, n/128] (numpy or torch)."""
    S, A = torch.as_tensor(S).to(F64), torch.as_tensor(A).to(F64)
    return (S * A.repeat_interleave(GROUP, dim=2)).sum(0)


def half_tanh(g):
    """(1 + tanh y) / 2 = 1 / (1 + exp(-2 y)), y = C (g + B g^3): the second
    form, since 1 + tanh y keeps no digit below 2^-53."""
    return 1 / (1 + torch.exp(-2 * C * (g + B * g ** 3)))


def act(kind, g):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    return g * half_tanh(g)


def act_slope(kind, g):
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    s = half_tanh(g)
    return s + g * 2 * s * (1 - s) * C * (1 + 3 * B * g * g)


def stacked_rows(m):
    return 16 * ((m + 7) // 8)


def stack_index(m):
    """Stacked columns of the gate and the up values of outputs 0 .. m - 1."""
    i = torch.arange(m)
    gate = 16 * (i // 8) + i % 8
    return gate, gate + 8


def stack(g, u):
    out = torch.zeros(g.shape[0], stacked_rows(g.shape[1]), dtype=g.dtype)
    ig, iu = stack_index(g.shape[1])
    out[:, ig], out[:, iu] = g, u
    return out


def scale_grad(S, dY, X):
    S = torch.as_tensor(S).to(F64)
    K, m, n = S.shape
    dW = dY.to(F64).t() @ X.to(F64)
    return (S * dW).view(K, m, n // GROUP, GROUP).sum(-1)


def distill(Z, l, idx, tau, lse=None, weight=None):
    """(loss [T], dZ [T, V]) row by row, entry by entry."""
    Z, l = Z.to(F64), l.to(F64)
    T, V = Z.shape
    loss, dZ = torch.zeros(T, dtype=F64), torch.zeros(T, V, dtype=F64)
    for t in range(T):
        w = 1.0 if weight is None else float(weight[t])
        if w == 0.0:
            continue
        logq = torch.log_softmax(Z[t] / tau, 0)
        q = logq.exp()
        entries = [(int(v), float(x) / tau) for v, x in zip(idx[t], l[t]) if 0 <= int(v) < V]
        if lse is None:
            logs = torch.tensor([x for _, x in entries], dtype=F64)
            if not len(entries) or float(logs.max()) == -math.inf:
                continue  # no teacher weight
            logp = logs - torch.logsumexp(logs, 0)
        else:
            logp = torch.tensor([x for _, x in entries], dtype=F64) - float(lse[t])
        p = logp.exp()
        kl, grad = 0.0, q.clone()
        for (v, _), pj, lpj in zip(entries, p.tolist(), logp.tolist()):
            if pj > 0:
                kl += pj * (lpj - float(logq[v]))
            grad[v] -= pj
        if lse is not None:
            free = torch.ones(V, dtype=torch.bool)
            free[[v for v, _ in entries]] = False
            pr, qr = max(0.0, 1.0 - float(p.sum())), float(q[free].sum())
            if pr > 0 and qr > 0:
                kl += pr * math.log(pr / qr)
                grad[free] -= q[free] * (pr / qr)
        loss[t] = w * tau * tau * kl
        dZ[t] = w * tau * grad
    return loss, dZ
