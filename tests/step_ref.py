"""Plain float64 references of the layer with its epilogue, the policy and
preference losses and the optimizer step (torch on the CPU), written from
their formulas and sharing nothing with the HIP path."""
import math

import numpy as np
import torch

import finetune_ref as ref

F64 = torch.float64
BLOCK = 256


def act(kind, z):
    return z if kind == "none" else ref.act(kind, z)


def act_slope(kind, z):
    return torch.ones_like(z) if kind == "none" else ref.act_slope(kind, z)


def linear(W, X, bias=None, kind="none", residual=None):
    """(Y, z)"""
    z = X.to(F64) @ W.t()
    if bias is not None:
        z = z + bias.to(F64)
    y = act(kind, z)
    return (y if residual is None else residual.to(F64) + y), z


def logp(Z, label, tau):
    """(log-probabilities [T], softmax [T, V]); 0 where there is no token."""
    logq = torch.log_softmax(Z.to(F64) / tau, -1)
    out = torch.zeros(Z.shape[0], dtype=F64)
    for t, a in enumerate(label.tolist()):
        if 0 <= a < Z.shape[1]:
            out[t] = logq[t, a]
    return out, logq.exp()


def onehot(label, V):
    out = torch.zeros(len(label), V, dtype=F64)
    for t, a in enumerate(label.tolist()):
        if 0 <= a < V:
            out[t, a] = 1.0
    return out


def logp_grad(Z, label, tau, dlogp):
    V = Z.shape[1]
    _, q = logp(Z, label, tau)
    there = ((label >= 0) & (label < V)).to(F64)
    return (onehot(label, V) - q) * (there * dlogp.to(F64) / tau)[:, None]


def policy(lp, label, V, A, old=None, ref_lp=None, w=None, low=0.2, high=0.2, kl=0.0):
    """(loss, dlogp, size of the slope's terms) from log-probabilities [T]."""
    T = len(lp)
    loss, slope, size = (torch.zeros(T, dtype=F64) for _ in range(3))
    for t in range(T):
        wt = 1.0 if w is None else float(w[t])
        if not 0 <= int(label[t]) < V or wt == 0.0:
            continue
        l, a = float(lp[t]), float(A[t])
        r = math.exp(l - float(old[t])) if old is not None else 1.0
        cut = min(max(r, 1 - low), 1 + high)
        if a != 0.0:
            loss[t] = -min(r * a, cut * a)
            if not (r > 1 + high if a > 0 else r < 1 - low):
                slope[t] = -r * a
        size[t] = abs(r * a)
        if ref_lp is not None:
            x = float(ref_lp[t]) - l
            loss[t] += kl * (math.expm1(x) - x)
            slope[t] -= kl * math.expm1(x)
            size[t] += kl * (math.exp(x) + 1)
        loss[t] *= wt
        slope[t] *= wt
        size[t] *= abs(wt)
    return loss, slope, size


def preference(lp, offsets, label=None, ref_lp=None, w=None, beta=0.1, smoothing=0.0, margin=0.0,
               mean=False, V=1 << 30):
    """(loss [pairs], dlogp [T]; NaN in rows outside every sequence)"""
    T, pairs = len(lp), len(offsets) // 2
    counted = torch.ones(T, dtype=torch.bool) if label is None else (label >= 0) & (label < V)
    diff = lp.to(F64) - (0 if ref_lp is None else ref_lp.to(F64))
    dlogp, loss = torch.full((T,), math.nan, dtype=F64), torch.zeros(pairs, dtype=F64)
    for p in range(pairs):
        rows, size, score = [], [], []
        for s in (2 * p, 2 * p + 1):
            r = torch.arange(int(offsets[s]), int(offsets[s + 1]))
            live = r[counted[r]]
            size.append(max(1, len(live)) if mean else 1)
            score.append(float(diff[live].sum()) / size[-1])
            rows.append((r, live))
        h = beta * (score[0] - score[1]) - margin
        wp = 1.0 if w is None else float(w[p])
        sig = 1 / (1 + math.exp(-h))
        loss[p] = wp * ((1 - smoothing) * math.log1p(math.exp(-h)) +
                        smoothing * math.log1p(math.exp(h)))
        dh = wp * beta * (smoothing * sig - (1 - smoothing) * (1 - sig))
        for sign, (r, live), n in zip((1, -1), rows, size):
            dlogp[r] = 0.0
            dlogp[live] = sign * dh / n
    return loss, dlogp


def adamw(p, g, m, v, t, lr, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, c=1.0):
    """(p, m, v) after one step, in float64."""
    p, g, m, v = (x.to(F64) for x in (p, g, m, v))
    g = g * c
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** t), v / (1 - b2 ** t)
    return p * (1 - lr * wd) - lr * mh / (vh.sqrt() + eps), m, v


def packed_scales(p, d):
    """The scales of param [K, m, G] in the packed order [RB, G, K, 64]; NaN in the
    padding."""
    K, m, G = d.K, d.m, d.n // 128
    rb = (m + 63) // 64
    x = torch.full((K, rb * 64, G), math.nan, dtype=p.dtype)
    x[:, :m] = p.view(K, m, G)
    return x.view(K, rb, 64, G).permute(1, 3, 0, 2).contiguous()


# ------------------------------------------------ the 8-bit states, bit for bit

def e4m3_values():
    """Value of each of the 256 codes (NaN codes included)."""
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(F64)


def random_bits(count, tensor, step, seed):
    """The two 16-bit random numbers of each value, from the documented hash's
    definition: 32-bit wrapping arithmetic on (index, tensor, step, seed)."""
    u = np.uint32
    with np.errstate(over="ignore"):
        key = u(seed & 0xffffffff) + u(step & 0xffffffff) * u(0x9E3779B1) + \
            u(tensor) * u(0x6A09E667)
        h = np.arange(count, dtype=np.uint64).astype(u) * u(0xBB67AE85) + key
        h = (h ^ (h >> u(16))) * u(0x3C6EF373)
        h = (h ^ (h >> u(15))) * u(0xA54FF53B)
        h = h ^ (h >> u(16))
    return h & u(0xffff), h >> u(16)


def encode(x, rnd, least):
    """float32 values -> (codes uint8, scales float32): stochastic rounding to e4m3
    with one power-of-two scale per block, by integer arithmetic on multiples of the
    local step."""
    n = len(x)
    blocks = (n + BLOCK - 1) // BLOCK
    codes, scales = np.zeros(n, np.uint8), np.zeros(blocks, np.float32)
    for b in range(blocks):
        at = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        v = np.abs(x[at]).astype(np.float64)
        if not np.isfinite(v).all():
            scales[b] = np.nan
            continue
        top = v.max()
        e = max(int(np.floor(np.log2(top))) if top > 0 else -80, -80) - 7
        scales[b] = np.float32(2.0 ** e)
        y = v * 2.0 ** -e  # exact, in [0, 256)
        u = (rnd[at].astype(np.float64) * 16 + 8) * 2.0 ** -20
        ye = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
        step = 2.0 ** (ye - 3)
        k = np.floor(y / step + u)  # 8 .. 16 (normal), 0 .. 8 below 2^-6
        c = np.where(y >= 2.0 ** -6, (ye + 7) * 8 + (k - 8), k).astype(np.int64)
        c = np.where((y > 0) & (c < least), least, c)
        codes[at] = (c | np.where(x[at] < 0, 128, 0)).astype(np.uint8)
    return codes, scales
