"""Workloads of the Boolean-kernel fine-tuning operators, for measurement.

Five operators on a weight kept as K Boolean kernels with group scales
(W_hat = sum_k alpha_k (.) B_k, one alpha per output row and 128 columns):

  gated      H = act(X Wg^T) (.) (X Wu^T): the gated feed-forward block, one
             token up to a training batch, optionally keeping the
             pre-activations for the backward pass
  gated_bwd  the block's backward: gradients of the pre-activations and of X
  gemmt      dX = dY W_hat for T tokens: the activation gradient of one layer
  scale_grad d loss / d alpha = sum over a group's columns of B_k (.) (dY^T X)
  distill    KL divergence from a teacher's top logits, with its gradient

Each is given twice: `run` with own = False computes the formula in plain
32-bit torch operations; with own = True it calls the package.  `exact` is
the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128
F64 = torch.float64


# ----------------------------------------------------------------- the cases

def listed():
    mlp = dict(m=11008, n=4096, K=3, scales="f16", act="silu")
    down = dict(m=4096, n=11008, K=3, scales="f16")
    return [
        # the LLaMA-7B-shaped MLP's gate|up for one decoded token
        dict(name="gated 1 token", op="gated", T=1, keep=False, **mlp),
        # the same for a small serving batch
        dict(name="gated 16 tokens", op="gated", T=16, keep=False, **mlp),
        # the forward of a training step: the pre-activations are kept
        dict(name="gated 2048 tokens", op="gated", T=2048, keep=True, **mlp),
        # its backward
        dict(name="gated_bwd 2048 tokens", op="gated_bwd", T=2048, **mlp),
        # backward of a small block: odd token count, a hidden width that is
        # no multiple of a tile, fp32 scales, the other activation
        dict(name="gated_bwd 37 tokens", op="gated_bwd", T=37, m=1001, n=640, K=2, scales="f32",
             act="gelu"),
        # activation gradient of the down projection in a training step
        dict(name="gemmt 2048 tokens", op="gemmt", T=2048, **down),
        # a short sequence through a 13B-shaped attention projection
        dict(name="gemmt 16 tokens", op="gemmt", T=16, m=5120, n=5120, K=3, scales="f16"),
        # scale gradients of the down projection in a training step
        dict(name="scale_grad 2048 tokens", op="scale_grad", T=2048, **down),
        # the smallest layer of the workloads, a few tokens: latency
        dict(name="scale_grad 33 tokens", op="scale_grad", T=33, m=256, n=512, K=2, scales="f32"),
        # the loss of a training step, loss and gradient in one call
        dict(name="distill step 2048 rows", op="distill", mode="step", T=2048, V=32000, top=64,
             z="bf16", rest=False, tau=2.0),
        # loss and gradient as two calls, fp32 logits of an odd vocabulary,
        # the teacher's remaining mass kept as one class
        dict(name="distill pair 301 rows", op="distill", mode="pair", T=301, V=12345, top=20,
             z="f32", rest=True, tau=1.0),
        # the loss of one row alone (evaluation): latency
        dict(name="distill loss 1 row", op="distill", mode="loss", T=1, V=32000, top=16, z="bf16",
             rest=False, tau=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated_bwd", "gemmt", "scale_grad", "distill"])
    if op == "distill":
        V = _log_int(rng, 500, 32000)
        return dict(op=op, mode=rng.choice(["step", "pair", "loss"]), T=_log_int(rng, 1, 2048),
                    V=V, top=_log_int(rng, 1, 128), z=rng.choice(["bf16", "f16", "f32"]),
                    rest=rng.random() < 0.5, tau=rng.choice([1.0, 2.0, 4.0]))
    n = GROUP * _log_int(rng, 1, 86)
    m = _log_int(rng, 8, 11008)
    most = 11008 * 4096 * 2048
    T = _log_int(rng, 1, min(2048, max(1, most // (m * n))))
    case = dict(op=op, T=T, m=m, n=n, K=rng.choice([1, 2, 3, 4]),
                scales=rng.choice(["f16", "f32"]))
    if op in ("gated", "gated_bwd"):
        case["act"] = rng.choice(["silu", "gelu"])
    if op == "gated":
        case["keep"] = rng.random() < 0.5
    return case


def work(case):
    T = case["T"]
    if case["op"] == "distill":
        zb = 4 if case["z"] == "f32" else 2
        row = case["V"] * zb
        passes = {"loss": 1, "step": 2, "pair": 3}[case["mode"]]
        return {"bytes": T * (passes * row + case["top"] * 8 + 16), "flops": 0}
    m, n, K = case["m"], case["n"], case["K"]
    sb = 2 if case["scales"] == "f16" else 4
    weights = K * m * n // 8 + K * m * (n // GROUP) * sb
    if case["op"] == "gated":
        out = T * m * 2 * (3 if case["keep"] else 1)
        return {"bytes": 2 * weights + T * n * 2 + out, "flops": 4 * T * m * n}
    if case["op"] == "gated_bwd":
        return {"bytes": 2 * weights + T * m * 2 * 5 + T * n * 2, "flops": 4 * T * m * n}
    if case["op"] == "gemmt":
        return {"bytes": weights + T * m * 2 + T * n * 2, "flops": 2 * T * m * n}
    return {"bytes": K * m * n // 8 + T * (m + n) * 2 + K * m * (n // GROUP) * 4,
            "flops": 2 * T * m * n}


# ---------------------------------------------------------------- the inputs

def _greedy(W, K, scales):
    """K kernels and scales of W by successive sign and mean magnitude."""
    m, n = W.shape
    dt = torch.float16 if scales == "f16" else torch.float32
    R, S, A = W.clone(), [], []
    for _ in range(K):
        s = torch.where(R >= 0, 1.0, -1.0)
        a = R.abs().view(m, n // GROUP, GROUP).mean(-1).to(dt)
        R -= (s.view(m, n // GROUP, GROUP) * a.float()[..., None]).view(m, n)
        S.append(s.to(torch.int8))
        A.append(a)
    return torch.stack(S).contiguous(), torch.stack(A).contiguous()


def _layer(case, gen, count):
    out = []
    for _ in range(count):
        W = torch.randn(case["m"], case["n"], generator=gen, device=DEV) * 0.02
        out.append(_greedy(W, case["K"], case["scales"]))
    return out


def _bf16(gen, rows, cols, scale=1.0):
    return (torch.randn(rows, cols, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def _inputs(case, seed):
    """The case's data, from the seed alone."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 13)
    T, s = case["T"], dict(case=case)
    if case["op"] == "distill":
        return _distill_inputs(case, gen)
    m, n = case["m"], case["n"]
    if case["op"] in ("gated", "gated_bwd"):
        s["gate"], s["up"] = _layer(case, gen, 2)
        if case["op"] == "gated":
            s["X"] = _bf16(gen, T, n)
        else:
            # pre-activations of unit-variance inputs have a spread of about 1.3
            s["pre"] = _bf16(gen, T, _stacked_rows(m), 1.3)
            s["dH"] = _bf16(gen, T, m, 0.01)
    else:
        s["layer"], = _layer(case, gen, 1)
        s["dY"] = _bf16(gen, T, m, 0.01)
        if case["op"] == "scale_grad":
            s["X"] = _bf16(gen, T, n)
    return s


def _distill_inputs(case, gen):
    """Teacher logits with a few likely tokens per row, a student near the
    teacher; some rows list fewer entries (index -1), one in ten is a prompt
    row of weight 0."""
    T, V, top = case["T"], case["V"], min(case["top"], case["V"])
    zt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[case["z"]]
    teacher = torch.randn(T, V, generator=gen, device=DEV) * 2.5
    Z = (teacher + 0.8 * torch.randn(T, V, generator=gen, device=DEV)).to(zt)
    val, idx = teacher.topk(top, dim=-1)
    lse = torch.logsumexp(teacher / case["tau"], -1)
    del teacher
    listed_n = torch.randint(1, top + 1, (T, 1), generator=gen, device=DEV)
    short = torch.rand(T, 1, generator=gen, device=DEV) < 0.2
    drop = short & (torch.arange(top, device=DEV)[None] >= listed_n)
    idx = torch.where(drop, -1, idx).to(torch.int32).contiguous()
    # mean over the rows; fp16 gradients under a loss scale, as they are kept
    mean = (4096.0 if case["z"] == "f16" else 1.0) / T
    weight = (torch.rand(T, generator=gen, device=DEV) >= 0.1).float() * mean
    weight[0] = mean
    dloss = 0.5 + torch.rand(T, generator=gen, device=DEV)
    return dict(case=case, Z=Z, val=val.contiguous(), idx=idx, lse=lse if case["rest"] else None,
                weight=weight, dloss=dloss)


def _stacked_rows(m):
    return 16 * ((m + 7) // 8)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(case, s)
    return s


# ----------------------------------------------- the package's own operators

def _prepare_own(case, s):
    """What a program keeps: the packed layer, output buffers, workspaces."""
    import boolean_weight_amd as bw
    T = case["T"]
    bf = dict(dtype=torch.bfloat16, device=DEV)
    if case["op"] == "distill":
        s["d"] = bw.mbok_distill_desc_init(case["V"], s["idx"].shape[1], case["tau"])
        s["loss"] = torch.empty(T, device=DEV)
        s["stats"] = torch.empty(T, bw.MBOK_DISTILL_STATS, device=DEV)
        s["dZ"] = torch.empty_like(s["Z"])
        return
    m, n = case["m"], case["n"]
    dt = bw.MBOK_F16 if case["scales"] == "f16" else bw.MBOK_F32
    s["d"] = d = bw.mbok_desc_init(m, n, case["K"], dt)
    if case["op"] in ("gated", "gated_bwd"):
        d2 = bw.mbok_gated_stack(d)
        s["packed"] = torch.empty(bw.mbok_packed_bytes(d2), dtype=torch.uint8, device=DEV)
        bw.mbok_gated_pack(d, *s.pop("gate"), *s.pop("up"), s["packed"])
        if case["op"] == "gated":
            s["H"] = torch.empty(T, m, **bf)
            s["keep"] = torch.empty(T, d2.m, **bf) if case["keep"] else None
        else:
            s["dpre"] = torch.empty(T, d2.m, **bf)
            s["dX"] = torch.empty(T, n, **bf)
        return
    s["packed"] = torch.empty(bw.mbok_packed_bytes(d), dtype=torch.uint8, device=DEV)
    bw.mbok_pack(d, *s.pop("layer"), s["packed"])
    if case["op"] == "gemmt":
        s["dX"] = torch.empty(T, n, **bf)
    else:
        s["dalpha"] = torch.empty(case["K"], m, n // GROUP, device=DEV)


def _run_own(case, s):
    import boolean_weight_amd as bw
    if case["op"] == "distill":
        more = dict(t_lse=s["lse"], weight=s["weight"])
        if case["mode"] == "loss":
            bw.mbok_distill(s["d"], s["Z"], s["val"], s["idx"], s["loss"], **more)
            return [s["loss"]]
        if case["mode"] == "step":
            bw.mbok_distill(s["d"], s["Z"], s["val"], s["idx"], s["loss"], dZ=s["dZ"], **more)
        else:
            bw.mbok_distill(s["d"], s["Z"], s["val"], s["idx"], s["loss"], stats=s["stats"],
                            **more)
            bw.mbok_distill_backward(s["d"], s["Z"], s["val"], s["idx"], s["stats"], s["dloss"],
                                     s["dZ"], **more)
        return [s["loss"], s["dZ"]]
    if case["op"] == "gemmt":
        bw.mbok_gemmt(s["d"], s["packed"], s["dY"], s["dX"])
        return [s["dX"]]
    if case["op"] == "scale_grad":
        bw.mbok_scale_grad(s["d"], s["packed"], s["dY"], s["X"], s["dalpha"])
        return [s["dalpha"]]
    act = bw.MBOK_ACT_SILU if case["act"] == "silu" else bw.MBOK_ACT_GELU
    if case["op"] == "gated":
        bw.mbok_gated(s["d"], s["packed"], s["X"], s["H"], pre=s["keep"], act=act)
        return [s["H"]] + ([s["keep"]] if case["keep"] else [])
    bw.mbok_gated_backward(s["d"], s["packed"], s["pre"], s["dH"], s["dpre"], s["dX"], act=act)
    return [s["dpre"], s["dX"]]


# ------------------------------------------------------------ the plain form

def _dense(layer):
    """W_hat [m, n] in fp32 from int8 signs [K, m, n] and scales [K, m, n/128]."""
    S, A = layer
    K, m, n = S.shape
    return (S.view(K, m, n // GROUP, GROUP).float() * A.float()[..., None]).sum(0).view(m, n)


def _stack(gate, up):
    """[T, m] gate and up values in the stacked order: 8 gate rows, 8 up rows."""
    T, m = gate.shape
    pad = -m % 8
    g, u = (torch.nn.functional.pad(v, (0, pad)).view(T, -1, 1, 8) for v in (gate, up))
    return torch.cat([g, u], 2).reshape(T, -1)


def _unstack(v, m):
    v = v.view(v.shape[0], -1, 2, 8)
    return v[:, :, 0].reshape(v.shape[0], -1)[:, :m], v[:, :, 1].reshape(v.shape[0], -1)[:, :m]


C_GELU, B_GELU = math.sqrt(2.0 / math.pi), 0.044715


def _act(act, g):
    """The activation and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(C_GELU * (g + B_GELU * g * g * g))
    return 0.5 * g * (1.0 + t), (0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * C_GELU *
                                 (1.0 + 3.0 * B_GELU * g * g))


def _plain_distill(case, s):
    # row statistics and the few listed entries in 64 bits: the loss is a
    # small difference of logarithms; what spans the vocabulary is 32 bits
    tau, V, Z = case["tau"], case["V"], s["Z"].float() / case["tau"]
    used = (s["idx"] >= 0) & (s["idx"] < V)
    at = torch.where(used, s["idx"], 0).long()
    t = torch.where(used, s["val"].double() / tau, -math.inf)
    top = Z.max(-1, keepdim=True).values
    e = torch.exp(Z - top)
    total = e.sum(-1, keepdim=True, dtype=F64)
    if s["lse"] is None:
        peak = t.max(-1, keepdim=True).values
        has = peak > -math.inf
        p = torch.where(has, torch.exp(t - torch.where(has, peak, 0.0)), 0.0)
        norm = torch.where(has, p.sum(-1, keepdim=True), 1.0)
        log_p = t - peak - torch.log(norm)
        p = p / norm
        has = has.float()
    else:
        log_p = t - s["lse"].double()[:, None]
        p, has = torch.exp(log_p), 1.0
    log_q = Z.gather(1, at).double() - top - torch.log(total)
    kl = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(-1)
    factor = 1.0
    if s["lse"] is not None:
        hit = torch.zeros_like(Z).scatter_add(1, at, used.float()) > 0
        rest = torch.where(hit, 0.0, e).sum(-1, dtype=F64) / total[:, 0]
        p_rest = (1.0 - p.sum(-1)).clamp_min(0.0)
        p_rest = torch.where(rest > 0, p_rest, 0.0)
        kl = kl + torch.where(p_rest > 0, p_rest * torch.log(p_rest / rest), 0.0)
        ratio = torch.where(p_rest > 0, p_rest / rest, 0.0)[:, None].float()
        factor = torch.where(hit, 1.0, 1.0 - ratio)
    w = s["weight"]
    loss = (w * tau * tau * kl).float()
    if case["mode"] == "loss":
        return [loss]
    dz = (e / total.float() * factor * has).scatter_add(1, at, torch.where(used, -p, 0.0).float())
    scale = w * tau * (s["dloss"] if case["mode"] == "pair" else 1.0)
    return [loss, (dz * scale[:, None]).to(s["Z"].dtype)]


def _plain(case, s):
    bf = torch.bfloat16
    if case["op"] == "distill":
        return _plain_distill(case, s)
    if case["op"] == "gemmt":
        return [(s["dY"].float() @ _dense(s["layer"])).to(bf)]
    if case["op"] == "scale_grad":
        S = s["layer"][0]
        K, m, n = S.shape
        dW = s["dY"].float().t() @ s["X"].float()
        return [(S.view(K, m, n // GROUP, GROUP) * dW.view(1, m, n // GROUP, GROUP)).sum(-1)]
    Wg, Wu = _dense(s["gate"]), _dense(s["up"])
    if case["op"] == "gated":
        X = s["X"].float()
        g, u = X @ Wg.t(), X @ Wu.t()
        out = [(_act(case["act"], g)[0] * u).to(bf)]
        return out + ([_stack(g, u).to(bf)] if case["keep"] else [])
    g, u = _unstack(s["pre"].float(), case["m"])
    a, da = _act(case["act"], g)
    dH = s["dH"].float()
    dg, du = dH * u * da, dH * a
    return [_stack(dg, du).to(bf), (dg @ Wg + du @ Wu).to(bf)]


def run(state):
    return _run_own(state["case"], state) if own else _plain(state["case"], state)


# ------------------------------------------------- the definition in 64 bits

def _exact_weight(layer):
    S, A = layer
    W = torch.zeros(S.shape[1:], dtype=F64, device=S.device)
    for k in range(S.shape[0]):
        W += S[k].to(F64) * A[k].to(F64).repeat_interleave(GROUP, dim=1)
    return W


def _exact_act(act, g):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    y = C_GELU * (g + B_GELU * g ** 3)
    t = torch.tanh(y)
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t ** 2) * C_GELU * (1 + 3 * B_GELU * g ** 2)


def _interleave(gate, up):
    T, m = gate.shape
    out = torch.zeros(T, _stacked_rows(m), dtype=F64, device=gate.device)
    i = torch.arange(m, device=gate.device)
    out[:, 16 * (i // 8) + i % 8] = gate
    out[:, 16 * (i // 8) + 8 + i % 8] = up
    return out


def _exact_distill(case, s):
    tau, V, T = case["tau"], case["V"], case["T"]
    loss = torch.zeros(T, dtype=F64, device=DEV)
    dZ = torch.zeros(T, V, dtype=F64, device=DEV)
    step = 256
    for r in range(0, T, step):
        rows = slice(r, min(T, r + step))
        logq = torch.log_softmax(s["Z"][rows].to(F64) / tau, -1)
        idx = s["idx"][rows].long()
        used = (idx >= 0) & (idx < V)
        at = idx.clamp(0, V - 1)
        t = (s["val"][rows].to(F64) / tau).masked_fill(~used, -math.inf)
        if s["lse"] is None:
            has = (t > -math.inf).any(-1, keepdim=True)
            logp = t - torch.where(has, torch.logsumexp(t, -1, keepdim=True), 0.0)
        else:
            has = torch.ones(t.shape[0], 1, dtype=torch.bool, device=DEV)
            logp = t - s["lse"][rows, None].to(F64)
        p = logp.exp()
        kl = torch.where(p > 0, p * (logp - logq.gather(1, at)), 0.0).sum(-1)
        q = logq.exp()
        grad = torch.where(has, q, 0.0)
        if s["lse"] is not None:
            member = torch.zeros(q.shape, dtype=torch.int32, device=DEV)
            member.scatter_add_(1, at, used.int())
            q_rest = q.masked_fill(member > 0, 0.0).sum(-1)
            p_rest = (1 - p.sum(-1)).clamp_min(0.0)
            live = (q_rest > 0) & (p_rest > 0)
            one = torch.ones_like(q_rest)
            ratio = torch.where(live, p_rest, 0 * one) / torch.where(live, q_rest, one)
            kl = kl + torch.where(live, p_rest * ratio.clamp_min(1e-300).log(), 0 * one)
            grad = grad - torch.where(member > 0, 0.0, q * ratio[:, None])
        grad = grad.scatter_add(1, at, -torch.where(used, p, 0.0))
        w = s["weight"][rows].to(F64)
        loss[rows] = w * tau ** 2 * kl
        if case["mode"] == "pair":
            w = w * s["dloss"][rows].to(F64)
        dZ[rows] = grad * (w * tau)[:, None]
    return [loss] if case["mode"] == "loss" else [loss, dZ]


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "distill":
        return _exact_distill(case, s)
    if case["op"] == "gemmt":
        return [s["dY"].to(F64) @ _exact_weight(s["layer"])]
    if case["op"] == "scale_grad":
        S = s["layer"][0]
        dW = s["dY"].to(F64).t() @ s["X"].to(F64)
        return [torch.stack([(dW * S[k]).unflatten(1, (-1, GROUP)).sum(2)
                             for k in range(S.shape[0])])]
    Wg, Wu = _exact_weight(s["gate"]), _exact_weight(s["up"])
    if case["op"] == "gated":
        X = s["X"].to(F64)
        g, u = X @ Wg.t(), X @ Wu.t()
        out = [_exact_act(case["act"], g)[0] * u]
        return out + ([_interleave(g, u)] if case["keep"] else [])
    m = case["m"]
    i = torch.arange(m, device=DEV)
    pre = s["pre"].to(F64)
    g, u = pre[:, 16 * (i // 8) + i % 8], pre[:, 16 * (i // 8) + 8 + i % 8]
    a, da = _exact_act(case["act"], g)
    dH = s["dH"].to(F64)
    dg, du = dH * u * da, dH * a
    return [_interleave(dg, du), dg @ Wg + du @ Wu]
