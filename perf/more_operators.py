"""Workloads of the layer's epilogue, the policy and preference losses and the
optimizer step, for measurement.

  linear      Y = R + act(X W_hat^T + b): the Boolean-kernel product with bias,
              activation and residual, one token up to a training batch
  linear_bwd  its backward: gradients of the pre-activations, the bias and X
  policy      clipped policy loss with a KL term on a row of logits per token,
              with the logits' gradient
  preference  loss of paired log ratios over chosen and rejected sequences,
              with the logits' gradient
  adamw       one AdamW step over many tensors, states in 32 or in 8 bits; the
              scales of a layer go into its packed buffer

W_hat = sum_k alpha_k (.) B_k with one alpha per output row and 128 columns.
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
FLOATS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # the LLaMA-7B-shaped MLP's down projection for one decoded token, added
        # to the residual stream
        dict(name="linear 1 token", op="linear", T=1, m=4096, n=11008, K=3, scales="f16",
             act="none", bias="none", residual=True, keep=False),
        # the up projection of an ungated block for a small serving batch
        dict(name="linear 16 tokens", op="linear", T=16, m=11008, n=4096, K=3, scales="f16",
             act="gelu", bias="bf16", residual=False, keep=False),
        # the same in a training step: the pre-activations are kept
        dict(name="linear 2048 tokens", op="linear", T=2048, m=11008, n=4096, K=3, scales="f16",
             act="gelu", bias="f32", residual=False, keep=True),
        # its backward
        dict(name="linear_bwd 2048 tokens", op="linear_bwd", T=2048, m=11008, n=4096, K=3,
             scales="f16", act="gelu", bias="f32"),
        # backward of a small layer: odd token count, a width that is no
        # multiple of a tile, fp32 scales, no activation
        dict(name="linear_bwd 37 tokens", op="linear_bwd", T=37, m=1001, n=640, K=2, scales="f32",
             act="none", bias="f32"),
        # the policy step of a batch, loss and gradient in one call
        dict(name="policy 2048 rows", op="policy", T=2048, V=32000, z="bf16", tau=1.0, kl=0.05),
        # fp32 logits of an odd vocabulary, sampled at another temperature, no
        # KL term
        dict(name="policy 301 rows", op="policy", T=301, V=12345, z="f32", tau=0.7, kl=0.0),
        # a batch of 8 chosen and 8 rejected sequences, loss and gradient
        dict(name="preference 2048 rows", op="preference", mode="step", T=2048, pairs=8, V=32000,
             z="bf16", mean=False),
        # the loss of one short pair alone (evaluation): latency
        dict(name="preference loss 37 rows", op="preference", mode="loss", T=37, pairs=1, V=32000,
             z="bf16", mean=True),
        # scales of eight LLaMA-7B-shaped decoder layers (per layer four
        # attention projections and two of the MLP's width) and their vectors
        dict(name="adamw 32-bit 48 layers", op="adamw", blocks=8, m=4096, f=11008, K=3,
             scales="f16", states="f32", vectors=16, vgrad="bf16"),
        # the same with states in 8 bits
        dict(name="adamw 8-bit 48 layers", op="adamw", blocks=8, m=4096, f=11008, K=3,
             scales="f16", states="f8", vectors=16, vgrad="bf16"),
        # one small block: latency
        dict(name="adamw small", op="adamw", blocks=1, m=256, f=512, K=2, scales="f32",
             states="f32", vectors=1, vgrad="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "policy", "preference", "adamw"])
    if op == "policy":
        return dict(op=op, T=_log_int(rng, 1, 2048), V=_log_int(rng, 500, 32000),
                    z=rng.choice(["bf16", "f16", "f32"]), tau=rng.choice([0.7, 1.0, 1.5]),
                    kl=rng.choice([0.0, 0.02, 0.2]))
    if op == "preference":
        T = _log_int(rng, 2, 2048)
        return dict(op=op, mode=rng.choice(["step", "loss"]), T=T,
                    pairs=_log_int(rng, 1, min(16, T // 2)), V=_log_int(rng, 500, 32000),
                    z=rng.choice(["bf16", "f16", "f32"]), mean=rng.random() < 0.5)
    if op == "adamw":
        return dict(op=op, blocks=_log_int(rng, 1, 8), m=GROUP * _log_int(rng, 1, 32),
                    f=GROUP * _log_int(rng, 1, 86), K=rng.choice([1, 2, 3]),
                    scales=rng.choice(["f16", "f32"]), states=rng.choice(["f32", "f8"]),
                    vectors=rng.randint(0, 12), vgrad=rng.choice(["bf16", "f16", "f32"]))
    n = GROUP * _log_int(rng, 1, 86)
    m = _log_int(rng, 8, 11008)
    most = 11008 * 4096 * 2048
    T = _log_int(rng, 1, min(2048, max(1, most // (m * n))))
    case = dict(op=op, T=T, m=m, n=n, K=rng.choice([1, 2, 3, 4]),
                scales=rng.choice(["f16", "f32"]), act=rng.choice(["none", "silu", "gelu"]))
    if op == "linear":
        case.update(bias=rng.choice(["none", "bf16", "f32"]), residual=rng.random() < 0.5,
                    keep=rng.random() < 0.5)
    else:
        case["bias"] = rng.choice(["none", "f32"])
    return case


def _layers(case):
    """(rows, columns) of the layers of an optimizer case: per block four square
    projections, one up and one down."""
    m, f = case["m"], case["f"]
    return [(m, m)] * 4 * case["blocks"] + [(f, m), (m, f)] * case["blocks"]


def work(case):
    op = case["op"]
    if op in ("policy", "preference"):
        row = case["V"] * FLOATS[case["z"]].itemsize
        passes = 2 if op == "policy" else 3 if case["mode"] == "step" else 1
        return {"bytes": case["T"] * (passes * row + 32), "flops": 0}
    if op == "adamw":
        scales = case["K"] * sum(m * (n // GROUP) for m, n in _layers(case))
        states = 16 if case["states"] == "f32" else 4
        vectors = case["vectors"] * case["m"]
        return {"bytes": scales * (8 + 4 + states + FLOATS[case["scales"]].itemsize) +
                vectors * (8 + FLOATS[case["vgrad"]].itemsize + states + 2), "flops": 0}
    T, m, n, K = case["T"], case["m"], case["n"], case["K"]
    weights = K * m * n // 8 + K * m * (n // GROUP) * FLOATS[case["scales"]].itemsize
    if op == "linear":
        out = T * m * 2 * (1 + case["residual"] + case["keep"])
        return {"bytes": weights + T * n * 2 + out, "flops": 2 * T * m * n}
    act = 2 if case["act"] != "none" else 0  # pre read, dpre written
    return {"bytes": weights + T * m * 2 * (1 + act) + T * n * 2, "flops": 2 * T * m * n}


# ---------------------------------------------------------------- the inputs

def _greedy(W, K, scales):
    """K kernels and scales of W by successive sign and mean magnitude."""
    m, n = W.shape
    R, S, A = W.clone(), [], []
    for _ in range(K):
        s = torch.where(R >= 0, 1.0, -1.0)
        a = R.abs().view(m, n // GROUP, GROUP).mean(-1).to(FLOATS[scales])
        R -= (s.view(m, n // GROUP, GROUP) * a.float()[..., None]).view(m, n)
        S.append(s.to(torch.int8))
        A.append(a)
    return torch.stack(S).contiguous(), torch.stack(A).contiguous()


def _inputs(case, seed):
    """The case's data, from the seed alone."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    if case["op"] == "adamw":
        return _adamw_inputs(case, gen)
    if case["op"] in ("policy", "preference"):
        return _loss_inputs(case, gen)

    def bf16(rows, cols, scale=1.0):
        return (torch.randn(rows, cols, generator=gen, device=DEV) * scale).to(torch.bfloat16)

    T, m, n = case["T"], case["m"], case["n"]
    s = dict(case=case, layer=_greedy(torch.randn(m, n, generator=gen, device=DEV) * 0.02,
                                      case["K"], case["scales"]))
    if case["op"] == "linear":
        s["X"] = bf16(T, n)
        s["bias"] = None
        if case["bias"] != "none":
            s["bias"] = (torch.randn(m, generator=gen, device=DEV) * 0.1).to(FLOATS[case["bias"]])
        s["R"] = bf16(T, m) if case["residual"] else None
        return s
    s["dY"] = bf16(T, m, 0.01)
    # pre-activations of unit-variance inputs have a spread of about 1.3
    s["pre"] = bf16(T, m, 1.3) if case["act"] != "none" else None
    return s


def _loss_inputs(case, gen):
    """Logits with a few likely tokens per row and the tokens sampled from them;
    the sampling policy and the reference near the present one.  Prompt rows have
    label -1; sequences are of any length, some empty."""
    T, V, tau = case["T"], case["V"], case.get("tau", 1.0)
    Z = (torch.randn(T, V, generator=gen, device=DEV) * 2.5).to(FLOATS[case["z"]])
    logq = torch.log_softmax(Z.float() / tau, -1)
    noise = torch.rand(T, V, generator=gen, device=DEV).clamp_min(1e-9)
    label = (logq - torch.log(-torch.log(noise))).argmax(-1)
    logp = logq.gather(1, label[:, None])[:, 0]
    del logq, noise
    near = [0.3 * torch.randn(T, generator=gen, device=DEV) for _ in range(2)]
    prompt = torch.rand(T, generator=gen, device=DEV) < 0.1
    prompt[0] = False
    s = dict(case=case, Z=Z, label=torch.where(prompt, -1, label).to(torch.int32))
    if case["op"] == "policy":
        s["old"] = logp + near[0]
        s["ref"] = logp + near[1] if case["kl"] else None
        s["adv"] = torch.randn(T, generator=gen, device=DEV)
        # mean over the rows; fp16 gradients under a loss scale, as they are kept
        mean = (4096.0 if case["z"] == "f16" else 1.0) / T
        s["weight"] = (torch.rand(T, generator=gen, device=DEV) >= 0.05).float() * mean
        s["weight"][0] = mean
        return s
    pairs = case["pairs"]
    s["ref"] = torch.where(s["label"] < 0, 0.0, logp + near[1])
    cuts = torch.randint(0, T + 1, (2 * pairs - 1,), generator=gen, device=DEV).sort().values
    s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
    s["weight"] = (0.5 + torch.rand(pairs, generator=gen, device=DEV)) * (
        (256.0 if case["z"] == "f16" else 1.0) / pairs)
    return s


BLOCK = 256  # values that share a scale of an 8-bit state


def _arena(counts):
    """Start of each tensor in a flat buffer of whole blocks, and its size."""
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += (c + BLOCK - 1) // BLOCK * BLOCK
    return starts, at


def _adamw_inputs(case, gen):
    """Scales of layers, and vectors (norm weights, biases), as a program holds
    them: one flat buffer for parameters, for gradients and for each state, and
    the packed layers."""
    K, sb = case["K"], FLOATS[case["scales"]]
    shapes = _layers(case)
    counts = [K * m * (n // GROUP) for m, n in shapes] + [case["m"]] * case["vectors"]
    starts, size = _arena(counts)
    split = starts[len(shapes)] if case["vectors"] else size
    s = dict(case=case, counts=counts, starts=starts, shapes=shapes, size=size)

    def rand(scale, count=size):
        return torch.randn(count, generator=gen, device=DEV) * scale

    # which values are parameters (the rest fills blocks and stays 0)
    s["tensor"] = torch.zeros(size, dtype=torch.int64, device=DEV)
    s["index"] = torch.zeros(size, dtype=torch.int64, device=DEV)
    live = torch.zeros(size, device=DEV)
    s["decay"] = torch.zeros(size, device=DEV)
    for i, (a, c) in enumerate(zip(starts, counts)):
        s["tensor"][a:a + c] = i
        s["index"][a:a + c] = torch.arange(c, device=DEV)
        live[a:a + c] = 1.0
        s["decay"][a:a + c] = 0.01 if i < len(shapes) else 0.0
    s["p"] = (0.02 + rand(0.005).abs()) * live
    size_of = torch.exp(rand(1.0))  # gradients of very different sizes
    s["glayers"] = (rand(1e-3) * size_of * live)[:split].contiguous()
    s["gvectors"] = (rand(1e-3) * live)[split:].to(FLOATS[case["vgrad"]])
    m = rand(3e-4) * size_of * live
    r = (rand(1e-3).abs() + 1e-4) * size_of * live
    if case["states"] == "f32":
        s["m"], s["v"] = m, r * r
    else:
        for name, x in (("m", m), ("r", r)):
            top = x.view(-1, BLOCK).abs().amax(-1)
            scale = torch.exp2(torch.floor(torch.log2(top.clamp_min(1e-12))) - 7)
            s[name + "_scale"] = scale
            s[name] = (x.view(-1, BLOCK) / scale[:, None]).view(-1).to(torch.float8_e4m3fn)
    s["packed"] = []
    for m_, n_ in shapes:
        rows = (m_ + 63) // 64 * 64
        bits = K * rows * n_ // 8
        s["packed"].append(torch.zeros(bits + K * rows * (n_ // GROUP) * sb.itemsize,
                                       dtype=torch.uint8, device=DEV))
    s["copy"] = torch.zeros(size - split, dtype=torch.bfloat16, device=DEV)
    s["split"] = split
    return s


ADAMW = dict(lr=1e-4, step=100, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=0.5, seed=12345)
POLICY = dict(low=0.2, high=0.28)
PREFERENCE = dict(beta=0.1, smoothing=0.1, margin=0.05)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(case, s)
    return s


# ----------------------------------------------- the package's own operators

def _prepare_own(case, s):
    """What a program keeps: the packed layer, output buffers, workspaces, the
    optimizer's plan."""
    import boolean_weight_amd as bw
    op = case["op"]
    if op == "adamw":
        s["plan"] = _plan(bw, case, s)
        return
    T = case["T"]
    if op in ("policy", "preference"):
        f32 = dict(device=DEV)
        s["logp"], s["dZ"] = torch.zeros(T, **f32), torch.empty_like(s["Z"])
        if op == "policy":
            s["d"] = bw.mbok_policy_desc_init(case["V"], case["tau"], POLICY["low"],
                                              POLICY["high"], case["kl"])
            s["loss"] = torch.empty(T, **f32)
        else:
            s["d"] = bw.mbok_logp_desc_init(case["V"])
            s["dp"] = bw.mbok_preference_desc_init(PREFERENCE["beta"], PREFERENCE["smoothing"],
                                                   PREFERENCE["margin"], case["mean"])
            s["loss"] = torch.empty(case["pairs"], **f32)
            s["stats"] = torch.empty(T, bw.MBOK_LOGP_STATS, **f32)
            s["dlogp"] = torch.zeros(T, **f32)
        return
    m, n, bf = case["m"], case["n"], dict(dtype=torch.bfloat16, device=DEV)
    s["d"] = d = bw.mbok_desc_init(m, n, case["K"],
                                   bw.MBOK_F16 if case["scales"] == "f16" else bw.MBOK_F32)
    s["packed"] = torch.empty(bw.mbok_packed_bytes(d), dtype=torch.uint8, device=DEV)
    bw.mbok_pack(d, *s.pop("layer"), s["packed"])
    s["act"] = {"none": bw.MBOK_ACT_NONE, "silu": bw.MBOK_ACT_SILU,
                "gelu": bw.MBOK_ACT_GELU}[case["act"]]
    # rows of 16-byte pieces, as a program lays its activations out
    wide = (m + 7) // 8 * 8
    if op == "linear":
        s["Y"] = torch.empty(T, wide, **bf)[:, :m]
        s["keep"] = torch.empty(T, wide, **bf)[:, :m] if case["keep"] else None
    else:
        s["dX"] = torch.empty(T, n, **bf)
        s["dpre"] = torch.empty(T, wide, **bf)[:, :m] if case["act"] != "none" else None
        s["dbias"] = torch.empty(m, device=DEV) if case["bias"] != "none" else None


def _plan(bw, case, s):
    dt = bw.MBOK_F16 if case["scales"] == "f16" else bw.MBOK_F32
    tensors = []
    for i, (a, c) in enumerate(zip(s["starts"], s["counts"])):
        at, block = slice(a, a + c), slice(a // BLOCK, (a + c + BLOCK - 1) // BLOCK)
        t = dict(param=s["p"][at], m=s["m"][at])
        if case["states"] == "f32":
            t["v"] = s["v"][at]
        else:
            t.update(v=s["r"][at], m_scale=s["m_scale"][block], v_scale=s["r_scale"][block])
        if i < len(s["shapes"]):
            t.update(grad=s["glayers"][at], out=s["packed"][i], weight_decay=0.01,
                     layer=bw.mbok_desc_init(*s["shapes"][i], case["K"], dt))
        else:
            b = a - s["split"]
            t.update(grad=s["gvectors"][b:b + c], out=s["copy"][b:b + c])
        tensors.append(t)
    return bw.mbok_adamw_plan_init(tensors)


def _run_own(case, s):
    import boolean_weight_amd as bw
    op = case["op"]
    if op == "linear":
        bw.mbok_linear(s["d"], s["packed"], s["X"], s["Y"], bias=s["bias"], act=s["act"],
                       residual=s["R"], pre=s["keep"])
        return [s["Y"]] + ([s["keep"]] if case["keep"] else [])
    if op == "linear_bwd":
        bw.mbok_linear_backward(s["d"], s["packed"], s["dY"], pre=s["pre"], dpre=s["dpre"],
                                dbias=s["dbias"], dX=s["dX"], act=s["act"])
        return [v for v in (s["dpre"], s["dbias"], s["dX"]) if v is not None]
    if op == "policy":
        bw.mbok_policy(s["d"], s["Z"], s["label"], s["adv"], s["loss"], old_logp=s["old"],
                       ref_logp=s["ref"], weight=s["weight"], logp=s["logp"], dZ=s["dZ"])
        return [s["loss"], s["logp"], s["dZ"]]
    if op == "preference":
        step = case["mode"] == "step"
        bw.mbok_logp(s["d"], s["Z"], s["label"], s["logp"], stats=s["stats"] if step else None)
        bw.mbok_preference(s["dp"], s["offsets"], s["logp"], s["loss"], ref_logp=s["ref"],
                           label=s["label"], weight=s["weight"],
                           dlogp=s["dlogp"] if step else None)
        if not step:
            return [s["loss"], s["logp"]]
        bw.mbok_logp_backward(s["d"], s["Z"], s["label"], s["stats"], s["dlogp"], s["dZ"])
        return [s["loss"], s["logp"], s["dZ"]]
    bw.mbok_adamw(s["plan"], **ADAMW)
    return _adamw_outputs(case, s)


def _scales_of(case, s, i):
    """Layer i's scales in its packed buffer, [row blocks, groups, K, 64]."""
    m, n = s["shapes"][i]
    rows = (m + 63) // 64
    bits = case["K"] * rows * 64 * n // 8
    return s["packed"][i][bits:].view(FLOATS[case["scales"]]).view(rows, n // GROUP, case["K"], 64)


def _adamw_outputs(case, s):
    states = [s["m"], s["v"]] if case["states"] == "f32" else [s["m"], s["r"], s["m_scale"],
                                                               s["r_scale"]]
    return [s["p"]] + states + [s["copy"]] + [_scales_of(case, s, i)
                                               for i in range(len(s["shapes"]))]


# ------------------------------------------------------------ the plain form

def _dense(layer):
    """W_hat [m, n] in fp32 from int8 signs [K, m, n] and scales [K, m, n/128]."""
    S, A = layer
    K, m, n = S.shape
    return (S.view(K, m, n // GROUP, GROUP).float() * A.float()[..., None]).sum(0).view(m, n)


C_GELU, B_GELU = math.sqrt(2.0 / math.pi), 0.044715


def _act(act, g):
    """The activation and its derivative."""
    if act == "none":
        return g, torch.ones_like(g)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(C_GELU * (g + B_GELU * g * g * g))
    return 0.5 * g * (1.0 + t), (0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * C_GELU *
                                 (1.0 + 3.0 * B_GELU * g * g))


def _plain_logp(Z, label, tau):
    """Row log-probabilities in 64 bits (the ratios are next to a border) from
    exponentials in 32, those exponentials and their sums."""
    there = label >= 0
    at = torch.where(there, label, 0).long()[:, None]
    z = Z.float() / tau
    top = z.max(-1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True, dtype=F64)
    logp = (z.gather(1, at) - top).double() - torch.log(total)
    return there, at, torch.where(there, logp[:, 0], 0.0), e / total.float()


def _plain_dz(Z, at, q, slope, tau):
    """d / dZ of sum_t slope_t logp_t from the probabilities q."""
    dz = (-q).scatter_add(1, at, torch.ones_like(at, dtype=q.dtype))
    return (dz * (slope / tau).float()[:, None]).to(Z.dtype)


def _plain_policy(case, s):
    there, at, logp, q = _plain_logp(s["Z"], s["label"], case["tau"])
    A = s["adv"].double()
    ratio = torch.exp(logp - s["old"].double())
    low, high = 1.0 - POLICY["low"], 1.0 + POLICY["high"]
    gain = torch.minimum(ratio * A, ratio.clamp(low, high) * A)
    inside = torch.where(A >= 0, ratio <= high, ratio >= low)
    slope = torch.where(inside, -ratio * A, 0.0)
    loss = -gain
    if s["ref"] is not None:
        x = s["ref"].double() - logp
        loss = loss + case["kl"] * (torch.expm1(x) - x)
        slope = slope - case["kl"] * torch.expm1(x)
    w = torch.where(there, s["weight"], 0.0).double()
    return [(loss * w).float(), logp.float(), _plain_dz(s["Z"], at, q, slope * w, case["tau"])]


def _plain_preference(case, s):
    there, at, logp, q = _plain_logp(s["Z"], s["label"], 1.0)
    T, pairs, off = case["T"], case["pairs"], s["offsets"].long()
    row = torch.arange(T, device=DEV)
    seq = torch.searchsorted(off[1:], row, right=True)
    diff = torch.where(there, logp.float().double() - s["ref"].double(), 0.0)
    sums = torch.zeros(2 * pairs, dtype=F64, device=DEV).index_add(0, seq, diff)
    size = torch.ones(2 * pairs, dtype=F64, device=DEV)
    if case["mean"]:
        size = torch.zeros_like(size).index_add(0, seq, there.double()).clamp_min(1.0)
    score = (sums / size).view(pairs, 2)
    beta, ls = PREFERENCE["beta"], PREFERENCE["smoothing"]
    h = beta * (score[:, 0] - score[:, 1]) - PREFERENCE["margin"]
    soft = torch.log1p(torch.exp(-h.abs()))
    w = s["weight"].double()
    loss = w * ((1 - ls) * (soft + (-h).clamp_min(0.0)) + ls * (soft + h.clamp_min(0.0)))
    if case["mode"] == "loss":
        return [loss.float(), logp.float()]
    sig = 1.0 / (1.0 + torch.exp(-h))
    dh = w * beta * (ls * sig - (1 - ls) * (1.0 - sig))
    dseq = torch.stack([dh, -dh], 1).view(-1) / size
    slope = torch.where(there, dseq[seq], 0.0)
    return [loss.float(), logp.float(), _plain_dz(s["Z"], at, q, slope, 1.0)]


# Stochastic rounding of the 8-bit states takes its bits from a hash of the
# value's index, its tensor's place, the step and the seed.
H = (0x9E3779B1, 0x6A09E667, 0xBB67AE85, 0x3C6EF373, 0xA54FF53B)
M32 = 0xFFFFFFFF


def _bits(s):
    key = (ADAMW["seed"] + ADAMW["step"] * H[0]) & M32
    h = (s["index"] * H[2] + s["tensor"] * H[1] + key) & M32
    h = ((h ^ (h >> 16)) * H[3]) & M32
    h = ((h ^ (h >> 15)) * H[4]) & M32
    h = h ^ (h >> 16)
    return [((b << 4) | 8).int() for b in (h & 0xFFFF, h >> 16)]


def _to_e4m3(x, bits, least):
    """x in e4m3 codes with one power-of-two scale per block, the block's largest
    in [128, 256); `bits`: 20 random bits each; `least`: the smallest code of a
    value that is not 0."""
    top = x.abs().view(-1, BLOCK).amax(-1).view(torch.int32) >> 23
    top = top.clamp_min(47) - 7
    scale = (top << 23).view(torch.float32)
    up = ((254 - top) << 23).view(torch.float32)
    y = x.abs() * up.repeat_interleave(BLOCK)
    normal = ((y.view(torch.int32) + bits) >> 20) - 960
    small = torch.floor(y * 512.0 + bits.float() * 2.0 ** -20).int()
    code = torch.where(y >= 2.0 ** -6, normal, small)
    code = torch.where(x != 0, code.clamp_min(least), code)
    code = torch.where(x < 0, code | 128, code)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), scale


def _plain_adamw(case, s):
    o, eight = ADAMW, case["states"] == "f8"
    b1, b2 = o["beta1"], o["beta2"]
    g = torch.cat([s["glayers"], s["gvectors"].float()]) * o["grad_scale"]
    if eight:
        m = s["m"].float() * s["m_scale"].repeat_interleave(BLOCK)
        r = s["r"].float() * s["r_scale"].repeat_interleave(BLOCK)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = torch.sqrt(v)
    step = o["lr"] / (1 - b1 ** o["step"])
    den = r * (1 / math.sqrt(1 - b2 ** o["step"])) + o["eps"]
    s["p"].copy_(s["p"] * (1.0 - o["lr"] * s["decay"]) - step * (m / den))
    if eight:
        bits = _bits(s)
        for name, x, b, least in (("m", m, bits[0], 0), ("r", r, bits[1], 1)):
            code, scale = _to_e4m3(x, b, least)
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    s["copy"].copy_(s["p"][s["split"]:])
    for i, (m_, n_) in enumerate(s["shapes"]):
        a, G, rows = s["starts"][i], n_ // GROUP, (m_ + 63) // 64
        x = s["p"][a:a + s["counts"][i]].view(case["K"], m_, G)
        x = torch.nn.functional.pad(x, (0, 0, 0, rows * 64 - m_)).view(case["K"], rows, 64, G)
        _scales_of(case, s, i).copy_(x.permute(1, 3, 0, 2))
    return _adamw_outputs(case, s)


def _plain(case, s):
    bf, op = torch.bfloat16, case["op"]
    if op == "policy":
        return _plain_policy(case, s)
    if op == "preference":
        return _plain_preference(case, s)
    if op == "adamw":
        return _plain_adamw(case, s)
    W = _dense(s["layer"])
    if op == "linear":
        z = s["X"].float() @ W.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(case["act"], z)[0]
        if s["R"] is not None:
            y = s["R"].float() + y
        return [y.to(bf)] + ([z.to(bf)] if case["keep"] else [])
    dz, out = s["dY"].float(), []
    if case["act"] != "none":
        dz = dz * _act(case["act"], s["pre"].float())[1]
        out.append(dz.to(bf))
    if case["bias"] != "none":
        out.append(dz.sum(0))
    return out + [(dz @ W).to(bf)]


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
    if act == "none":
        return g, torch.ones_like(g)
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    y = C_GELU * (g + B_GELU * g ** 3)
    t = torch.tanh(y)
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t ** 2) * C_GELU * (1 + 3 * B_GELU * g ** 2)


def _exact_rows(Z, label, tau, slope_of=None):
    """Row log-probabilities and, with slope_of(rows, logp), the gradient."""
    T, V = Z.shape
    logp = torch.zeros(T, dtype=F64, device=DEV)
    dZ = torch.zeros(T, V, dtype=F64, device=DEV) if slope_of else None
    for r in range(0, T, 256):
        rows = slice(r, min(T, r + 256))
        logq = torch.log_softmax(Z[rows].to(F64) / tau, -1)
        lab = label[rows].long()
        picked = logq.gather(1, lab.clamp_min(0)[:, None])[:, 0]
        logp[rows] = torch.where(lab >= 0, picked, torch.zeros_like(picked))
        if slope_of:
            d = -logq.exp()
            d.scatter_add_(1, lab.clamp_min(0)[:, None], torch.ones(len(lab), 1, dtype=F64,
                                                                    device=DEV))
            dZ[rows] = d * (slope_of(rows, logp[rows]) / tau)[:, None]
    return logp, dZ


def _exact_policy(case, s):
    loss = torch.zeros(case["T"], dtype=F64, device=DEV)

    def slope_of(rows, logp):
        A, keep = s["adv"][rows].to(F64), (s["label"][rows] >= 0).to(F64)
        ratio = torch.exp(logp - s["old"][rows].to(F64))
        cut = torch.clip(ratio, 1 - POLICY["low"], 1 + POLICY["high"])
        clipped = cut * A < ratio * A
        w = s["weight"][rows].to(F64) * keep
        part, slope = -torch.where(clipped, cut, ratio) * A, -torch.where(clipped, 0 * A, ratio * A)
        if s["ref"] is not None:
            k = s["ref"][rows].to(F64) - logp
            part = part + case["kl"] * (k.exp() - k - 1)
            slope = slope + case["kl"] * (1 - k.exp())
        loss[rows] = w * part
        return w * slope

    logp, dZ = _exact_rows(s["Z"], s["label"], case["tau"], slope_of)
    return [loss, logp, dZ]


def _exact_preference(case, s):
    logp, _ = _exact_rows(s["Z"], s["label"], 1.0)
    off, pairs = s["offsets"].tolist(), case["pairs"]
    counted = s["label"] >= 0
    diff = torch.where(counted, logp - s["ref"].to(F64), torch.zeros_like(logp))
    dlogp, losses = torch.zeros_like(logp), []
    for p in range(pairs):
        parts = []
        for q in (2 * p, 2 * p + 1):
            rows = slice(off[q], off[q + 1])
            size = max(1, int(counted[rows].sum())) if case["mean"] else 1
            parts.append((rows, size, diff[rows].sum() / size))
        h = PREFERENCE["beta"] * (parts[0][2] - parts[1][2]) - PREFERENCE["margin"]
        w, ls = s["weight"][p].to(F64), PREFERENCE["smoothing"]
        losses.append(-w * ((1 - ls) * torch.nn.functional.logsigmoid(h) +
                            ls * torch.nn.functional.logsigmoid(-h)))
        dh = -w * ((1 - ls) * torch.sigmoid(-h) - ls * torch.sigmoid(h)) * PREFERENCE["beta"]
        for sign, (rows, size, _) in zip((1, -1), parts):
            dlogp[rows] = sign * dh / size * counted[rows]
    out = [torch.stack(losses), logp]
    if case["mode"] == "step":
        out.append(_exact_rows(s["Z"], s["label"], 1.0, lambda rows, _: dlogp[rows])[1])
    return out


def _exact_adamw(case, s):
    o, eight = ADAMW, case["states"] == "f8"
    g = torch.cat([s["glayers"].to(F64), s["gvectors"].to(F64)]) * o["grad_scale"]
    if eight:
        m = (s["m"].to(F64).view(-1, BLOCK) * s["m_scale"].to(F64)[:, None]).view(-1)
        v = (s["r"].to(F64).view(-1, BLOCK) * s["r_scale"].to(F64)[:, None]).view(-1) ** 2
    else:
        m, v = s["m"].to(F64), s["v"].to(F64)
    m = o["beta1"] * m + (1 - o["beta1"]) * g
    v = o["beta2"] * v + (1 - o["beta2"]) * g ** 2
    mhat, vhat = m / (1 - o["beta1"] ** o["step"]), v / (1 - o["beta2"] ** o["step"])
    p = s["p"].to(F64) * (1 - o["lr"] * s["decay"].to(F64))
    p = p - o["lr"] * mhat / (vhat.sqrt() + o["eps"])
    out = [p] + ([None] * 4 if eight else [m, v]) + [p[s["split"]:]]
    for i, (m_, n_) in enumerate(s["shapes"]):
        G, rows = n_ // GROUP, (m_ + 63) // 64
        x = torch.zeros(case["K"], rows * 64, G, dtype=F64, device=DEV)
        x[:, :m_] = p[s["starts"][i]:s["starts"][i] + s["counts"][i]].view(case["K"], m_, G)
        out.append(x.view(case["K"], rows, 64, G).permute(1, 3, 0, 2).contiguous())
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "policy":
        return _exact_policy(case, s)
    if op == "preference":
        return _exact_preference(case, s)
    if op == "adamw":
        return _exact_adamw(case, s)
    W = _exact_weight(s["layer"])
    if op == "linear":
        z = s["X"].to(F64) @ W.t()
        if s["bias"] is not None:
            z = z + s["bias"].to(F64)
        y = _exact_act(case["act"], z)[0]
        if s["R"] is not None:
            y = y + s["R"].to(F64)
        return [y] + ([z] if case["keep"] else [])
    dz, out = s["dY"].to(F64), []
    if case["act"] != "none":
        dz = dz * _exact_act(case["act"], s["pre"].to(F64))[1]
        out.append(dz)
    if case["bias"] != "none":
        out.append(dz.sum(0))
    return out + [dz @ W]
