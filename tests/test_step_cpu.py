"""The layer with its epilogue, the policy and preference losses and the
optimizer step on the CPU: the references' gradients against differences, the
8-bit rounding's mean, the optimizer's table, and every refusal of the C ABI
and the binding (no call here reaches a kernel)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref
import step_ref as ref
from test_finetune_cpu import BAD_DESC, P, call, desc, differences

F64, BLOCK = torch.float64, bw.MBOK_ADAMW_BLOCK


# ------------------------------------------------- gradients by differences
# (see test_finetune_cpu.py for the step and the error)

@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_linear_gradient_is_the_slope(kind):
    gen = torch.Generator().manual_seed(5)
    T, m, n = 3, 4, 128
    W = torch.randn(m, n, generator=gen, dtype=F64) * 0.1
    X, R, b = (torch.randn(*s, generator=gen, dtype=F64) for s in ((T, n), (T, m), (m,)))
    up = torch.randn(T, m, generator=gen, dtype=F64)

    def loss():
        return float((up * ref.linear(W, X, b, kind, R)[0]).sum())

    dz = up * ref.act_slope(kind, ref.linear(W, X, b, kind, R)[1])
    assert torch.allclose(differences(loss, X), dz @ W, rtol=0, atol=1e-6)
    assert torch.allclose(differences(loss, b), dz.sum(0), rtol=0, atol=1e-6)
    assert torch.allclose(differences(loss, R), up, rtol=0, atol=1e-6)


@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_logp_gradient_is_the_slope(tau):
    gen = torch.Generator().manual_seed(6)
    Z = torch.randn(4, 9, generator=gen, dtype=F64)
    label, up = torch.tensor([3, -1, 0, 12]), torch.randn(4, generator=gen, dtype=F64)

    def loss():
        return float((up * ref.logp(Z, label, tau)[0]).sum())

    assert torch.allclose(differences(loss, Z), ref.logp_grad(Z, label, tau, up), rtol=0,
                          atol=1e-6)


@pytest.mark.parametrize("with_old,with_ref", [(True, True), (True, False), (False, True)])
def test_policy_slope_is_the_slope(with_old, with_ref):
    lp = torch.tensor([-1.0, -2.0, -0.3, -4.0, -1.5, -2.5], dtype=F64)
    # ratios 1.05, 1.5 (clipped up), 0.5 (A < 0: clipped), 0.5 (A > 0: not), 1.5, 0.9
    old = lp - torch.tensor([1.05, 1.5, 0.5, 0.5, 1.5, 0.9], dtype=F64).log()
    A = torch.tensor([1.0, 2.0, -1.0, 1.0, -1.0, -0.5], dtype=F64)
    w = torch.tensor([1.0, 0.5, 2.0, 1.0, 1.0, 0.0], dtype=F64)
    label = torch.zeros(6, dtype=torch.int32)
    more = dict(w=w, kl=0.3)
    if with_ref:
        more["ref_lp"] = lp + torch.tensor([0.2, -0.4, 1.0, 0.0, -1.0, 0.3], dtype=F64)
    fixed = old if with_old else lp.clone()

    def loss():
        return float(ref.policy(lp, label, 1, A, fixed, **more)[0].sum())

    slope = ref.policy(lp, label, 1, A, fixed if with_old else None, **more)[1]
    assert torch.allclose(differences(loss, lp), slope, rtol=0, atol=1e-6)


@pytest.mark.parametrize("mean", [False, True])
def test_preference_slope_is_the_slope(mean):
    gen = torch.Generator().manual_seed(9)
    lp = torch.randn(12, generator=gen, dtype=F64)
    more = dict(label=torch.tensor([1, 1, -1, 1, 1, 1, -1, 1, 1, 1, 1, 1]),
                ref_lp=torch.randn(12, generator=gen, dtype=F64),
                w=torch.tensor([1.0, 0.5], dtype=F64), beta=0.4, smoothing=0.1, margin=0.2,
                mean=mean)
    off = [0, 3, 7, 7, 11]  # an empty chosen sequence; row 11 in none

    def loss():
        return float(ref.preference(lp, off, **more)[0].sum())

    d = ref.preference(lp, off, **more)[1]
    assert math.isnan(float(d[11]))
    assert torch.allclose(differences(loss, lp)[:11], d[:11], rtol=0, atol=1e-6)


# ------------------------------------------------------------- 8-bit rounding

def test_stochastic_codes_have_the_value_as_their_mean():
    """A value y between two codes a step s apart: the mean of N roundings is off by a
    normal variable of deviation at most s / (2 sqrt N), and by 2^-17 s since the
    random numbers are multiples of 2^-16; 5 deviations."""
    N, values = 4096, ref.e4m3_values()
    for y in (200.0, 130.3, 17.77, 0.9, 0.02, 0.0041, 0.0007):
        x = np.full(BLOCK, y, np.float32)
        x[0] = 255.0
        got = []
        for step in range(N // (BLOCK - 1) + 1):
            rnd, _ = ref.random_bits(BLOCK, 3, step + 1, 77)
            codes, scales = ref.encode(x, rnd, 0)
            assert scales[0] == 1.0
            got.append(values[torch.from_numpy(codes[1:].astype(np.int64))])
        got = torch.cat(got)
        s = max(2.0 ** (math.floor(math.log2(y)) - 3), 2.0 ** -9)
        assert abs(float(got.mean()) - y) <= 5 * s / (2 * math.sqrt(len(got))) + 2.0 ** -17 * s
        assert float((got - y).abs().max()) < s


def test_random_bits_are_spread():
    """Each of the 16 bits of both numbers is set in half of the values, and
    neighbours, steps and tensors do not share them: 5 deviations of 1 / (2 sqrt N)."""
    N = 1 << 16
    base = ref.random_bits(N, 0, 1, 0)
    others = [ref.random_bits(N, 1, 1, 0), ref.random_bits(N, 0, 2, 0),
              ref.random_bits(N, 0, 1, 1)]
    tol = 5 / (2 * math.sqrt(N))
    for part in range(2):
        for bit in range(16):
            b = (base[part] >> bit) & 1
            assert abs(b.mean() - 0.5) <= tol
            assert abs((b[1:] ^ b[:-1]).mean() - 0.5) <= tol
            for o in others:
                assert abs((b ^ ((o[part] >> bit) & 1)).mean() - 0.5) <= tol


# ----------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    return bw.load_library()


def linear_args():
    d = desc(m=250)
    return dict(d=ctypes.byref(d), packed=P, X=P, xd=bw.MBOK_BF16, T=4, ldx=512, bias=P,
                bd=bw.MBOK_F32, act=2, R=2 * P, ldr=250, Y=P, yd=bw.MBOK_BF16, ldy=250, pre=3 * P,
                ldpre=250, s=None), d


LINEAR = [
    (dict(d=None), -1), (dict(d=ctypes.byref(BAD_DESC)), -2), (dict(packed=None), -1),
    (dict(X=None), -1), (dict(Y=None), -1), (dict(T=0), -2), (dict(T=bw.MBOK_MAX_T + 1), -2),
    (dict(xd=bw.MBOK_F32), -3), (dict(yd=bw.MBOK_F16), -3), (dict(yd=9), -3), (dict(bd=3), -3),
    (dict(act=3), -1), (dict(act=-1), -1), (dict(ldx=504), -1), (dict(ldy=249), -1),
    (dict(ldr=249), -1), (dict(ldpre=249), -1), (dict(R=P, ldr=256), -1),
    (dict(ldx=(1 << 32) + 8), -1), (dict(ldy=(1 << 32) + 1), -1), (dict(ldr=(1 << 32) + 1), -1),
    (dict(ldpre=(1 << 32) + 1), -1), (dict(ldx=516), -4), (dict(packed=P + 8), -4),
    (dict(X=P + 8), -4), (dict(Y=P + 1), -4), (dict(Y=P + 2, yd=bw.MBOK_F32), -4),
    (dict(R=2 * P + 1), -4), (dict(bias=P + 2), -4), (dict(bias=P + 1, bd=bw.MBOK_BF16), -4),
    (dict(pre=P + 1), -4), (dict(T=17, ldx=1 << 23), -1),
]


@pytest.mark.parametrize("change,err", LINEAR)
@pytest.mark.parametrize("name", ["mbok_linear", "mbok_linear_precise"])
def test_linear_refuses(lib, name, change, err):
    base, _d = linear_args()
    assert call(getattr(lib, name), base, **change) == err


def backward_args():
    d = desc(m=250)
    return dict(d=ctypes.byref(d), packed=P, pre=P, ldpre=250, dY=2 * P, lddy=250, T=4, act=0,
                dpre=3 * P, lddpre=250, dbias=P, acc=0, dX=P, lddx=512, ws=None, s=None), d


@pytest.mark.parametrize("change,err", [
    (dict(d=None), -1), (dict(packed=None), -1), (dict(dY=None), -1), (dict(T=0), -2),
    (dict(T=bw.MBOK_MAX_T + 1), -2), (dict(lddy=249), -1), (dict(act=7), -1),
    (dict(pre=None), -1), (dict(dpre=None), -1), (dict(ldpre=249), -1), (dict(lddpre=249), -1),
    (dict(act=2), -1), (dict(act=2, pre=None), -1), (dict(act=2, dpre=None), -1),
    (dict(act=2, pre=None, dpre=None, dbias=None, dX=None), -1),
    (dict(dpre=P, lddpre=256), -1), (dict(dpre=2 * P, lddpre=256), -1), (dict(lddx=504), -1),
    (dict(lddx=516), -4), (dict(packed=P + 8), -4), (dict(pre=P + 1), -4), (dict(dY=P + 1), -4),
    (dict(dpre=P + 1), -4), (dict(dbias=P + 2), -4), (dict(dX=P + 8), -4), (dict(ws=P + 16), -4),
    (dict(lddy=(1 << 32) + 1), -1), (dict(lddx=(1 << 32) + 8), -1),
])
@pytest.mark.parametrize("name", ["mbok_linear_backward", "mbok_linear_backward_precise"])
def test_linear_backward_refuses(lib, name, change, err):
    base, _d = backward_args()
    assert call(getattr(lib, name), base, **change) == err


def test_linear_backward_workspace(lib):
    d = desc(4096, 4096, 2)
    fn = lib.mbok_linear_backward_workspace_bytes
    assert fn(None, 4) == 0 and fn(ctypes.byref(BAD_DESC), 4) == 0
    assert fn(ctypes.byref(d), 0) == 0 and fn(ctypes.byref(d), bw.MBOK_MAX_T + 1) == 0
    # whole rounds of the product: the sums of 94 slices of 44 rows for dbias alone
    assert bw.mbok_linear_backward_workspace_bytes(d, 4096) == 94 * 4096 * 4
    # beside the product's own: slices of 16 rows at least
    own = bw.mbok_gemmt_workspace_bytes(d, 64)
    assert own % 256 == 0
    assert bw.mbok_linear_backward_workspace_bytes(d, 64) == own + 4 * 4096 * 4
    # up to 32 rows are one slice: the product's workspace
    assert bw.mbok_linear_backward_workspace_bytes(d, 32) == bw.mbok_gemmt_workspace_bytes(d, 32)


def logp_args(backward):
    d = bw.mbok_logp_desc_init(1000, 2.0)
    a = dict(d=ctypes.byref(d), Z=P, zd=bw.MBOK_F32, T=4, ldz=1000, label=P)
    if backward:
        a.update(stats=P, dlogp=P, dZ=2 * P, dzd=bw.MBOK_BF16, lddz=1000, s=None)
    else:
        a.update(logp=P, stats=P, s=None)
    return a, d


BAD_LOGP = bw.mbok_logp_desc(vocab=0, temperature=1.0)
COLD_LOGP = bw.mbok_logp_desc(vocab=10, temperature=0.0)
ROWS = [
    (dict(d=None), -1), (dict(Z=None), -1), (dict(label=None), -1), (dict(T=0), -2),
    (dict(T=bw.MBOK_MAX_DISTILL_ROWS + 1), -2), (dict(ldz=999), -1), (dict(ldz=(1 << 32) + 1), -1),
    (dict(zd=3), -3), (dict(Z=P + 2), -4), (dict(label=P + 2), -4), (dict(stats=P + 4), -4),
]
GRAD = [(dict(lddz=999), -1), (dict(lddz=(1 << 32) + 1), -1), (dict(dzd=bw.MBOK_F16), -3),
        (dict(dZ=P), -1), (dict(dZ=2 * P + 1), -4)]


@pytest.mark.parametrize("change,err", ROWS + [
    (dict(logp=None), -1), (dict(logp=P + 2), -4), (dict(d=ctypes.byref(BAD_LOGP)), -2),
    (dict(d=ctypes.byref(COLD_LOGP)), -1)])
def test_logp_refuses(lib, change, err):
    base, _d = logp_args(False)
    assert call(lib.mbok_logp, base, **change) == err


@pytest.mark.parametrize("change,err", ROWS + GRAD + [
    (dict(stats=None), -1), (dict(dlogp=None), -1), (dict(dlogp=P + 1), -4), (dict(dZ=None), -1),
    (dict(d=ctypes.byref(BAD_LOGP)), -2)])
def test_logp_backward_refuses(lib, change, err):
    base, _d = logp_args(True)
    assert call(lib.mbok_logp_backward, base, **change) == err


def policy_args():
    d = bw.mbok_policy_desc_init(1000)
    return dict(d=ctypes.byref(d), Z=P, zd=bw.MBOK_F32, T=4, ldz=1000, label=P, adv=P, old=P,
                ref=P, w=P, loss=P, logp=P, stats=P, dlogp=P, dZ=2 * P, dzd=bw.MBOK_BF16,
                lddz=1000, s=None), d


BAD_POLICY = bw.mbok_policy_desc(vocab=10, temperature=1.0, clip_low=2.0, clip_high=0.1, kl=0.0)


@pytest.mark.parametrize("change,err", ROWS + GRAD + [
    (dict(adv=None), -1), (dict(loss=None), -1), (dict(d=ctypes.byref(BAD_POLICY)), -1)] + [
    ({k: P + 2}, -4) for k in ("adv", "old", "ref", "w", "loss", "logp", "dlogp")])
def test_policy_refuses(lib, change, err):
    base, _d = policy_args()
    assert call(lib.mbok_policy, base, **change) == err


@pytest.mark.parametrize("args,err", [
    ((0,), -2), ((bw.MBOK_MAX_VOCAB + 1,), -2), ((10, 0.0), -1), ((10, math.inf), -1),
    ((10, 1.0, -0.1), -1), ((10, 1.0, 1.1), -1), ((10, 1.0, math.nan), -1),
    ((10, 1.0, 0.2, -0.1), -1), ((10, 1.0, 0.2, math.nan), -1), ((10, 1.0, 0.2, 0.2, -1.0), -1),
    ((10, 1.0, 0.2, 0.2, math.inf), -1)])
def test_policy_desc_refuses(args, err):
    with pytest.raises(bw.MbokError) as e:
        bw.mbok_policy_desc_init(*args)
    assert e.value.status == err


def test_policy_desc_takes_no_upper_clip():
    assert bw.mbok_policy_desc_init(10, 1.0, 1.0, math.inf).clip_high == math.inf


@pytest.mark.parametrize("kw,err", [
    (dict(beta=0.0), -1), (dict(beta=-1.0), -1), (dict(beta=math.inf), -1),
    (dict(beta=0.1, smoothing=-0.1), -1), (dict(beta=0.1, smoothing=0.6), -1),
    (dict(beta=0.1, margin=math.nan), -1), (dict(beta=0.1, vocab=0), -2),
    (dict(beta=0.1, vocab=bw.MBOK_MAX_VOCAB + 1), -2)])
def test_preference_desc_refuses(kw, err):
    with pytest.raises(bw.MbokError) as e:
        bw.mbok_preference_desc_init(**kw)
    assert e.value.status == err


@pytest.mark.parametrize("change,err", [
    (dict(d=None), -1), (dict(off=None), -1), (dict(logp=None), -1), (dict(loss=None), -1),
    (dict(T=0), -2), (dict(T=bw.MBOK_MAX_DISTILL_ROWS + 1), -2), (dict(pairs=0), -2),
    (dict(pairs=bw.MBOK_MAX_PAIRS + 1), -2)] + [
    ({k: P + 2}, -4) for k in ("off", "logp", "ref", "label", "w", "loss", "dlogp")])
def test_preference_refuses(lib, change, err):
    d = bw.mbok_preference_desc_init(0.1)
    base = dict(d=ctypes.byref(d), off=P, pairs=2, logp=P, ref=P, label=P, T=8, w=P, loss=P,
                dlogp=P, s=None)
    assert call(lib.mbok_preference, base, **change) == err


# --------------------------------------------------------- the optimizer's plan

M = 1 << 20


def tensor(i=0, count=1000, **kw):
    """A tensor whose buffers are 1 MiB apart, 8 MiB from the next tensor's."""
    at = P + 8 * M * i
    t = bw._AdamwTensor()
    t.param, t.grad, t.m, t.v, t.count = at, at + M, at + 2 * M, at + 3 * M, count
    t.grad_dtype, t.state_dtype, t.out_dtype = bw.MBOK_F32, bw.MBOK_F32, bw.MBOK_BF16
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def init(lib, *tensors, n=None, plan=True, table=True):
    a = (bw._AdamwTensor * max(1, len(tensors)))(*tensors)
    n = len(tensors) if n is None else n
    size = lib.mbok_adamw_table_bytes(a, n)
    p, buf = bw._AdamwPlan(), ctypes.create_string_buffer(max(size, 16))
    st = lib.mbok_adamw_plan_init(ctypes.byref(p) if plan else None, a, n,
                                  ctypes.addressof(buf) if table else None)
    return st, p, size, buf


EIGHT = dict(state_dtype=bw.MBOK_E4M3, m_scale=P + 4 * M, v_scale=P + 5 * M)
LAYER = bw.mbok_desc_init(100, 256, 2, bw.MBOK_F16)  # 2 * 100 * 2 scales


@pytest.mark.parametrize("kw,err", [
    (dict(param=None), -1), (dict(grad=None), -1), (dict(m=None), -1), (dict(v=None), -1),
    (dict(count=0), -1), (dict(count=(1 << 32) + 1), -2), (dict(weight_decay=-0.1), -1),
    (dict(weight_decay=math.nan), -1), (dict(weight_decay=math.inf), -1),
    (dict(grad_dtype=3), -3), (dict(state_dtype=bw.MBOK_BF16), -3),
    (dict(m_scale=P + 4 * M), -1), (dict(EIGHT, v_scale=None), -1), (dict(EIGHT, m_scale=None), -1),
    (dict(param=P + 2), -4), (dict(grad=P + M + 2), -4), (dict(m=P + 2 * M + 2), -4),
    (dict(v=P + 3 * M + 1), -4), (dict(EIGHT, m_scale=P + 4 * M + 2), -4),
    (dict(out=P + 6 * M, out_dtype=3), -3), (dict(out=P + 6 * M + 1), -4),
    (dict(out=P + 6 * M + 2, out_dtype=bw.MBOK_F32), -4),
    (dict(layer=ctypes.addressof(LAYER), count=400), -1),
    (dict(layer=ctypes.addressof(LAYER), count=399, out=P + 6 * M), -2),
    (dict(layer=ctypes.addressof(LAYER), count=400, out=P + 6 * M + 8), -4),
    (dict(layer=ctypes.addressof(BAD_DESC), count=400, out=P + 6 * M), -2),
    # what a step writes may meet nothing else that it writes or reads
    (dict(m=P), -1), (dict(m=P + 3996), -1), (dict(v=P + 2 * M), -1), (dict(out=P + 4 * 999), -1),
    (dict(grad=P), -1), (dict(grad=P + 3 * M + 4 * 999), -1), (dict(EIGHT, v_scale=P + 4 * M), -1),
])
def test_adamw_plan_refuses(lib, kw, err):
    st, _p, size, _b = init(lib, tensor(**kw))
    assert st == err and size == 0


def test_adamw_plan_refuses_sets(lib):
    assert init(lib, n=0)[0] == -2
    assert init(lib, tensor(), plan=False)[0] == -1
    assert init(lib, tensor(), table=False)[0] == -1
    a = (bw._AdamwTensor * 1)(tensor())
    assert lib.mbok_adamw_table_bytes(a, bw.MBOK_MAX_ADAMW_TENSORS + 1) == 0
    assert lib.mbok_adamw_table_bytes(None, 1) == 0
    # the same tensor twice, a state of one that is another's, a gradient of one
    # that is another's parameter; two gradients may be the same
    assert init(lib, tensor(0), tensor(0))[0] == -1
    assert init(lib, tensor(0), tensor(1, v=P + 2 * M + 400))[0] == -1
    assert init(lib, tensor(0), tensor(1, grad=P))[0] == -1
    assert init(lib, tensor(0), tensor(1, grad=P + M))[0] == 0
    # neighbours
    assert init(lib, tensor(0), tensor(1, param=P + 4000))[0] == 0


@pytest.mark.parametrize("counts", [(1,), (1024, 1025), (256, 5000, 3, 70000), (1 << 23, 7)])
def test_adamw_table_covers_every_value_once(lib, counts):
    at, items = P, []
    for c in counts:  # buffers one after the other
        t = tensor(count=c)
        for k in ("param", "grad", "m", "v"):
            setattr(t, k, at)
            at += 4 * c
        items.append(t)
    st, p, size, buf = init(lib, *items)
    assert st == 0 and p.table_bytes == size and p.tensors == len(counts) and p.lds_bytes == 0
    head = (size - 16 * p.parts) // len(counts)
    parts = np.frombuffer(buf, dtype=np.dtype([("start", "<i8"), ("tensor", "<i4"),
                                               ("len", "<i4")]),
                          count=p.parts, offset=head * len(counts))
    for i, c in enumerate(counts):
        mine = parts[parts["tensor"] == i]
        assert mine["start"][0] == 0 and (mine["start"] % bw.MBOK_ADAMW_BLOCK == 0).all()
        assert (mine["start"][1:] == mine["start"][:-1] + mine["len"][:-1]).all()
        assert mine["start"][-1] + mine["len"][-1] == c and (mine["len"] > 0).all()
        assert (mine["len"] <= 4096).all()


STEP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, grad_scale=1.0, seed=0)


@pytest.mark.parametrize("kw", [
    dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=math.nan),
    dict(beta2=1.0), dict(beta2=math.nan), dict(eps=0.0), dict(eps=-1e-8), dict(eps=1e-39),
    dict(eps=math.nan), dict(eps=1e39), dict(step=0), dict(step=-3), dict(step=1 << 53),
    dict(grad_scale=math.nan)])
def test_adamw_refuses_constants(lib, kw):
    st, p, _s, _b = init(lib, tensor())
    s = bw._AdamwStep(**dict(STEP, **kw))
    assert lib.mbok_adamw(ctypes.byref(p), P, ctypes.byref(s), None, None) == -1


def test_adamw_refuses_calls(lib):
    _st, p, _s, _b = init(lib, tensor())
    s, R = bw._AdamwStep(**STEP), ctypes.byref
    assert lib.mbok_adamw(None, P, R(s), None, None) == -1
    assert lib.mbok_adamw(R(p), None, R(s), None, None) == -1
    assert lib.mbok_adamw(R(p), P, None, None, None) == -1
    assert lib.mbok_adamw(R(p), P + 8, R(s), None, None) == -4
    assert lib.mbok_adamw(R(p), P, R(s), P + 2, None) == -4
    for field, value in (("tensors", 0), ("parts", 0), ("parts", 5), ("table_bytes", 8),
                         ("lds_bytes", -1), ("lds_bytes", 1 << 20)):
        q = bw._AdamwPlan(p.table_bytes, p.tensors, p.parts, p.lds_bytes)
        setattr(q, field, value)
        assert lib.mbok_adamw(R(q), P, R(s), None, None) == -1, field


# ----------------------------------------------------------------- the binding

def test_binding_refuses_host_tensors():
    x, f, i = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(4), torch.zeros(4).int()
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_linear(desc(), x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_linear_backward(desc(), x, x, dX=x)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_logp(bw.mbok_logp_desc_init(512), x, i, f)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_policy(bw.mbok_policy_desc_init(512), x, i, f, f)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_preference(bw.mbok_preference_desc_init(0.1), i[:3], f, f)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_adamw_plan_init([dict(param=f, grad=f, m=f, v=f)])
    with pytest.raises(ValueError):
        bw.mbok_adamw_plan_init([])
    with pytest.raises(ValueError, match="missing"):
        bw.mbok_adamw_plan_init([dict(grad=f)])
    with pytest.raises(TypeError):
        bw.mbok_adamw(None, 1e-3, 1)


def test_reference_act_is_the_gated_blocks():
    z = torch.linspace(-4, 4, 9, dtype=F64)
    assert torch.equal(ref.act("gelu", z), finetune_ref.act("gelu", z))
    assert torch.equal(ref.act("none", z), z)
