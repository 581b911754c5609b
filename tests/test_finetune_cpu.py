"""The fine-tuning operators on the CPU: the references' gradients against
differences, and every refusal of the C ABI (no call here reaches a kernel)."""
import ctypes
import math

import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref as ref

F64 = torch.float64
P = 1 << 20  # a "pointer" that is never read: 1 MiB aligned


# ------------------------------------------------- gradients by differences
# Central differences of a smooth function: the error is h^2/6 times the third
# derivative plus the rounding 2^-52 |f| / h; with h = 1e-4 and values and
# derivatives of order 1 to 10 both stay below 1e-6.

def differences(f, x, h=1e-4):
    out = torch.zeros_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        o[i] = (up - f()) / (2 * h)
        flat[i] = keep
    return out


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradient_is_the_slope(kind):
    gen = torch.Generator().manual_seed(5)
    T, m, n, K = 2, 3, 128, 2
    layers = []
    for _ in range(2):
        S = torch.randint(0, 2, (K, m, n), generator=gen) * 2 - 1
        layers.append((S, torch.rand(K, m, 1, generator=gen, dtype=F64) * 0.05))
    X = torch.randn(T, n, generator=gen, dtype=F64)
    R = torch.randn(T, m, generator=gen, dtype=F64)  # gradient of H
    Wg, Wu = (ref.dense(*x) for x in layers)

    def loss():
        return float((R * ref.act(kind, X @ ref.dense(*layers[0]).t()) *
                      (X @ ref.dense(*layers[1]).t())).sum())

    g, u = X @ Wg.t(), X @ Wu.t()
    dg, du = R * u * ref.act_slope(kind, g), R * ref.act(kind, g)
    assert torch.allclose(differences(loss, X), dg @ Wg + du @ Wu, rtol=0, atol=1e-6)
    for (S, A), d in zip(layers, (dg, du)):
        assert torch.allclose(differences(loss, A), ref.scale_grad(S, d, X), rtol=0, atol=1e-5)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_gradient_is_the_slope(rest, tau):
    gen = torch.Generator().manual_seed(8)
    T, V = 3, 11
    Z = torch.randn(T, V, generator=gen, dtype=F64)
    teacher = torch.randn(T, V, generator=gen, dtype=F64)
    idx = torch.tensor([[3, 0, 7, 3], [1, -1, 2, 40], [5, 6, 9, 10]])
    l = teacher.gather(1, idx.clamp(0, V - 1))
    lse = torch.logsumexp(teacher / tau, 1) + 0.3 if rest else None
    w = torch.tensor([1.0, 0.5, 2.0])

    def loss():
        return float(ref.distill(Z, l, idx, tau, lse, w)[0].sum())

    assert torch.allclose(differences(loss, Z), ref.distill(Z, l, idx, tau, lse, w)[1], rtol=0,
                          atol=1e-6)


def test_distill_of_the_teacher_itself_is_zero():
    Z = torch.randn(2, 9, dtype=F64)
    idx = torch.arange(9).repeat(2, 1)
    loss, dZ = ref.distill(Z, Z, idx, 2.0)
    assert float(loss.abs().max()) < 1e-14 and float(dZ.abs().max()) < 1e-14


# ----------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    return bw.load_library()


def desc(m=256, n=512, K=2):
    return bw.mbok_desc_init(m, n, K, bw.MBOK_F16)


BAD_DESC = bw.mbok_desc(m=4, n=100, K=1, group=128, alpha_dtype=1, layout=1)


def call(fn, base, **change):
    args = dict(base, **change)
    return fn(*args.values())


def gemmt_args():
    d = desc()
    return dict(d=ctypes.byref(d), packed=P, dY=P, T=4, lddy=256, dX=P, lddx=512, ws=None, s=None,
                ), d


@pytest.mark.parametrize("change,err", [
    (dict(d=None), -1), (dict(packed=None), -1), (dict(dY=None), -1), (dict(dX=None), -1),
    (dict(T=0), -2), (dict(T=bw.MBOK_MAX_T + 1), -2), (dict(lddy=255), -1), (dict(lddx=511), -1),
    (dict(lddy=(1 << 32) + 1), -1), (dict(lddx=516), -4), (dict(packed=P + 8), -4),
    (dict(dY=P + 1), -4), (dict(dX=P + 2), -4), (dict(ws=P + 16), -4),
])
def test_gemmt_refuses(lib, change, err):
    base, _d = gemmt_args()
    assert call(lib.mbok_gemmt, base, **change) == err


def scale_grad_args():
    d = desc()
    return dict(d=ctypes.byref(d), packed=P, dY=P, T=4, lddy=256, X=P, ldx=512, out=P, acc=0,
                ws=None, s=None), d


@pytest.mark.parametrize("change,err", [
    (dict(d=None), -1), (dict(packed=None), -1), (dict(dY=None), -1), (dict(X=None), -1),
    (dict(out=None), -1), (dict(T=0), -2), (dict(T=bw.MBOK_MAX_T + 1), -2), (dict(lddy=255), -1),
    (dict(ldx=504), -1), (dict(ldx=516), -4), (dict(packed=P + 8), -4), (dict(dY=P + 1), -4),
    (dict(X=P + 8), -4), (dict(out=P + 2), -4), (dict(ws=P + 16), -4),
])
def test_scale_grad_refuses(lib, change, err):
    base, _d = scale_grad_args()
    assert call(lib.mbok_scale_grad, base, **change) == err


def gated_args():
    d = desc(m=250)
    return dict(d=ctypes.byref(d), packed=P, X=P, xd=bw.MBOK_BF16, T=4, ldx=512, act=0, H=P,
                ldh=250, pre=P, ldpre=512, s=None), d


@pytest.mark.parametrize("change,err", [
    (dict(d=None), -1), (dict(packed=None), -1), (dict(X=None), -1), (dict(H=None), -1),
    (dict(T=0), -2), (dict(T=bw.MBOK_MAX_T + 1), -2), (dict(xd=bw.MBOK_F32), -3),
    (dict(act=2), -1), (dict(act=-1), -1), (dict(ldx=504), -1), (dict(ldh=249), -1),
    (dict(ldpre=504), -1), (dict(ldpre=516), -4), (dict(ldx=516), -4), (dict(packed=P + 8), -4),
    (dict(X=P + 8), -4), (dict(H=P + 1), -4), (dict(pre=P + 8), -4),
])
def test_gated_refuses(lib, change, err):
    base, _d = gated_args()
    assert call(lib.mbok_gated, base, **change) == err


def gated_backward_args():
    d = desc(m=250)
    return dict(d=ctypes.byref(d), packed=P, pre=P, ldpre=512, dH=P, lddh=250, T=4, act=0,
                dpre=2 * P, lddpre=512, dX=P, lddx=512, ws=None, s=None), d


@pytest.mark.parametrize("change,err", [
    (dict(d=None), -1), (dict(packed=None), -1), (dict(pre=None), -1), (dict(dH=None), -1),
    (dict(dpre=None), -1), (dict(T=0), -2), (dict(T=bw.MBOK_MAX_T + 1), -2), (dict(act=7), -1),
    (dict(ldpre=504), -1), (dict(lddpre=504), -1), (dict(lddh=249), -1), (dict(lddx=504), -1),
    (dict(dpre=P, lddpre=520), -1), (dict(ldpre=516), -4), (dict(lddpre=516), -4),
    (dict(lddx=516), -4), (dict(pre=P + 8), -4), (dict(dpre=P + 8), -4), (dict(dH=P + 1), -4),
    (dict(dX=P + 2), -4), (dict(ws=P + 16), -4),
])
def test_gated_backward_refuses(lib, change, err):
    base, _d = gated_backward_args()
    assert call(lib.mbok_gated_backward, base, **change) == err


def test_gated_backward_refuses_more_than_a_launch(lib):
    m = 1 << 19
    d = bw.mbok_desc_init(m, 512, 1, bw.MBOK_F16)
    base, _d = gated_backward_args()
    assert call(lib.mbok_gated_backward, base, d=ctypes.byref(d), T=bw.MBOK_MAX_T, lddh=m,
                ldpre=2 * m, lddpre=2 * m) == -2


@pytest.mark.parametrize("change,err", [
    (dict(d=None), -1), (dict(sg=None), -1), (dict(ag=None), -1), (dict(su=None), -1),
    (dict(au=None), -1), (dict(packed=None), -1), (dict(sg=P + 8), -4), (dict(ag=P + 8), -4),
    (dict(su=P + 8), -4), (dict(au=P + 8), -4), (dict(packed=P + 8), -4),
    (dict(d=ctypes.byref(BAD_DESC)), -2),
])
def test_gated_pack_refuses(lib, change, err):
    d = desc()
    base = dict(d=ctypes.byref(d), sg=P, ag=P, su=P, au=P, packed=P, s=None)
    assert call(lib.mbok_gated_pack, base, **change) == err


def test_gated_stack(lib):
    for m, rows in ((1, 16), (8, 16), (9, 32), (1001, 2016), (11008, 22016)):
        s = bw.mbok_gated_stack(bw.mbok_desc_init(m, 256, 3, bw.MBOK_F32))
        assert (s.m, s.n, s.K, s.alpha_dtype) == (rows, 256, 3, bw.MBOK_F32)
    with pytest.raises(bw.MbokError) as e:
        bw.mbok_gated_stack(bw.mbok_desc_init((1 << 23) + 1, 128, 1))
    assert e.value.status == -2
    d = desc()
    assert lib.mbok_gated_stack(ctypes.byref(d), None) == -1


def distill_args(backward):
    d = bw.mbok_distill_desc_init(1000, 16, 2.0)
    a = dict(d=ctypes.byref(d), Z=P, zd=bw.MBOK_F32, T=4, ldz=1000, l=P, td=bw.MBOK_F16, idx=P,
             ldt=16, lse=P, w=P)
    if backward:
        a.update(stats=P, dloss=P)
    else:
        a.update(loss=P, stats=P)
    a.update(dZ=2 * P, dzd=bw.MBOK_BF16, lddz=1000, s=None)
    return a, d


COMMON = [
    (dict(d=None), -1), (dict(Z=None), -1), (dict(l=None), -1), (dict(idx=None), -1),
    (dict(T=0), -2), (dict(T=bw.MBOK_MAX_DISTILL_ROWS + 1), -2), (dict(ldz=999), -1),
    (dict(ldt=15), -1), (dict(lddz=999), -1), (dict(zd=5), -3), (dict(td=-1), -3),
    (dict(dzd=bw.MBOK_F16), -3), (dict(dZ=P), -1), (dict(Z=P + 2), -4), (dict(l=P + 1), -4),
    (dict(idx=P + 2), -4), (dict(lse=P + 2), -4), (dict(w=P + 2), -4), (dict(dZ=P + 1), -4),
    (dict(stats=P + 4), -4),
]


@pytest.mark.parametrize("change,err", COMMON + [(dict(loss=None), -1), (dict(loss=P + 2), -4)])
def test_distill_refuses(lib, change, err):
    base, _d = distill_args(False)
    assert call(lib.mbok_distill, base, **change) == err


@pytest.mark.parametrize("change,err", COMMON + [(dict(stats=None), -1), (dict(dloss=None), -1),
                                                 (dict(dloss=P + 2), -4)])
def test_distill_backward_refuses(lib, change, err):
    base, _d = distill_args(True)
    assert call(lib.mbok_distill_backward, base, **change) == err


def test_distill_backward_needs_dz(lib):
    base, _d = distill_args(True)
    assert call(lib.mbok_distill_backward, base, dZ=None) == -1


@pytest.mark.parametrize("V,top,tau,err", [
    (0, 1, 1.0, -2), (bw.MBOK_MAX_VOCAB + 1, 1, 1.0, -2), (10, 0, 1.0, -2),
    (10, bw.MBOK_MAX_TOP + 1, 1.0, -2), (10, 4, 0.0, -1), (10, 4, -1.0, -1),
    (10, 4, math.inf, -1), (10, 4, math.nan, -1),
])
def test_distill_desc_refuses(V, top, tau, err):
    with pytest.raises(bw.MbokError) as e:
        bw.mbok_distill_desc_init(V, top, tau)
    assert e.value.status == err


def test_workspace_bytes(lib):
    d = desc(4096, 4096, 2)
    for fn in (lib.mbok_gemmt_workspace_bytes, lib.mbok_scale_grad_workspace_bytes):
        assert fn(None, 4) == 0
        assert fn(ctypes.byref(BAD_DESC), 4) == 0
        assert fn(ctypes.byref(d), 0) == 0
        assert fn(ctypes.byref(d), bw.MBOK_MAX_T + 1) == 0
    # few tokens: several slices of every 256-column tile's sums; many: of the
    # tiles past whole rounds; whole rounds: none
    assert bw.mbok_gemmt_workspace_bytes(d, 16) == 16 * 16 * (16 * 256 * 4)
    assert bw.mbok_gemmt_workspace_bytes(d, 4096 + 256) == 16 * 16 * (256 * 256 * 4)
    assert bw.mbok_gemmt_workspace_bytes(d, 4096) == 0


def test_binding_refuses_host_tensors():
    d = desc()
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_gemmt(d, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_gated(d, x, x, x)
    with pytest.raises(TypeError):
        bw.mbok_scale_grad(d, x, None, x, x)
    with pytest.raises(ValueError, match="GPU"):
        bw.mbok_distill(bw.mbok_distill_desc_init(8, 2), x, x, x, x)
