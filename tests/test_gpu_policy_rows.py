"""GPU tests of the row kernel's forms for 512 rows or more against float64, and of the
correction that the rows' sums carry.

Tolerances: see test_gpu_policy.py; those of the correction stand at its test."""
import math

import pytest
import torch

import boolean_weight_amd as bw
import step_ref as ref
from gpu_util import DEV, say
from test_gpu_policy import TYPES, check_dz, dev, inputs

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


# 256, 512 and 1024 threads with 2, 4, 8 and 16 vectors each, and rows that are read again
# (those in one type)
ROWS = [(T, V, z, grad) for z, grad in (("bf16", "same"), ("f16", "same"), ("f32", "same"),
                                        ("f16", "bf16"), ("f32", "bf16"))
        for T, V in ((600, 300), (520, 1500), (513, 9000), (600, 20000), (512, 32000),
                     (513, 40009), (512, 70000))] + [(512, 140003, "f32", "same")]


@pytest.mark.parametrize("T,V,z,grad", ROWS)
@pytest.mark.parametrize("aligned", [True, False])
def test_many_rows_by_value(T, V, z, grad, aligned):
    """Loss, log-probability, slope and gradient of a sample of rows; what lies between
    the rows stays."""
    say(f"policy many rows T={T} V={V} {z} grad={grad} aligned={aligned}")
    tau, pad = 1.25, (-V) % 8 + (8 if aligned else 3)
    off = 8 if aligned else 1
    gen = torch.Generator(device=DEV).manual_seed(T + V)
    out = TYPES[z] if grad == "same" else torch.bfloat16
    zbuf = torch.full((T, V + off + pad), math.nan, dtype=TYPES[z], device=DEV)
    gbuf = torch.full((T, V + off + pad), -7.0, dtype=out, device=DEV)
    Z, dZ = zbuf[:, off:off + V], gbuf[:, off:off + V]
    Z.copy_(2.5 * torch.randn(T, V, generator=gen, device=DEV))
    label = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    label[::11] = -1
    # the sampled tokens' ratios on both sides of both borders; some likely tokens
    rows = torch.arange(0, T, max(1, T * V // (1 << 21)))[:64]
    rows = torch.cat([rows, torch.tensor([T - 2, T - 1])]).unique()
    label[rows[::3].to(DEV)] = Z[rows[::3].to(DEV)].float().argmax(-1).int()
    Zs, labels = Z[rows.to(DEV)].cpu(), label[rows.to(DEV)].cpu()
    lp, _ = ref.logp(Zs, labels, tau)
    g = torch.Generator().manual_seed(V)
    ratio = torch.tensor([0.4, 0.75, 0.85, 1.0, 1.15, 1.25, 3.0], dtype=F64)[
        torch.arange(len(rows)) % 7]
    A, w = torch.randn(T, generator=g), torch.rand(T, generator=g) + 0.5
    old, refl = (-8 + torch.randn(T, generator=g) for _ in range(2))
    old[rows] = (lp - ratio.log()).float()
    refl[rows] = (lp + 0.5 * torch.randn(len(rows), generator=g, dtype=F64)).float()
    d = bw.mbok_policy_desc_init(V, tau, 0.2, 0.28, 0.05)
    loss, logp, dlogp = (torch.full((T,), -5.0, device=DEV) for _ in range(3))
    stats = torch.full((T, bw.MBOK_LOGP_STATS), math.nan, device=DEV)
    bw.mbok_policy(d, Z, label, dev(A), loss, old_logp=dev(old), ref_logp=dev(refl),
                   weight=dev(w), logp=logp, stats=stats, dlogp=dlogp, dZ=dZ)
    want, slope, size = ref.policy(lp, labels, V, A[rows], old[rows], refl[rows], w[rows],
                                   float(d.clip_low), float(d.clip_high), float(d.kl))
    D = 2.0 ** -16 + 2.0 ** -22 * lp.abs()

    def sample(x):
        return x[rows.to(DEV)].cpu().to(F64)

    assert ((sample(logp) - lp).abs() <= D).all()
    assert ((sample(loss) - want).abs() <= 2 * D * size + 2.0 ** -23 * want.abs()).all()
    assert ((sample(dlogp) - slope).abs() <= 2 * D * size + 2.0 ** -23 * slope.abs()).all()
    check_dz(dZ[rows.to(DEV)], Zs, labels, tau, slope, size, D)
    assert (gbuf[:, :off] == -7).all() and (gbuf[:, off + V:] == -7).all()
    # and the gradient from the statistics, in its own kernel; log-probabilities alone
    gbuf.fill_(-7.0)
    dl = bw.mbok_logp_desc_init(V, tau)
    bw.mbok_logp_backward(dl, Z, label, stats, dlogp, dZ)
    check_dz(dZ[rows.to(DEV)], Zs, labels, tau, slope, size, D)
    assert (gbuf[:, :off] == -7).all() and (gbuf[:, off + V:] == -7).all()
    alone = torch.full((T,), -5.0, device=DEV)
    bw.mbok_logp(dl, Z, label, alone)
    assert torch.equal(alone, logp)


@pytest.mark.parametrize("T,V", [(700, 40), (20, 40), (3, 140003)])
@pytest.mark.parametrize("tau", [1.0, 0.5])
def test_sums_carry_their_correction(T, V, tau):
    """Exponentials take z c - k, c = fl(log2 e / tau) and k = fl(zmax c): with k in 128
    .. 256 its rounding is up to 2^-17, the row's log-sum off by ln 2 times that, and put
    back.  Without that the log-probability would be off by `fix`.

    What stays, relative to the sum, eps = 2^-24: the arguments' own fma and c's rounding,
    2 |a| ln 2 eps for |a| <= 4 (the logits lie within 2 tau of the largest), 5.6 eps;
    exp2's 2 eps; at most 3 sums in fp32 (a thread's vector of 4; more are in float64), 3
    eps; rounded to fp32, eps |logp|.  16 eps + eps |logp| with some room."""
    say(f"logp correction T={T} V={V} tau={tau}")
    gen = torch.Generator().manual_seed(T + V)
    c = float(torch.tensor(1 / math.log(2) / tau, dtype=torch.float32))
    # largest logits whose k is rounded by 0.4 of its step or more
    top = (128 + 127 * torch.rand(200000, generator=gen, dtype=F64)) / c
    top = top.float()
    exact = top.double() * c
    fix = math.log(2) * ((top * torch.tensor(c, dtype=torch.float32)).double() - exact)
    pick = ((fix / math.log(2)).abs() >= 0.4 * 2.0 ** -16).nonzero()[:T, 0]
    assert len(pick) == T
    top, fix = top[pick], fix[pick]
    Z = top[:, None] - (2 * tau) * torch.rand(T, V, generator=gen)
    Z[:, V // 3] = top
    label = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32)
    logp = torch.empty(T, device=DEV)
    bw.mbok_logp(bw.mbok_logp_desc_init(V, tau), dev(Z), dev(label), logp)
    want, q = ref.logp(Z, label, tau)
    tol = 2.0 ** -24 * (16 + want.abs())
    # twice the tolerance apart, a value is within it of one of them only: leaving the
    # correction out, or taking it twice, is seen
    assert (fix.abs() > 2 * tol).all()
    got = logp.cpu().to(F64)
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()
    assert ((got - (want + fix)).abs() > tol).all()
    assert ((got - (want - fix)).abs() > tol).all()
    # the gradient's q needs none: numerator and sum are short of the same factor.
    # e 7.6 eps and the sum 10.6, as above, and 4 roundings: below 24 eps of q
    stats, dZ = torch.empty(T, 4, device=DEV), torch.empty(T, V, device=DEV)
    dl, up = bw.mbok_logp_desc_init(V, tau), torch.ones(T)
    bw.mbok_logp(dl, dev(Z), dev(label), logp, stats=stats)
    bw.mbok_logp_backward(dl, dev(Z), dev(label), stats, dev(up), dZ)
    want = ref.logp_grad(Z, label, tau, up)
    assert ((dZ.cpu().to(F64) - want).abs() <= 2.0 ** -24 * 24 * (q / tau + want.abs())).all()
