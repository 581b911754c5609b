"""GPU parity of the row log-probabilities, their gradient, the policy loss and
the preference loss, through the C ABI, against float64.

Tolerances (eps = 2^-24): as for the distillation loss (test_gpu_distill.py) a
row's log-sum is off by at most 2^-16 and q by 2^-16 relative.  So with D = 2^-16
+ 2 eps |logp|, a ratio or exp(ref - logp) by 2 D relative, a loss by 2 D times the
terms of its slope (|r A| + beta (e^x + 1)) w, and dlogp too; dZ = dlogp / tau
(onehot - q) by 2^-16 q |dlogp| / tau + 2 D times those terms, plus half a step of the
gradient's type, or half its smallest step near zero.
"""
import math

import pytest
import torch

import boolean_weight_amd as bw
import step_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def dev(x):
    return None if x is None else x.to(DEV)


def inputs(T, V, z, seed, scale=2.5):
    gen = torch.Generator().manual_seed(seed)
    Z = (torch.randn(T, V, generator=gen) * scale).to(TYPES[z])
    label = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32)
    return Z, label, gen


def small(info):
    return info.smallest_normal + (2.0 ** -25 if info.dtype == "float16" else 0.0)


def check_dz(got, Z, label, tau, dlogp, size, D):
    """size: the sum of the absolute terms of dlogp."""
    want = ref.logp_grad(Z, label, tau, dlogp)
    _, q = ref.logp(Z, label, tau)
    near = (ref.onehot(label, Z.shape[1]) - q).abs()
    info = torch.finfo(got.dtype)
    tol = (2.0 ** -16 * q * dlogp.abs()[:, None] + 2 * D[:, None] * size[:, None] * near) / tau + \
        info.eps / 2 * want.abs() + small(info)
    bad = (got.cpu().to(F64) - want).abs() > tol
    assert not bad.any(), ((got.cpu().to(F64) - want).abs() - tol).max()


# vocabularies around the vector width, each number of threads and vectors per
# thread, and past what the registers hold
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 63), (4, 513), (3, 2049), (2, 4097), (3, 8200), (2, 17000),
          (2, 33001), (1, 70001), (1, 140003), (1, bw.MBOK_MAX_VOCAB)]


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("z", ["bf16", "f16", "f32"])
def test_logp_and_gradient(T, V, z):
    for tau, grad in ((1.0, "same"), (0.7, "bf16")):
        say(f"logp T={T} V={V} {z} tau={tau} grad={grad}")
        Z, label, gen = inputs(T, V, z, T + V)
        label[T // 2] = V - 1
        d = bw.mbok_logp_desc_init(V, tau)
        off = 3  # rows at any element
        buf = torch.full((T, V + 5), NAN, dtype=Z.dtype, device=DEV)
        Zd = buf[:, off:off + V]
        Zd.copy_(Z)
        logp = torch.full((T + 2,), -5.0, device=DEV)
        stats = torch.full((T, bw.MBOK_LOGP_STATS), NAN, device=DEV)
        bw.mbok_logp(d, Zd, dev(label), logp[1:-1], stats=stats)
        # (tau as the descriptor holds it)
        t32 = float(torch.tensor(tau, dtype=torch.float32))
        want, _ = ref.logp(Z, label, t32)
        D = 2.0 ** -16 + 2.0 ** -23 * want.abs()
        assert ((logp[1:-1].cpu().to(F64) - want).abs() <= D).all()
        assert logp[0] == -5 and logp[-1] == -5
        plain = torch.empty(T, device=DEV)
        bw.mbok_logp(d, Zd, dev(label), plain)
        assert torch.equal(plain, logp[1:-1])
        up = torch.randn(T, generator=gen)
        dt = Z.dtype if grad == "same" else torch.bfloat16
        dbuf = torch.full((T, V + 3), -7.0, dtype=dt, device=DEV)
        dZ = dbuf[:, 1:1 + V]
        bw.mbok_logp_backward(d, Zd, dev(label), stats, dev(up), dZ)
        check_dz(dZ, Z, label, t32, up.to(F64), up.to(F64).abs(), D)
        assert (dbuf[:, 0] == -7).all() and (dbuf[:, 1 + V:] == -7).all()
        if grad == "same":  # in place
            bw.mbok_logp_backward(d, Zd, dev(label), stats, dev(up), Zd)
            assert torch.equal(Zd, dZ)


@pytest.mark.parametrize("T", [600, 1100])
@pytest.mark.parametrize("V", [300, 1500, 9000, 20000])
def test_many_rows(T, V):
    """The forms for 512 rows or more against those for few, row by row."""
    say(f"logp many rows T={T} V={V}")
    Z, label, gen = inputs(T, V, "bf16", V)
    label[::7] = -1
    d = bw.mbok_policy_desc_init(V, kl=0.1)
    lp, _ = ref.logp(Z[:8], label[:8], 1.0)
    adv, old = torch.randn(T, generator=gen), -8 + torch.randn(T, generator=gen)
    old[:8] = lp + 0.1

    def run(rows):
        n = len(range(*rows.indices(T)))
        loss, dZ = torch.empty(n, device=DEV), torch.empty(n, V, dtype=Z.dtype, device=DEV)
        bw.mbok_policy(d, dev(Z[rows]), dev(label[rows]), dev(adv[rows]), loss,
                       old_logp=dev(old[rows]), ref_logp=dev(old[rows]), dZ=dZ)
        return loss, dZ

    loss, dZ = run(slice(0, T))
    for at in (0, T // 2, T - 5):
        l, g = run(slice(at, at + 5))
        # sums in another order: both within the bound of the reference
        want_l = l.cpu().to(F64)
        size = (adv[at:at + 5].abs().to(F64) * 40 + want_l.abs() + 1)
        assert ((loss[at:at + 5].cpu().to(F64) - want_l).abs() <= 2.0 ** -13 * size).all()
        assert torch.equal(dZ[at:at + 5] == 0, g == 0)


def policy_case(T, V, z, seed, tau):
    """Ratios on both sides of both borders and away from them."""
    Z, label, gen = inputs(T, V, z, seed)
    lp, _ = ref.logp(Z, label, tau)
    ratio = torch.tensor([0.4, 0.75, 0.85, 1.0, 1.15, 1.25, 3.0])[torch.arange(T) % 7]
    A = torch.randn(T, generator=gen)
    A[torch.arange(T) % 5 == 4] = 0.0
    old = (lp - ratio.to(F64).log()).float()
    refl = (lp + 0.5 * torch.randn(T, generator=gen, dtype=F64)).float()
    w = torch.rand(T, generator=gen) + 0.5
    if T > 3:
        label[1], label[2] = -1, V
        w[3] = 0.0
    return Z, label, A, old, refl, w


@pytest.mark.parametrize("T,V", [(1, 50), (14, 1000), (35, 4097), (7, 33001), (2, 140003)])
@pytest.mark.parametrize("z", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("with_old,with_ref", [(True, True), (True, False), (False, True)])
def test_policy(T, V, z, with_old, with_ref):
    say(f"policy T={T} V={V} {z} old={with_old} ref={with_ref}")
    tau = 1.5
    Z, label, A, old, refl, w = policy_case(T, V, z, T + V, tau)
    old, refl = old if with_old else None, refl if with_ref else None
    d = bw.mbok_policy_desc_init(V, tau, 0.2, 0.28, 0.05)
    low, high, kl = (float(v) for v in (d.clip_low, d.clip_high, d.kl))
    loss, logp, dlogp = (torch.full((T,), -5.0, device=DEV) for _ in range(3))
    stats = torch.full((T, bw.MBOK_LOGP_STATS), NAN, device=DEV)
    dZ = torch.full((T, V), -7.0, dtype=Z.dtype, device=DEV)
    kw = dict(old_logp=dev(old), ref_logp=dev(refl), weight=dev(w))
    bw.mbok_policy(d, dev(Z), dev(label), dev(A), loss, logp=logp, stats=stats, dlogp=dlogp,
                   dZ=dZ, **kw)
    lp, _ = ref.logp(Z, label, tau)
    want, slope, size = ref.policy(lp, label, V, A, old, refl, w, low, high, kl)
    D = 2.0 ** -16 + 2.0 ** -22 * lp.abs()
    assert ((logp.cpu().to(F64) - lp).abs() <= D).all()
    assert ((loss.cpu().to(F64) - want).abs() <= 2 * D * size + 2.0 ** -23 * want.abs()).all()
    assert ((dlogp.cpu().to(F64) - slope).abs() <= 2 * D * size + 2.0 ** -23 * slope.abs()).all()
    check_dz(dZ, Z, label, tau, slope, size, D)
    # the loss alone; the gradient later, from statistics and dlogp; in place
    alone = torch.empty_like(loss)
    bw.mbok_policy(d, dev(Z), dev(label), dev(A), alone, **kw)
    assert torch.equal(alone, loss)
    later = torch.full_like(dZ, -7.0)
    dl = bw.mbok_logp_desc_init(V, tau)
    bw.mbok_logp_backward(dl, dev(Z), dev(label), stats, dlogp, later)
    check_dz(later, Z, label, tau, slope, size, D)
    Zd = dev(Z)
    bw.mbok_policy(d, Zd, dev(label), dev(A), alone, dZ=Zd, **kw)
    assert torch.equal(Zd, dZ) and torch.equal(alone, loss)


def test_policy_borders_and_extremes():
    """Ratios that overflow or vanish, advantages of 0, infinite clips."""
    say("policy extremes")
    V = 40
    Z, label, _ = inputs(6, V, "f32", 3)
    lp, _ = ref.logp(Z, label, 1.0)
    old = lp.float() - torch.tensor([200.0, -800.0, 800.0, 800.0, 0.0, 5.0])
    A = torch.tensor([1.0, -1.0, 0.0, -1.0, 0.0, 1.0])
    loss, dlogp = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    dZ = torch.empty(6, V, device=DEV)
    d = bw.mbok_policy_desc_init(V, clip_low=0.2, clip_high=0.25)
    bw.mbok_policy(d, dev(Z), dev(label), dev(A), loss, old_logp=dev(old), dlogp=dlogp, dZ=dZ)
    got, sl = loss.cpu(), dlogp.cpu()
    assert got[0] == -1.25 and sl[0] == 0 and (dZ[0] == 0).all()          # clipped above
    assert abs(float(got[1]) - 0.8) < 1e-6 and sl[1] == 0                  # clipped below
    assert got[2] == 0 and sl[2] == 0                                       # no advantage
    assert got[3] == INF and sl[3] == INF                                   # -r A, unbounded
    assert got[4] == 0 and (dZ[4] == 0).all()
    assert got[5] == -1.25
    d = bw.mbok_policy_desc_init(V, clip_low=1.0, clip_high=INF)
    bw.mbok_policy(d, dev(Z), dev(label), dev(A), loss, old_logp=dev(old), dlogp=dlogp)
    assert abs(float(loss[5]) + math.exp(5)) <= 2.0 ** -14 * math.exp(5)


@pytest.mark.parametrize("z", ["bf16", "f32"])
def test_rows_that_hold_no_numbers(z):
    """NaN, infinities and rows of -inf; masked logits of -inf and of the type's
    lowest value cost nothing; rows without a token are not read."""
    say(f"logp non-finite {z}")
    V, T = 700, 9
    Z, label, _ = inputs(T, V, z, 5)
    low = torch.finfo(Z.dtype).min
    label[:] = 10
    Z[0, 3] = NAN
    Z[1, 3] = INF
    Z[2] = -INF
    Z[3, 50:] = -INF
    Z[4, 50:] = low
    Z[5, 10] = -INF
    Z[6] = NAN
    label[6] = -3
    Z[7] = low
    Z[8] = 0.0
    d = bw.mbok_logp_desc_init(V)
    logp, up = torch.empty(T, device=DEV), torch.ones(T, device=DEV)
    stats, dZ = torch.empty(T, 4, device=DEV), torch.empty(T, V, dtype=Z.dtype, device=DEV)
    bw.mbok_logp(d, dev(Z), dev(label), logp, stats=stats)
    bw.mbok_logp_backward(d, dev(Z), dev(label), stats, up, dZ)
    got, g = logp.cpu(), dZ.cpu().to(F64)
    assert torch.isnan(got[:3]).all() and torch.isnan(g[:3]).all()
    want, q = ref.logp(Z[3:5], label[3:5], 1.0)
    assert ((got[3:5].to(F64) - want).abs() <= 2.0 ** -16 + 2.0 ** -22 * want.abs()).all()
    assert (g[3:5, 50:] == 0).all()
    assert got[5] == -INF and got[6] == 0 and (g[6] == 0).all()
    assert ((got[7:].to(F64) + math.log(V)).abs() <= 2.0 ** -15).all()
    # a weight of 0 hides a row that holds no numbers
    loss = torch.empty(T, device=DEV)
    w = torch.zeros(T, device=DEV)
    bw.mbok_policy(bw.mbok_policy_desc_init(V, kl=0.1), dev(Z), dev(label), up, loss, weight=w,
                   ref_logp=up, dZ=dZ, logp=logp)
    assert (loss == 0).all() and (dZ == 0).all()


def test_far_logits():
    """Largest logits of 1e4 and 3e38 beside near ones: the subtracted form."""
    say("logp far logits")
    V = 600
    for top in (1e4, 3e38, -1e4, -3e38):
        Z = torch.full((2, V), top, dtype=torch.float32)
        Z[1] -= torch.arange(V, dtype=torch.float32) * (abs(top) * 2.0 ** -22)
        label = torch.tensor([5, 2], dtype=torch.int32)
        logp = torch.empty(2, device=DEV)
        bw.mbok_logp(bw.mbok_logp_desc_init(V), dev(Z), dev(label), logp)
        want, _ = ref.logp(Z, label, 1.0)
        assert ((logp.cpu().to(F64) - want).abs() <= 2.0 ** -15 + 2.0 ** -22 * want.abs()).all()


PREF = [dict(), dict(smoothing=0.1), dict(margin=0.5), dict(mean=True), dict(beta=2.0, mean=True,
                                                                             smoothing=0.3)]


@pytest.mark.parametrize("kw", PREF)
@pytest.mark.parametrize("T,pairs", [(1, 1), (2, 1), (37, 1), (500, 7), (3000, 2), (40, 33)])
def test_preference(kw, T, pairs):
    """fp32 inputs, float64 sums: loss and dlogp round once (2^-24), the constants
    enter as the descriptor holds them; 2^-40 for the float64 functions."""
    say(f"preference T={T} pairs={pairs} {kw}")
    gen = torch.Generator().manual_seed(T + pairs)
    lp, refl = (-4 * torch.rand(T, generator=gen) for _ in range(2))
    label = torch.randint(-1, 5, (T,), generator=gen, dtype=torch.int32)
    off = torch.randint(0, T + 1, (2 * pairs + 1,), generator=gen).sort().values.int()
    w = torch.rand(pairs, generator=gen) + 0.1
    w[0] = 0.0 if pairs > 2 else 1.0
    d = bw.mbok_preference_desc_init(kw.get("beta", 0.1), kw.get("smoothing", 0.0),
                                     kw.get("margin", 0.0), kw.get("mean", False), vocab=4)
    loss, dlogp = torch.full((pairs,), -5.0, device=DEV), torch.full((T,), -7.0, device=DEV)
    bw.mbok_preference(d, dev(off), dev(lp), loss, ref_logp=dev(refl), label=dev(label),
                       weight=dev(w), dlogp=dlogp)
    want, slope = ref.preference(lp, off, label, refl, w, float(d.beta), float(d.smoothing),
                                 float(d.margin), bool(d.mean), V=4)
    r = 2.0 ** -23
    assert ((loss.cpu().to(F64) - want).abs() <= r * want.abs() + 2.0 ** -40).all()
    outside = torch.isnan(slope)
    got = dlogp.cpu().to(F64)
    assert (got[outside] == -7).all()  # rows of no sequence are left as they were
    assert ((got - slope).abs() <= r * slope.abs() + 2.0 ** -40)[~outside].all()
    bare = torch.empty_like(loss)
    bw.mbok_preference(d, dev(off), dev(lp), bare)
    want0, _ = ref.preference(lp, off, beta=float(d.beta), smoothing=float(d.smoothing),
                              margin=float(d.margin), mean=bool(d.mean))
    assert ((bare.cpu().to(F64) - want0).abs() <= r * want0.abs() + 2.0 ** -40).all()


def test_preference_offsets_out_of_range_read_nothing_outside():
    say("preference bad offsets")
    T = 10
    lp = torch.arange(T, dtype=torch.float32)
    d = bw.mbok_preference_desc_init(0.1)
    loss, dlogp = torch.empty(2, device=DEV), torch.full((T,), -7.0, device=DEV)
    off = torch.tensor([-5, 3, 100, 2, 1 << 30], dtype=torch.int32)
    bw.mbok_preference(d, dev(off), dev(lp), loss, dlogp=dlogp)
    # read as 0 3 10 and (cut to 10) 10 10 10
    want, slope = ref.preference(lp, [0, 3, 10], beta=float(d.beta))
    assert abs(float(loss[0]) - float(want[0])) <= 1e-6 * float(want[0])
    assert abs(float(loss[1]) - math.log(2)) <= 1e-7
    assert ((dlogp.cpu().to(F64) - slope).abs() <= 1e-8).all()


def test_preference_far_apart():
    """|h| of thousands: no overflow, the exact limits; a NaN reaches its pair alone."""
    say("preference extremes")
    lp = torch.tensor([0.0, -1e6, -1e6, 0.0, NAN, 0.0])
    off = torch.tensor([0, 1, 2, 3, 4, 5, 6], dtype=torch.int32)
    loss, dlogp = torch.empty(3, device=DEV), torch.empty(6, device=DEV)
    d = bw.mbok_preference_desc_init(1.0)
    bw.mbok_preference(d, dev(off), dev(lp), loss, dlogp=dlogp)
    assert loss[0] == 0 and loss[1] == 1e6 and torch.isnan(loss[2])
    g = dlogp.cpu()
    assert (g[:2] == 0).all() and g[2] == -1 and g[3] == 1 and torch.isnan(g[4:]).all()


def test_preference_step_by_differences():
    """logits -> logp -> pair loss -> dlogp -> dZ against differences of the whole
    chain in float64 (the kernels' fp32 results are too coarse to difference): the
    reference's gradient, which the CPU tests difference, in one place."""
    say("preference step")
    T, V, pairs, tau = 24, 300, 3, 1.0
    Z, label, gen = inputs(T, V, "f32", 11)
    label[::5] = -1
    off = torch.tensor([0, 4, 9, 9, 15, 20, 24], dtype=torch.int32)
    lp, _ = ref.logp(Z, label, tau)
    refl = (lp + 0.4 * torch.randn(T, generator=gen, dtype=F64)).float()
    d, dp = bw.mbok_logp_desc_init(V), bw.mbok_preference_desc_init(0.3, 0.1)
    logp, dlogp, loss = (torch.zeros(n, device=DEV) for n in (T, T, pairs))
    stats, dZ = torch.empty(T, 4, device=DEV), torch.empty(T, V, device=DEV)
    bw.mbok_logp(d, dev(Z), dev(label), logp, stats=stats)
    bw.mbok_preference(dp, dev(off), logp, loss, ref_logp=dev(refl), label=dev(label),
                       dlogp=dlogp)
    bw.mbok_logp_backward(d, dev(Z), dev(label), stats, dlogp, dZ)
    want, slope = ref.preference(lp, off, label, refl, beta=float(dp.beta),
                                 smoothing=float(dp.smoothing))
    # a score is off by at most 8 D, h by 0.3 of that and two scores
    D = 2.0 ** -16 + 2.0 ** -22 * lp.abs()
    assert ((loss.cpu().to(F64) - want).abs() <= 0.3 * 16 * D.max() + 2.0 ** -22).all()
    check_dz(dZ, Z, label, tau, slope, torch.full((T,), 0.3 * 6, dtype=F64), D)
