"""The distillation loss and gradient where the teacher's masses do not add to
1, are not numbers, or lie where the student has next to nothing, against the
float64 definition, in one pass and as two calls.

Tolerances, with eps = 2^-24 (the fp32 half step):
  loss  log S and the logarithms of the listed entries are off by at most 2^-17
        (a row's exponentials are summed in fp32, at most 128 terms each),
        every p by 2^-22 relative, and the teacher's rest, 1 less a sum, by
        2^-22 absolute; so by w tau^2 mass (2^-16 + 2^-20 spread), spread being
        the largest |log p - log q| and mass the sum of the teacher's masses.
  dZ    2^-16 of the magnitudes a value is the difference of (the reference's
        `size`), then one rounding: eps_t / 2 relative, or half the smallest
        step (fp16 2^-25; below the smallest normal value fp32 and bf16
        results may be flushed).
"""
import math

import pytest
import torch

import boolean_weight_amd as bw
import distill_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MODES = ("step", "pair")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def dev(x):
    return None if x is None else x.to(DEV)


def run(Z, l, idx, tau, lse=None, w=None, mode="step", dloss=None, grad=None):
    T, V = Z.shape
    d = bw.mbok_distill_desc_init(V, l.shape[1], tau)
    args = [dev(Z), dev(l), dev(idx.to(torch.int32))]
    kw = dict(t_lse=dev(lse), weight=dev(w))
    loss = torch.full((T,), -5.0, device=DEV)
    dZ = torch.full((T, V), -7.0, dtype=grad or Z.dtype, device=DEV)
    if mode == "step":
        bw.mbok_distill(d, *args, loss, dZ=dZ, **kw)
    else:
        stats = torch.full((T, bw.MBOK_DISTILL_STATS), math.nan, device=DEV)
        bw.mbok_distill(d, *args, loss, stats=stats, **kw)
        dl = torch.ones(T, device=DEV) if dloss is None else dev(dloss)
        bw.mbok_distill_backward(d, *args, stats, dl, dZ, **kw)
    return loss.cpu(), dZ.cpu()


def check(Z, l, idx, tau, lse=None, w=None, grad=None, modes=MODES):
    T = Z.shape[0]
    for mode in modes:
        dloss = torch.linspace(0.5, 2.0, T) if mode == "pair" else None
        loss, dZ = run(Z, l, idx, tau, lse, w, mode, dloss, grad)
        want, grads, size = ref.distill(Z, l, idx, tau, lse, w, dloss)
        assert torch.equal(torch.isnan(loss), torch.isnan(want)), (mode, loss, want)
        wt = torch.ones(T, dtype=F64) if w is None else w.to(F64).abs()
        for t in range(T):
            if math.isnan(float(want[t])) or float(wt[t]) == 0.0:
                continue
            row = ref.masses(Z.shape[1], l[t], idx[t], tau, None if lse is None else lse[t])
            if row is None:
                assert float(loss[t]) == 0.0
                continue
            x = Z[t].to(F64) / tau
            spread = float((x.max() - x[x > -math.inf].min())) + math.log(Z.shape[1]) + \
                float(row[2][row[1] > 0].abs().max() if bool((row[1] > 0).any()) else 0.0)
            mass = max(1.0, float(row[1].sum()))
            tol = float(wt[t]) * tau * tau * mass * (2.0 ** -16 + 2.0 ** -20 * spread)
            assert abs(float(loss[t]) - float(want[t])) <= tol, (mode, t, loss[t], want[t], tol)
        assert torch.equal(torch.isnan(dZ), torch.isnan(grads)), mode
        info = torch.finfo(dZ.dtype)
        least = 2.0 ** -25 if dZ.dtype == torch.float16 else info.smallest_normal
        tol = 2.0 ** -16 * size + info.eps / 2 * grads.abs() + least
        off = (dZ.to(F64) - grads).abs()
        ok = (off <= tol) | torch.isnan(grads)
        assert ok.all(), (mode, (off - tol).nan_to_num(-1.0).max(), off.nan_to_num(0).max())


def inputs(T, V, top, seed, z="f32", scale=2.5):
    gen = torch.Generator().manual_seed(seed)
    teacher = torch.randn(T, V, generator=gen) * scale
    Z = (teacher + torch.randn(T, V, generator=gen)).to(TYPES[z])
    l, idx = teacher.topk(top, -1)
    return Z, l.contiguous(), idx, teacher


@pytest.mark.parametrize("z,grad", [("f32", "f32"), ("bf16", "bf16"), ("f16", "bf16")])
@pytest.mark.parametrize("V,top", [(17, 8), (1000, 20), (33001, 64)])
def test_masses_that_do_not_add_to_one(z, grad, V, top):
    """A likely index listed twice and three times (more than 1), a log-sum that
    is too small (more than 1) and too large (a larger rest)."""
    say(f"distill masses V={V} top={top} {z}->{grad}")
    Z, l, idx, teacher = inputs(5, V, top, 3 * V, z)
    for t, j in ((0, 1), (1, 1), (1, 2), (4, top - 1)):
        idx[t, j], l[t, j] = idx[t, 0], l[t, 0]
    for tau in (1.0, 2.0):
        lse = torch.logsumexp(teacher / tau, -1) + torch.tensor([0.0, 0.0, -0.5, 0.5, -0.1])
        check(Z, l, idx, tau, lse, grad=TYPES[grad])
        check(Z, l, idx, tau, grad=TYPES[grad])


def test_everything_unlisted_masked():
    """Nothing is left for the teacher's rest: q_r is 0 and its class drops out,
    so the row's masses add to less than 1 (and to nothing in the last row)."""
    for z in ("f32", "bf16"):
        say(f"distill unlisted masked {z}")
        Z, l, idx, teacher = inputs(4, 300, 6, 21, z)
        for t in range(4):
            free = torch.ones(300, dtype=torch.bool)
            free[idx[t]] = False
            Z[t, free] = -math.inf
        lse = torch.logsumexp(teacher, -1)
        l[3, :] = -math.inf
        w = torch.tensor([1.0, 0.25, 3.0, 1.0])
        check(Z, l, idx, 1.0, lse, w)


def test_differences_with_a_repeated_token():
    """dZ against central differences of the call's own loss, masses above 1.
    With h = 2^-5 the third derivative (below 2) leaves h^2 / 6 2 < 4e-4, and
    the fp32 loss (below 8, off by 2^-18) adds 2^-18 / h = 2^-13."""
    say("distill differences")
    V, h = 40, 2.0 ** -5
    Z, l, idx, teacher = inputs(1, V, 5, 9, scale=1.0)
    idx[0, 1], l[0, 1] = idx[0, 0], l[0, 0]
    lse = torch.logsumexp(teacher, -1) - 1.0
    many = Z.repeat(2 * V, 1)
    for v in range(V):
        many[2 * v, v] += h
        many[2 * v + 1, v] -= h
    loss, _ = run(many, l.repeat(2 * V, 1), idx.repeat(2 * V, 1), 1.0, lse.repeat(2 * V))
    diff = (loss.to(F64).view(V, 2) @ torch.tensor([1.0, -1.0], dtype=F64)) / (2 * h)
    for mode in MODES:
        dZ = run(Z, l, idx, 1.0, lse, mode=mode)[1][0].to(F64)
        assert (diff - dZ).abs().max() < 6e-4


@pytest.mark.parametrize("rest", [False, True])
def test_teacher_logits_that_are_no_numbers(rest):
    """NaN or +inf among the listed teacher logits (an overflowed fp16 row): loss
    and gradient of the row are NaN, beside entries of -inf too, and of that row
    only; not where the entry is not there or the row has no weight."""
    for z, td in (("f32", "f32"), ("bf16", "f16"), ("f16", "bf16")):
        say(f"distill teacher non-finite {z} teacher {td} rest={rest}")
        Z, l, idx, teacher = inputs(9, 300, 6, 22, z)
        l = l.to(TYPES[td])
        l[0, 3] = math.nan
        l[1, 0] = math.inf
        l[2, 2] = l[2, 4] = math.inf
        l[3, :] = -math.inf
        l[3, 5] = math.nan
        l[4, :] = math.nan
        l[5, 1] = math.nan
        idx[5, 1] = -1
        l[6, :] = math.nan
        idx[6, :] = 300
        l[7, 0] = math.nan
        lse = torch.logsumexp(teacher, -1) if rest else None
        w = torch.tensor([1.0] * 7 + [0.0, 2.0])
        check(Z, l, idx, 1.0, lse, w)
        loss, dZ = run(Z, l, idx, 1.0, lse, w)
        assert torch.isnan(loss).tolist() == [True] * 5 + [False] * 4
        assert torch.isnan(dZ[:5]).all() and not torch.isnan(dZ[5:]).any()
        if not rest:
            assert float(loss[6]) == 0.0 and not dZ[6].any()
        assert float(loss[7]) == 0.0 and not dZ[7].any()


@pytest.mark.parametrize("gap", [60.0, 85.0, 87.0, 88.0, 90.0, 200.0, 1000.0])
def test_rest_far_below_the_listed(gap):
    """Everything unlisted lies `gap` tau below the listed tokens, where its
    exponentials relative to the largest logit leave fp32: the teacher's rest
    keeps its term, and its gradient stays w tau p_r at most."""
    for z, grad, V, top in (("f32", "f32", 1000, 12), ("bf16", "bf16", 1000, 12),
                            ("f32", "bf16", 33001, 64), ("bf16", "bf16", 140003, 7)):
        for tau, w in ((1.0, 1.0), (0.5, 65536.0), (4.0, 65536.0)):
            say(f"distill gap={gap} V={V} {z}->{grad} tau={tau} w={w}")
            T = 3
            Z, l, idx, _ = inputs(T, V, top, 17, "f32", scale=1.0)
            idx[2, 1], l[2, 1] = idx[2, 0], l[2, 0]
            up = torch.zeros(T, V).scatter_(1, idx, gap * tau)
            Z = (Z + up).to(TYPES[z])
            lse = torch.logsumexp(l / tau, -1) - math.log(0.9)
            check(Z, l, idx, tau, lse, torch.full((T,), w), TYPES[grad])


def test_rest_far_below_with_bad_values():
    """NaN and +inf among the listed, among the unlisted far below, and rows of
    only -inf with and without listed entries."""
    say("distill gap bad values")
    T, V = 8, 700
    Z, l, idx, _ = inputs(T, V, 9, 18)
    Z.scatter_add_(1, idx, torch.full((T, 9), 150.0))
    free = [v for v in range(V) if all(v not in idx[t].tolist() for t in range(T))][5]
    Z[0, free] = math.nan
    Z[1, free] = math.inf
    Z[2, int(idx[2, 4])] = math.nan
    Z[3, int(idx[3, 4])] = math.inf
    Z[4, :] = -math.inf
    Z[5, :] = -math.inf
    idx[5, :] = -1
    Z[6, free] = -math.inf
    idx[7, :] = -1
    lse = torch.logsumexp(l, -1) + 0.2
    check(Z, l, idx, 1.0, lse)


def test_smallest_temperature():
    """tau = 2^-126: all of q is on the largest logit."""
    say("distill smallest temperature")
    Z, l, idx, _ = inputs(3, 100, 5, 2)
    Z[0, 50] = Z[0].max() + 1.0  # zero shifted logits and others
    Z[1] -= Z[1].max()
    tau = 2.0 ** -126
    l = l / 20  # below 0.5; the largest entry's log-sum is exact
    l[:, 0] = 0.5
    for lse in (None, torch.full((3,), 0.5 / tau)):
        for mode in MODES:
            loss, dZ = run(Z, l, idx, tau, lse, mode=mode)
            assert torch.isfinite(loss).all() and torch.isfinite(dZ).all()
            assert (dZ.abs() <= 2.0 ** -125).all()


@pytest.mark.parametrize("z", ["f32", "bf16"])
@pytest.mark.parametrize("V", [131072, 262144, bw.MBOK_MAX_VOCAB])
def test_small_terms_beside_a_large_one(V, z):
    """Each 1 in the sum is followed by terms just below half its step: a thread
    that adds n of them in fp32 loses up to n 2^-24 of S.  With 128 at most log S
    is off by 2^-17, the exponentials by 2^-23, log2(e) / tau by 2^-24 log V and
    the loss's rounding by 2^-24 of a value below 16."""
    say(f"distill small terms V={V} {z}")
    Z = torch.full((1, V), math.log(0.97 * 2.0 ** -24)).to(TYPES[z])
    # the first 1024 vectors of 16 bytes hold one logit of 0 each
    Z[0, :1024 * (4 if z == "f32" else 8):4 if z == "f32" else 8] = 0.0
    l, idx = torch.zeros(1, 1), torch.zeros(1, 1, dtype=torch.int64)
    want = float(torch.logsumexp(Z[0].to(F64), 0))
    for lse in (None, torch.zeros(1)):
        loss, _ = run(Z, l, idx, 1.0, lse)
        assert abs(float(loss) - want) <= 2.0 ** -17 + 2.0 ** -23 + 13.2 * 2.0 ** -24 + 2.0 ** -20


@pytest.mark.parametrize("shift", [-5.0e4, -300.0, 0.0, 2.0e4])
def test_unlisted_masked_far_from_zero(shift):
    """Nothing unlisted is left and the listed logits lie anywhere: no factor of
    what is not there gets into the row."""
    for z, grad in (("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")):
        say(f"distill unlisted masked at {shift} {z}->{grad}")
        Z, l, idx, teacher = inputs(3, 300, 6, 25, "f32")
        Z = (Z + shift).to(TYPES[z])
        for t in range(3):
            free = torch.ones(300, dtype=torch.bool)
            free[idx[t]] = False
            Z[t, free] = -math.inf
        check(Z, l, idx, 1.0, torch.logsumexp(teacher, -1), grad=TYPES[grad])
        check(Z, l, idx, 0.25, torch.logsumexp(teacher * 4, -1) - 0.5, grad=TYPES[grad])


@pytest.mark.parametrize("gap", [15.0, 20.0, 20.8, 25.0, 30.0])
def test_rest_around_the_second_sum(gap):
    """On both sides of the unlisted share from which its sum is taken again."""
    for z, grad, V in (("f32", "f32", 1000), ("bf16", "bf16", 33001), ("f32", "bf16", 140003)):
        say(f"distill gap={gap} V={V} {z}->{grad}")
        Z, l, idx, _ = inputs(4, V, 12, 19, "f32", scale=1.0)
        Z = (Z + torch.zeros(4, V).scatter_(1, idx, gap + math.log(V))).to(TYPES[z])
        lse = torch.logsumexp(l, -1) - math.log(0.95)
        check(Z, l, idx, 1.0, lse, torch.full((4,), 100.0), TYPES[grad])
