"""GPU tests of the policy loss on rows that hold no numbers: what the formula gives
in float64, not-a-number and infinities included."""
import math

import pytest
import torch

import boolean_weight_amd as bw
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def broken_rows(V, dtype, T=7):
    """Rows 0 to 2 have no log-probability (a NaN, a +inf, -inf alone); the others do."""
    gen = torch.Generator().manual_seed(V)
    Z = torch.randn(T, V, generator=gen).to(dtype)
    Z[0, V // 2] = NAN
    Z[1, V - 1] = INF
    Z[2] = -INF
    return Z.to(DEV), torch.full((T,), 1, dtype=torch.int32, device=DEV)


def outputs(T, Z):
    return dict(loss=torch.full((T,), -5.0, device=DEV), dlogp=torch.full((T,), -5.0, device=DEV),
                dZ=torch.full_like(Z, -7.0))


# vocabularies of the register forms of few and of many rows, and past them
@pytest.mark.parametrize("T,V", [(7, 40), (600, 9000), (7, 140003)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("advantage", [1.5, 0.0, -2.0])
@pytest.mark.parametrize("with_ref", [False, True])
def test_broken_rows_without_old_logp(T, V, dtype, advantage, with_ref):
    """exp(logp - logp) of a NaN is NaN: loss, slope and gradient say so, and no other
    row does."""
    say(f"policy broken rows T={T} V={V} {dtype} A={advantage} ref={with_ref}")
    Z, label = broken_rows(V, dtype, T)
    A = torch.full((T,), advantage, device=DEV)
    out = outputs(T, Z)
    ref = torch.full((T,), -3.0, device=DEV) if with_ref else None
    bw.mbok_policy(bw.mbok_policy_desc_init(V, kl=0.1), Z, label, A, ref_logp=ref, **out)
    for name, x in out.items():
        bad = torch.isnan(x.float()).view(T, -1)
        assert bad[:3].all(), name
        assert torch.isfinite(x.float()).view(T, -1)[3:].all(), name
    if not with_ref:  # a ratio of 1
        assert (out["loss"][3:] == -advantage).all() and (out["dlogp"][3:] == -advantage).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_old", [False, True])
def test_no_kl_term_at_weight_zero(dtype, with_old):
    """With kl = 0 there is no KL term, whatever the reference model's values are: the
    bits of the call without them."""
    say(f"policy kl=0 {dtype} old={with_old}")
    T, V = 8, 50
    gen = torch.Generator().manual_seed(3)
    Z = torch.randn(T, V, generator=gen).to(dtype)
    Z[1, 1] = -INF  # the row's token: logp -inf
    Z, label = Z.to(DEV), torch.full((T,), 1, dtype=torch.int32, device=DEV)
    A = torch.tensor([1.0, 1.0, -1.0, 0.0, 2.0, -2.0, 1.0, 1.0], device=DEV)
    old = torch.full((T,), -4.0, device=DEV) if with_old else None
    ref = torch.tensor([-INF, -2.0, 2000.0, NAN, INF, -1e30, 3e38, 0.0], device=DEV)
    d = bw.mbok_policy_desc_init(V, kl=0.0)
    got, want = outputs(T, Z), outputs(T, Z)
    bw.mbok_policy(d, Z, label, A, old_logp=old, ref_logp=ref, **got)
    bw.mbok_policy(d, Z, label, A, old_logp=old, **want)
    for name in got:
        assert torch.isfinite(got[name].float()).all(), name
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_old", [False, True])
def test_kl_term_of_a_masked_token(dtype, with_old):
    """x = ref - logp: exp(x) - x - 1 grows without bound both ways.  A token at -inf that
    the reference model finds possible costs +inf, with slope -inf; one that both rule out
    has no x (NaN); one that only the reference rules out costs +inf too, with slope beta
    beside the ratio's."""
    say(f"policy token at -inf {dtype} old={with_old}")
    T, V, kl = 6, 50, 0.25
    gen = torch.Generator().manual_seed(4)
    Z = torch.randn(T, V, generator=gen).to(dtype)
    Z[:3, 1] = -INF
    Z, label = Z.to(DEV), torch.full((T,), 1, dtype=torch.int32, device=DEV)
    A = torch.ones(T, device=DEV)
    # the ratio of a masked token is 0, or 1 without old_logp
    old = torch.full((T,), -4.0, device=DEV) if with_old else None
    ref = torch.tensor([-2.0, -1e4, -INF, -INF, 2000.0, -3.0], device=DEV)
    out = outputs(T, Z)
    logp = torch.empty(T, device=DEV)
    bw.mbok_policy(bw.mbok_policy_desc_init(V, clip_high=INF, kl=kl), Z, label, A, old_logp=old,
                   ref_logp=ref, logp=logp, **out)
    loss, slope, lp = out["loss"].cpu(), out["dlogp"].cpu(), logp.cpu().double()
    assert (lp[:3] == -INF).all() and torch.isfinite(lp[3:]).all()
    assert (loss[:2] == INF).all() and (slope[:2] == -INF).all()
    assert torch.isnan(loss[2]) and torch.isnan(slope[2])
    assert loss[3] == INF and loss[4] == INF and slope[4] == -INF
    r = (lp + 4.0).exp() if with_old else torch.ones(T, dtype=torch.float64)
    # logp's 2^-16 (see test_gpu_policy.py) in a slope of |r A| <= e^4 and in x
    tol = 2.0 ** -15 * (r[3] + 1)
    assert abs(float(slope[3]) - float(kl - r[3])) <= tol
    x = -3.0 - float(lp[5])
    want = -float(r[5]) + kl * (math.expm1(x) - x)
    assert abs(float(loss[5]) - want) <= 2.0 ** -15 * (float(r[5]) + kl * (math.exp(x) + 1))
