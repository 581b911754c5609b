"""The distillation reference's gradient against differences of its own loss,
for teacher masses that add to 1, to less and to more, on the CPU."""
import math

import pytest
import torch

import distill_ref as ref

F64 = torch.float64


def differences(Z, l, idx, tau, lse, h=1e-4):
    """Central differences of each row's loss: h^2 / 6 times a third derivative
    below 10 plus 2^-52 of a loss below 100 over h, together below 1e-7."""
    out = torch.zeros_like(Z)
    for t in range(Z.shape[0]):
        for v in range(Z.shape[1]):
            f = []
            for s in (h, -h):
                z = Z[t].clone()
                z[v] += s
                f.append(ref.distill_row(z, l[t], idx[t], tau, None if lse is None else lse[t])[0])
            out[t, v] = (f[0] - f[1]) / (2 * h)
    return out


@pytest.mark.parametrize("tau", [1.0, 2.5])
@pytest.mark.parametrize("shift", [None, 0.3, 0.0, -0.4])
def test_gradient_is_the_slope(tau, shift):
    gen = torch.Generator().manual_seed(8)
    T, V = 4, 11
    Z = torch.randn(T, V, generator=gen, dtype=F64)
    teacher = torch.randn(T, V, generator=gen, dtype=F64)
    # a repeated likely token, missing entries, distinct tokens, most tokens twice
    idx = torch.tensor([[3, 0, 7, 3, -1, -1, -1, -1, -1, -1, -1, -1],
                        [1, -1, 2, 40, -1, -1, -1, -1, -1, -1, -1, -1],
                        [5, 6, 9, 10, 0, -1, -1, -1, -1, -1, -1, -1],
                        [0, 1, 2, 3, 4, 5, 0, 1, 2, 3, 4, 5]])
    l = teacher.gather(1, idx.clamp(0, V - 1))
    lse = None if shift is None else torch.logsumexp(teacher / tau, 1) + shift
    _, dZ, size = ref.distill(Z, l, idx, tau, lse)
    assert torch.allclose(differences(Z, l, idx, tau, lse), dZ, rtol=0, atol=1e-6)
    assert (size >= dZ.abs() - 1e-15).all()


def test_gradient_with_everything_unlisted_masked():
    """No class is left for the teacher's rest: what is listed carries less than 1."""
    gen = torch.Generator().manual_seed(4)
    V = 9
    Z = torch.randn(1, V, generator=gen, dtype=F64)
    idx = torch.tensor([[2, 5, 7]])
    teacher = torch.randn(1, V, generator=gen, dtype=F64)
    free = [v for v in range(V) if v not in (2, 5, 7)]
    Z[0, free] = -math.inf
    l, lse = teacher.gather(1, idx), torch.logsumexp(teacher, 1)
    dZ = ref.distill(Z, l, idx, 1.0, lse)[1]
    diff = differences(Z, l, idx, 1.0, lse)
    assert torch.allclose(diff[0, idx[0]], dZ[0, idx[0]], rtol=0, atol=1e-6)
    assert not dZ[0, free].any()
    assert abs(float(dZ.sum())) < 1e-12  # q and the masses cancel over the row


def test_teacher_logits_that_are_no_numbers():
    Z = torch.zeros(1, 4, dtype=F64)
    idx = torch.tensor([[0, 2]])
    for lse in (None, torch.tensor([1.0])):
        for bad in ((math.nan, 0.0), (math.inf, 0.0), (math.inf, math.inf), (-math.inf, math.nan)):
            loss, dZ, _ = ref.distill(Z, torch.tensor([bad]), idx, 1.0, lse)
            assert torch.isnan(loss).all() and torch.isnan(dZ).all()
    loss, dZ, _ = ref.distill(Z, torch.tensor([[-math.inf, -math.inf]]), idx, 1.0)
    assert float(loss) == 0.0 and not dZ.any()
