"""GPU tests of the optimizer step's constants that are read on the device."""
import math

import pytest
import torch

import boolean_weight_amd as bw
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def tensors(eight, seed=5, count=3000):
    """A flat tensor and a layer's scales."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    d = bw.mbok_desc_init(70, 256, 2, bw.MBOK_F16)
    out = []
    for n in (count, 2 * 70 * 2):
        t = dict(param=torch.randn(n, generator=gen, device=DEV),
                 grad=torch.randn(n, generator=gen, device=DEV))
        if eight:
            blocks = (n + bw.MBOK_ADAMW_BLOCK - 1) // bw.MBOK_ADAMW_BLOCK
            for k in "mv":
                t[k] = torch.rand(n, generator=gen, device=DEV).to(torch.float8_e4m3fn)
                t[k + "_scale"] = torch.full((blocks,), 2.0 ** -6, device=DEV)
        else:
            t["m"] = torch.randn(n, generator=gen, device=DEV)
            t["v"] = torch.rand(n, generator=gen, device=DEV)
        out.append(t)
    out[0]["out"] = torch.full((count,), -5.0, dtype=torch.bfloat16, device=DEV)
    out[1].update(layer=d, out=torch.full((bw.mbok_packed_bytes(d),), 0x5A, dtype=torch.uint8,
                                          device=DEV))
    return out


def bits(ts):
    return [x.clone().view(torch.uint8) for t in ts for x in t.values()
            if isinstance(x, torch.Tensor)]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("t", [0.0, -0.0, -3.0, 0.5, math.nan, -math.inf])
def test_no_step_before_the_first(eight, t):
    """The bias corrections divide by 1 - beta^t: a count below 1, as a zeroed buffer
    holds it, is no step, and nothing is written.  1 is the first step, as by the host's
    constants."""
    say(f"adamw live t={t} eight={eight}")
    ts = tensors(eight)
    plan, before = bw.mbok_adamw_plan_init(ts), bits(ts)
    live = torch.tensor([1e-3, 1.0, t, 0.0], device=DEV)
    bw.mbok_adamw(plan, lr=1e-3, step=1, live=live, seed=2)
    assert all(torch.equal(a, b) for a, b in zip(before, bits(ts)))
    live[2] = 1.0
    bw.mbok_adamw(plan, lr=7.0, step=9, live=live, seed=2)
    other = tensors(eight)
    bw.mbok_adamw(bw.mbok_adamw_plan_init(other), lr=float(live[0]), step=1, seed=2)
    assert all(torch.equal(a, b) for a, b in zip(bits(other), bits(ts)))
    assert all(torch.isfinite(t["param"]).all() for t in ts)
