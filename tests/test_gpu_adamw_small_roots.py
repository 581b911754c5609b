"""GPU test of how far down the 8-bit second moment's roots are kept from 0."""
import pytest
import torch

import boolean_weight_amd as bw
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

B = bw.MBOK_ADAMW_BLOCK


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("beta2", [0.5, 0.95, 0.999])
def test_roots_down_to_2_74_stay(beta2):
    """Every code from 1 up under scales that make code 1 worth 2^-74 and more; no
    gradient.  r^2 is 2^-148 at least, two of fp32's smallest steps, and half of it one:
    no product is 0."""
    say(f"adamw small roots beta2={beta2}")
    scales = [2.0 ** -65, 2.0 ** -60, 2.0 ** -30]  # code 1 is 2^-9 of the scale
    n = len(scales) * B
    codes = torch.arange(1, 126, dtype=torch.uint8).repeat(3)[:B].repeat(len(scales))
    for seed in range(5):
        t = dict(param=torch.zeros(n, device=DEV), grad=torch.zeros(n, device=DEV),
                 m=torch.zeros(n, dtype=torch.float8_e4m3fn, device=DEV),
                 v=codes.to(DEV).view(torch.float8_e4m3fn),
                 m_scale=torch.ones(len(scales), device=DEV),
                 v_scale=torch.tensor(scales, device=DEV))
        bw.mbok_adamw(bw.mbok_adamw_plan_init([t]), lr=1.0, step=2, beta2=beta2, seed=seed)
        r = t["v"].cpu().double() * t["v_scale"].cpu().double().repeat_interleave(B)
        assert (r > 0).all()
        assert (t["param"] == 0).all()
