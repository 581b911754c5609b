"""GPU test of an optimizer plan dropped while its step waits on another stream."""
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


def test_ids_tell_whose_a_stream_is():
    own = torch.cuda.Stream()
    assert own.stream_id != own.cuda_stream
    outside = torch.cuda.ExternalStream(own.cuda_stream)
    assert outside.stream_id == outside.cuda_stream
    assert torch.cuda.default_stream().cuda_stream == 0


def test_dropped_plan_keeps_its_table():
    """A step behind a long queue on a side stream; the plan goes.  Its table's memory is
    given to nobody while the queue runs (new tensors of its size lie elsewhere; they
    are not written)."""
    say("adamw plan dropped")
    n = 5000
    t = dict(param=torch.ones(n, device=DEV), grad=torch.ones(n, device=DEV),
             m=torch.zeros(n, device=DEV), v=torch.zeros(n, device=DEV))
    side = torch.cuda.Stream()
    plan = bw.mbok_adamw_plan_init([t])
    at, size = plan.table.data_ptr(), plan.table.numel()
    a = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(400):
            b = a @ a
    bw.mbok_adamw(plan, lr=0.5, step=1, stream=side)
    waiting = not side.query()
    del plan
    new = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(8)]
    still = not side.query()
    torch.cuda.synchronize()
    # m / sqrt(v) of a first step is 1 but for the roundings
    assert ((t["param"] - 0.5).abs() <= 2.0 ** -18).all()
    del b
    if not (waiting and still):
        pytest.skip("the queue ended before the plan was dropped")
    assert all(x.data_ptr() != at for x in new)
