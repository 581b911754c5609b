"""Which streams the memory of an optimizer plan's table waits for, on a recorded GPU
(no kernel runs): a plan dropped after a step must not give its table away while the
step, on whatever stream, may still read addresses from it."""
import pytest
import torch

import boolean_weight_amd as bw
import fake_gpu
from fake_gpu import DeviceTensor, Gpu


class Stream(fake_gpu.Stream):
    """With an id: torch's own streams number themselves, others are their handle."""

    def __init__(self, handle, device=0, own=True):
        super().__init__(handle, device)
        self.stream_id = handle and (3 if own else handle)


class Table(DeviceTensor):
    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


@pytest.fixture
def gpu(monkeypatch):
    g = Gpu(monkeypatch)
    monkeypatch.setattr(torch.cuda, "Stream", fake_gpu.Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: Stream(handle, own=False))
    g.stack()[:] = [Stream(0)]
    return g


def plan():
    table = torch.zeros(64, dtype=torch.uint8).as_subclass(Table)
    table.recorded = []
    return bw.mbok_adamw_plan(bw._AdamwPlan(64, 1, 1, 0), table, [])


SIDE = Stream(0x77)


@pytest.mark.parametrize("stream,handle", [(None, 0), (0, 0), (Stream(0), 0), (SIDE, 0x77)])
def test_the_table_waits_for_the_step(gpu, stream, handle):
    p = plan()
    for t in (1, 2, 3):  # once per stream
        bw.mbok_adamw(p, lr=1e-3, step=t, stream=stream)
    assert p.table.recorded == [handle]
    assert {args[-1] or 0 for _, args in gpu.launched} == {handle}


def test_the_current_stream_counts(gpu):
    p = plan()
    for s in (SIDE, Stream(0x88), SIDE):
        with gpu.use(s):
            bw.mbok_adamw(p, lr=1e-3, step=1)
    bw.mbok_adamw(p, lr=1e-3, step=1)
    assert p.table.recorded == [0x77, 0x88, 0]
    assert [args[-1] or 0 for _, args in gpu.launched] == [0x77, 0x88, 0x77, 0]


@pytest.mark.parametrize("stream", [0x99, Stream(0x99, own=False)])
def test_another_owners_stream_is_not_waited_for(gpu, stream):
    """It may have ended when the memory is freed."""
    p = plan()
    bw.mbok_adamw(p, lr=1e-3, step=1, stream=stream)
    with gpu.use(Stream(0x99, own=False)):
        bw.mbok_adamw(p, lr=1e-3, step=2)
    assert p.table.recorded == []
    with gpu.use(Stream(0x99)):  # ended, and its handle torch's since
        bw.mbok_adamw(p, lr=1e-3, step=3)
    assert p.table.recorded == [0x99]
    assert [args[-1] for _, args in gpu.launched] == [0x99] * 3
