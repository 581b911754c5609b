"""The workspaces the binding keeps: which stream their memory belongs to, on a
recorded GPU (no kernel runs)."""
import pytest
import torch

import boolean_weight_amd as bw
from fake_gpu import Gpu, Stream, on_device


@pytest.fixture
def gpu(monkeypatch):
    return Gpu(monkeypatch)


def gemmt(m, stream=None, T=16, n=4096):
    d = bw.mbok_desc(m=m, n=n, K=1, group=128, alpha_dtype=1, layout=1)
    packed = on_device(bw._packed_bytes(m, n, 1, 1), dtype=torch.uint8)
    bw.mbok_gemmt(d, packed, on_device(T, m), on_device(T, n), stream=stream)


def gemvt(m, stream=None, n=1024):
    d = bw.mbok_desc(m=m, n=n, K=1, group=128, alpha_dtype=1, layout=1)
    packed = on_device(bw._packed_bytes(m, n, 1, 1), dtype=torch.uint8)
    bw.mbok_gemvt(d, packed, on_device(m), on_device(n, dtype=torch.float32), stream=stream)


SIDE = Stream(0x77)


@pytest.mark.parametrize("stream,handle", [(None, 0), (0, 0), (Stream(0), 0), (SIDE, 0x77),
                                           (0x77, 0x77)])
@pytest.mark.parametrize("call,small,large", [(gemmt, 256, 2048)])
def test_kept_memory_belongs_to_the_launch_stream(gpu, call, small, large, stream, handle):
    """Also where a larger request replaces it, and with another stream current:
    memory tied to another stream could be given away while the launches of
    this one still use it."""
    call(small, stream)
    with gpu.use(Stream(0x55)):
        if stream is not None:
            call(large, stream)
    call(large, stream)
    assert {args[-1] or 0 for _, args in gpu.launched} == {handle}
    assert gpu.allocated and {h for h, _ in gpu.allocated} == {handle}


def test_kept_memory_follows_the_current_stream(gpu):
    with gpu.use(SIDE):
        gemmt(256)
    gemmt(256)
    assert [h for h, _ in gpu.allocated] == [0x77, 0]
    assert [args[-1] or 0 for _, args in gpu.launched] == [0x77, 0]


@pytest.mark.parametrize("stream,handle", [(None, 0), (0, 0), (Stream(0), 0), (SIDE, 0x77),
                                           (0x77, 0x77)])
def test_workspace_for(gpu, stream, handle):
    a = bw.workspace_for(100, "cuda:0", stream)
    b = bw.workspace_for(2 << 20, "cuda:0", stream)
    assert a.numel() >= 100 and b.numel() >= 2 << 20
    assert bw.workspace_for(300, "cuda:0", stream) is b
    assert [h for h, _ in gpu.allocated] == [handle] * 2
