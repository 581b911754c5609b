"""The workspaces the binding keeps: which stream their memory belongs to, on a
recorded GPU (no kernel runs)."""
import threading
import time

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


def scale_grad(m, stream=None, T=256, n=256):
    d = bw.mbok_desc(m=m, n=n, K=1, group=128, alpha_dtype=1, layout=1)
    packed = on_device(bw._packed_bytes(m, n, 1, 1), dtype=torch.uint8)
    bw.mbok_scale_grad(d, packed, on_device(T, m), on_device(T, n),
                       on_device(m * (n // 128), dtype=torch.float32), stream=stream)


def gated_backward(m, stream=None, T=16, n=1024):
    d = bw.mbok_desc(m=m, n=n, K=1, group=128, alpha_dtype=1, layout=1)
    packed = on_device(bw._packed_bytes(2 * m, n, 1, 1), dtype=torch.uint8)
    bw.mbok_gated_backward(d, packed, on_device(T, 2 * m), on_device(T, m), on_device(T, 2 * m),
                           on_device(T, n), stream=stream)


def gemv(m, stream=None, n=4096):
    d = bw.mbok_desc(m=m, n=n, K=1, group=128, alpha_dtype=1, layout=1)
    packed = on_device(bw._packed_bytes(m, n, 1, 1), dtype=torch.uint8)
    bw.mbok_gemv(d, packed, on_device(n), on_device(m, dtype=torch.float32), stream=stream)


class Launches:
    """Launch times of calls from several threads: each takes a while between its
    first and its last kernel, as a call of two kernels does."""

    def __init__(self):
        self.active, self.met, self.lock = [], [], threading.Lock()

    def __call__(self, name, args):
        ws = args[-2]
        assert ws, name
        with self.lock:
            self.met += [(ws, other) for other in self.active]
            self.active.append(ws)
        time.sleep(0.02)
        with self.lock:
            self.active.remove(ws)


def together(*calls):
    errors = []

    def run(call):
        try:
            call()
        except BaseException as e:  # noqa: B902
            errors.append(e)
    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors, errors


@pytest.mark.parametrize("first,m", [(gemmt, 256), (scale_grad, 256), (gated_backward, 256),
                                     (gemvt, 8192), (gemv, 256)])
def test_threads_on_one_stream_take_turns_with_the_kept_workspace(monkeypatch, first, m):
    """Two threads' calls on one stream: no launch of one falls between the two
    kernels of another."""
    monkeypatch.setenv("MBOK_GEMV_VARIANT", "split")
    launches = Launches()
    gpu = Gpu(monkeypatch, launches)
    first(m), gemmt(512)  # the kept workspace is there
    together(*[lambda f=f, k=k, s=s: f(k, s) for f, k in ((first, m), (gemmt, 512))
               for s in (None, 0, Stream(0))])
    assert len(gpu.launched) == 8
    assert launches.met == []


def test_threads_on_two_streams_do_not_wait_for_each_other(monkeypatch):
    both = threading.Barrier(2, timeout=30)
    Gpu(monkeypatch, lambda name, args: both.wait())
    together(lambda: gemmt(256, SIDE), lambda: gemmt(256, 0))


def test_a_failed_call_gives_the_workspace_back(monkeypatch):
    def refuse(name, args):
        raise RuntimeError("no")
    Gpu(monkeypatch, refuse)
    with pytest.raises(RuntimeError):
        gemmt(256)
    with pytest.raises(RuntimeError):
        gemvt(8192)
    calls = []
    Gpu(monkeypatch, lambda name, args: calls.append(name))
    together(lambda: gemmt(256), lambda: gemvt(8192))
    assert sorted(calls) == ["mbok_gemmt", "mbok_gemvt"]


@pytest.mark.parametrize("call,m", [(gemmt, 256), (scale_grad, 256), (gated_backward, 256),
                                    (gemvt, 8192), (gemv, 256)])
@pytest.mark.parametrize("stream", [None, 0, SIDE])
def test_captured_calls_have_memory_of_their_own(gpu, monkeypatch, call, m, stream):
    """A graph's workspace is neither the kept one, which a larger request of
    any other call frees, nor another captured call's, nor kept afterwards."""
    monkeypatch.setenv("MBOK_GEMV_VARIANT", "split")
    handle = 0 if not isinstance(stream, Stream) else stream.cuda_stream
    call(m, stream)
    gpu.capturing = {handle}
    call(m, stream), call(m, stream)
    gpu.capturing = set()
    gemmt(2048, stream), call(m, stream)
    used = [args[-2] for _, args in gpu.launched]
    assert used[1] not in (used[0], used[2], used[3], used[4])
    assert used[2] not in (used[0], used[3], used[4])
    assert {w.data_ptr() for w in bw._WORKSPACES.values()} == {used[4]}
    # each belongs to the launch stream
    assert {h for h, _ in gpu.allocated} == {handle}


def test_workspace_for_under_capture(gpu):
    kept = bw.workspace_for(100, "cuda:0")
    gpu.capturing = {0}
    a, b = (bw.workspace_for(100, "cuda:0") for _ in range(2))
    gpu.capturing = set()
    assert len({x.data_ptr() for x in (kept, a, b)}) == 3
    assert bw.workspace_for(100, "cuda:0") is kept
