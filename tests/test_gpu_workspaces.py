"""The workspaces the binding keeps, on the GPU: their memory belongs to the
launch stream, and what is computed through them is what a caller's own
workspace gives."""
import threading

import pytest
import torch

import boolean_weight_amd as bw
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def layer(m, n, seed, K=2):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    d = bw.mbok_desc_init(m, n, K)
    signs = torch.randint(0, 2, (K, m, n), generator=gen, device=DEV, dtype=torch.int8) * 2 - 1
    alpha = torch.rand((K, m, n // 128), generator=gen, device=DEV).to(torch.float16)
    packed = torch.empty(bw.mbok_packed_bytes(d), dtype=torch.uint8, device=DEV)
    bw.mbok_pack(d, signs, alpha, packed)
    return d, packed


def gemmt_case(m, n, T, seed):
    """(call with a workspace argument, output, result with a workspace of its own)."""
    d, packed = layer(m, n, seed)
    dY = torch.randn(T, m, generator=torch.Generator(device=DEV).manual_seed(seed + 1),
                     device=DEV).to(BF)
    dX = torch.empty(T, n, dtype=BF, device=DEV)
    own = torch.empty(bw.mbok_gemmt_workspace_bytes(d, T), dtype=torch.uint8, device=DEV)

    def call(**kw):
        bw.mbok_gemmt(d, packed, dY, dX, **kw)
    call(workspace=own)
    torch.cuda.synchronize()
    return call, dX, dX.clone()


def test_kept_workspace_belongs_to_the_launch_stream(monkeypatch):
    say("kept workspaces and their streams")
    small, large = gemmt_case(256, 512, 16, 1), gemmt_case(2048, 4096, 200, 2)
    side = torch.cuda.Stream()
    empty, seen = torch.empty, []

    def spy(*args, **kw):
        if kw.get("dtype") == torch.uint8:
            seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)

    for stream, handle in ((None, 0), (0, 0), (torch.cuda.default_stream(), 0),
                           (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream)):
        monkeypatch.setattr(bw, "_WORKSPACES", {})
        del seen[:]
        with monkeypatch.context() as patch:
            patch.setattr(torch, "empty", spy)
            for call, out, want in (small, large, small):
                out.fill_(-1)
                torch.cuda.synchronize()
                call(stream=stream)
                torch.cuda.synchronize()
                assert torch.equal(out, want)
        assert seen == [handle] * 2, (stream, seen)


def test_threads_on_one_stream():
    """Two threads launch on the default stream at once, through its kept
    workspace: each gets its own result every time."""
    say("kept workspace and threads")
    cases = [gemmt_case(512, 512, 16, 5), gemmt_case(2048, 4096, 40, 6)]
    wrong = []

    def run(call, out, want):
        for i in range(60):
            call()
            if not torch.equal(out, want):
                wrong.append((tuple(out.shape), i))

    threads = [threading.Thread(target=run, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong[:5]
