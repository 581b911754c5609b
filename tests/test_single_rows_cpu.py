"""Leading dimensions the binding passes for one row: the row's own stride is
arbitrary, so one buffer seen through views of different widths is one buffer."""
import pytest
import torch

import boolean_weight_amd as bw
from fake_gpu import Gpu, on_device


@pytest.fixture
def gpu(monkeypatch):
    return Gpu(monkeypatch)


def test_in_place_gradient_of_a_wider_single_row(gpu):
    Z = on_device(1, 1030, dtype=torch.float32)
    d = bw.mbok_distill_desc(vocab=1001, top=3, temperature=1.0)
    l, idx = on_device(1, 3, dtype=torch.float32), on_device(1, 3, dtype=torch.int32)
    bw.mbok_distill(d, Z, l, idx, on_device(1, dtype=torch.float32), dZ=Z[:, :1001])
    (_, args), = gpu.launched
    z, ldz, dz, lddz = args[1], args[4], args[13], args[15]
    assert z == dz and ldz == lddz >= 1001


def test_in_place_pre_gradient_of_a_wider_single_row(gpu):
    d = bw.mbok_desc(m=100, n=256, K=1, group=128, alpha_dtype=1, layout=1)
    packed = on_device(bw._packed_bytes(208, 256, 1, 1), dtype=torch.uint8)
    pre = on_device(1, 216)
    bw.mbok_gated_backward(d, packed, pre, on_device(1, 100), pre[:, :208])
    (_, args), = gpu.launched
    assert args[2] == args[8] and args[3] == args[9] >= 208
