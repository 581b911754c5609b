"""The two-term forms refuse what the one-term forms refuse (no call here
reaches a kernel)."""
import pytest

import boolean_weight_amd as bw
import test_finetune_cpu as one


@pytest.fixture(scope="module")
def lib():
    return bw.load_library()


def marks(test):
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize")


@pytest.mark.parametrize("change,err", marks(one.test_gemmt_refuses))
def test_gemmt_precise_refuses(lib, change, err):
    base, _d = one.gemmt_args()
    assert one.call(lib.mbok_gemmt_precise, base, **change) == err


@pytest.mark.parametrize("change,err", marks(one.test_gated_refuses))
def test_gated_precise_refuses(lib, change, err):
    base, _d = one.gated_args()
    assert one.call(lib.mbok_gated_precise, base, **change) == err


@pytest.mark.parametrize("change,err", marks(one.test_gated_backward_refuses))
def test_gated_backward_precise_refuses(lib, change, err):
    base, _d = one.gated_backward_args()
    assert one.call(lib.mbok_gated_backward_precise, base, **change) == err
