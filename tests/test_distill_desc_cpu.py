"""Temperatures the distillation takes: log2(e) / tau has to be an fp32 number."""
import ctypes

import pytest

import boolean_weight_amd as bw

P = 1 << 20  # a "pointer" that is never read


@pytest.mark.parametrize("tau", [1e-45, 1e-40, 2.0 ** -127])
def test_subnormal_temperatures_are_refused(tau):
    with pytest.raises(bw.MbokError) as e:
        bw.mbok_distill_desc_init(10, 4, tau)
    assert e.value.status == -1
    d = bw.mbok_distill_desc(vocab=10, top=4, temperature=tau)  # filled by hand
    assert bw.load_library().mbok_distill(
        ctypes.byref(d), P, bw.MBOK_F32, 1, 10, P, bw.MBOK_F32, P, 4, None, None, P, None, None,
        bw.MBOK_F32, 0, None) == -1


@pytest.mark.parametrize("tau", [2.0 ** -126, 1.0, 2.0 ** 127])
def test_normal_temperatures_are_taken(tau):
    assert bw.mbok_distill_desc_init(10, 4, tau).temperature == tau
