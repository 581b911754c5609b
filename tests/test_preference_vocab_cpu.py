"""The preference loss's vocabulary in the binding: a descriptor without one says so
where labels are given, since padding ids count as tokens then (no kernel runs)."""
import warnings

import pytest
import torch

import boolean_weight_amd as bw
from fake_gpu import Gpu, on_device


@pytest.fixture
def gpu(monkeypatch):
    return Gpu(monkeypatch)


def call(d, label):
    f32, i32 = dict(dtype=torch.float32), dict(dtype=torch.int32)
    bw.mbok_preference(d, on_device(3, **i32), on_device(5, **f32), on_device(1, **f32),
                       label=on_device(5, **i32) if label else None)


def test_labels_without_a_vocabulary_warn_once(gpu):
    d = bw.mbok_preference_desc_init(0.1, mean=True)
    assert d.vocab == bw.MBOK_MAX_VOCAB
    with pytest.warns(UserWarning, match="vocab"):
        call(d, True)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call(d, True)
    assert [name for name, _ in gpu.launched] == ["mbok_preference"] * 2


@pytest.mark.parametrize("vocab,label", [(100, True), (100, False), (None, False),
                                         (bw.MBOK_MAX_VOCAB, True)])
def test_no_warning_otherwise(gpu, vocab, label):
    d = bw.mbok_preference_desc_init(0.1, vocab=vocab)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call(d, label)
    assert len(gpu.launched) == 1


def test_a_descriptor_filled_by_hand_is_taken_as_it_is(gpu):
    d = bw.mbok_preference_desc(beta=0.1, smoothing=0.0, margin=0.0, mean=0, vocab=100)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call(d, True)
