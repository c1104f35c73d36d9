"""Dropouts and tensors in 4 bits say what the kernels read: what is described to
them once cannot be assigned afterwards."""
import pytest
import torch

from implicit_attribute_decode_amd import pipeline


@pytest.mark.parametrize("name,value", [("p", 0.9), ("seed", 8), ("offset", 7), ("step", None)])
def test_dropouts_are_not_changed_by_assignment(name, value):
    d = pipeline.Dropout(0.5, 2 ** 64 - 1, 2 ** 40)
    with pytest.raises(AttributeError):
        setattr(d, name, value)
    assert (d.p, d.seed, d.offset, d.step) == (0.5, 2 ** 64 - 1, 2 ** 40, None)
    assert (d.c.p, d.c.seed, d.c.offset, d.c.step) == (0.5, 2 ** 64 - 1, 2 ** 40, None)


@pytest.mark.parametrize("name,value", [("rows", 2), ("cols", 64), ("group", 64), ("codes", None), ("words", None)])
def test_4_bit_tensors_are_not_changed_by_assignment(name, value):
    q = pipeline.Q4Tensor.empty(3, 100, 32, device="cpu")
    with pytest.raises(AttributeError):
        setattr(q, name, value)
    assert (q.rows, q.cols, q.group) == (q.c.rows, q.c.cols, q.c.group) == (3, 100, 32)
    assert q.codes.shape == (3, 64) and q.words.shape == (3, 4)


@pytest.mark.parametrize("name,value", [("rows", 2), ("cols", 64), ("codes", None), ("scales", None)])
def test_mxfp4_tensors_are_not_changed_by_assignment(name, value, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    q = pipeline.Mx4Tensor.empty(3, 100, device="cpu")
    with pytest.raises(AttributeError):
        setattr(q, name, value)
    assert (q.rows, q.cols) == (q.c.rows, q.c.cols) == (3, 100)
