"""Dropouts and 4-bit tensors say what the kernels read: what is described to
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
