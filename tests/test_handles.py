"""Handles keep the memory and the sizes that the library was given: a Rotary's attributes cannot be replaced
(no GPU needed)."""
import copy

import pytest
import torch

from scale_search_weights_amd import rotary
from test_abi import G


def _rotary():
    return rotary.Rotary(G(32, dtype=torch.float64), G(32, dtype=torch.int32), axes=3)


@pytest.mark.parametrize("make", [_rotary], ids=["Rotary"])
def test_attributes_stay(make):
    h = make()
    for name, value in list(vars(h).items()):
        with pytest.raises(AttributeError):
            setattr(h, name, value.clone() if isinstance(value, torch.Tensor) else object())
        with pytest.raises(AttributeError):
            delattr(h, name)
        assert getattr(h, name) is value
    h.note = "the caller's own"
    assert copy.copy(h)._c is h._c


def test_a_rotarys_tensors_may_be_changed():
    h = _rotary()
    h.inv_freq += 1
    h.axis.fill_(2)
    assert h._c.inv_freq == h.inv_freq.data_ptr() and h._c.axis == h.axis.data_ptr()
