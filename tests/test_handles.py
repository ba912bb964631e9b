"""Handles keep the memory and the sizes that the library was given: attributes of a Rotary and of a KVCache
cannot be replaced (no GPU needed)."""
import copy

import pytest
import torch

from scale_search_weights_amd import kvcache, rotary
from test_abi import G


def _rotary():
    return rotary.Rotary(G(32, dtype=torch.float64), G(32, dtype=torch.int32), axes=3)


def _cache():
    u8 = torch.uint8
    return kvcache.KVCache(G(4, 2, 16, 32, dtype=u8), G(4, 2, 16, 4, dtype=u8), G(4, 2, 16, 32, dtype=u8),
                           G(4, 2, 16, 4, dtype=u8), G(2), G(2))


@pytest.mark.parametrize("make", [_rotary, _cache], ids=["Rotary", "KVCache"])
def test_attributes_stay(make):
    h = make()
    for name, value in [(n, v) for n, v in vars(h).items() if n[0] != "_"]:
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
