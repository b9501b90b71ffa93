"""The tensors behind a cache's or pool's handle: the handle holds their
addresses, so that exchanging one for another has to fail."""
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn


@pytest.mark.parametrize("kind,names", [(qbn.KVPool, ("table", "lens", "refs")), (qbn.KVCache, ("k", "v", "k_scales", "v_scales"))])
def test_tensors_of_a_handle_cannot_be_exchanged(kind, names):
    h = kind.__new__(kind)  # no device here: the attributes alone
    for name in names:
        mine = torch.zeros(3)
        h.__dict__["_" + name] = mine
        assert getattr(h, name) is mine
        setattr(h, name, mine)  # what `h.lens += 1` does
        with pytest.raises(AttributeError):
            setattr(h, name, torch.zeros(3))
        with pytest.raises(AttributeError):
            delattr(h, name)
        assert getattr(h, name) is mine
