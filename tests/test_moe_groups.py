"""Buffers of the pairs by expert, and operands of the experts' products that the binding
refuses before a launch: nothing here needs a GPU."""
import pytest
import torch

import adapter_lora_amd as ml


@pytest.mark.parametrize("name", ["pairs", "offsets"])
def test_buffers_stay_what_the_calls_know(name):
    """The calls keep the buffers' addresses, so a buffer cannot be replaced by another
    one that they would not see."""
    g = ml.MoeGroups(8, 4, device="cpu")
    kept = getattr(g, name)
    with pytest.raises(AttributeError):
        setattr(g, name, torch.empty(64, dtype=torch.int32))
    assert getattr(g, name) is kept
    assert (g.pairs_ptr, g.offsets_ptr) == (g.pairs.data_ptr(), g.offsets.data_ptr())
