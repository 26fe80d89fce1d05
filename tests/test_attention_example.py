"""What the attention example turns down before anything runs (no GPU needed)."""
import os
import sys
import types

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_prompts_longer_than_the_cache():
    """Such a prompt's places would be looked up past the page table, which ends in a device assert."""
    from attention_layer import AttentionLayer
    layer = types.SimpleNamespace(qmm=None, max_len=128)
    with pytest.raises(ValueError):
        AttentionLayer.prefill(layer, torch.zeros(129, 2048))
