"""Arguments of the operators around the routed experts that contradict each other (no GPU is touched)."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe


def test_a_place_for_saved_values_without_save():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    gu, dn = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="save=True"):
        moe.ffn_fwd(x, gu, dn, saved=torch.empty(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="device tensor"):   # with save the next check is reached
        moe.ffn_fwd(x, gu, dn, save=True, saved=torch.empty(1 << 16, dtype=torch.uint8))
