"""Host-only checks of the maps that the training calls take (no GPU): a map that does not fit its tokens is refused
for that, before anything else is looked at."""
import pytest
import torch

import token_dispatch_expert_amd as moe

F8, F32, I32 = torch.float8_e4m3fn, torch.float32, torch.int32


@pytest.mark.parametrize("T,entries", [(0, 8), (0, 1), (4, 7), (4, 3), (4, 0)])
def test_unpack_refuses_a_map_without_k_entries_for_every_row(T, entries):
    """No tokens with a non-empty map too: its rows would be left unwritten without a word."""
    codes, scales = torch.zeros((T, 16), dtype=F8), torch.zeros((T, 1), dtype=F32)
    with pytest.raises(ValueError, match="k entries for every row"):
        moe.moe_checkpoint_unpack(codes, scales, torch.zeros((entries, 16), dtype=F32),
                                  flat_to_sorted=torch.zeros(entries, dtype=I32))
