"""The binding's checks of what an argument holds beside its address."""
import pytest
import torch

import paged_kv_attention_21_gb300 as pkv


def test_the_binding_checks_the_rotations_table_on_every_call():
    """make_rope's check holds for the device that was current then."""
    r = pkv.Rope(0x1000, 64, 0, 16, 0)
    r.table = torch.zeros(16, 32, 2)
    with pytest.raises(ValueError, match="rope table: on cpu, expected the current CUDA device"):
        pkv.pkv_rope_rotate(r, torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 64))
    r = pkv.Rope(0x1000, 64, 0, 16, 0)  # filled by hand: its address is the caller's affair
    with pytest.raises(ValueError, match="q: on cpu"):
        pkv.pkv_rope_rotate(r, torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 64))
