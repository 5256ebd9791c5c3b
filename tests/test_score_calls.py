"""Calls of the weights and of eviction that are refused without a GPU."""
import pytest
import torch

import paged_kv_attention_21_gb300 as pkv
from paged_kv_attention_21_gb300 import build as libbuild
from test_score_abi import desc, rule


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkv.load_library()


def test_weights_of_ragged_queries_need_their_bound(lib):
    """Without max_q_len only each sequence's first query would count."""
    q, lens = torch.zeros(3, 8, 128).bfloat16(), torch.zeros(1, dtype=torch.int32)
    args = (None, None, lens, 16, None, None)
    with pytest.raises(ValueError, match="max_q_len: needed"):
        pkv.pkv_score_mass(desc(), rule(), q, torch.zeros(2, dtype=torch.int32), *args)
    with pytest.raises(ValueError, match="on cpu"):  # goes on to the tensors
        pkv.pkv_score_mass(desc(), rule(), q, torch.zeros(2, dtype=torch.int32), *args, max_q_len=3)
    with pytest.raises(ValueError, match="on cpu"):
        pkv.pkv_score_mass(desc(), rule(), q[:1], None, *args)
