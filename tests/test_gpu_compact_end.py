"""A move of 2^31 - 1 rows, on the GPU."""
import pytest
import torch

import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("n", [MOST, MOST - 63])
def test_the_last_rows(n):
    """Rows behind the last one are of no sequence.  (All blocks but the last eight go over one
    another into one block, of which nothing is looked at.)"""
    blocks, tail = 2 ** 27, 8
    gen = torch.Generator(device=DEV).manual_seed(n)
    src = [torch.randint(0, 256, (tail, 1, 16, 64), generator=gen, dtype=torch.uint8, device=DEV) for _ in range(2)]
    dst = [torch.zeros(tail + 1, 1, 16, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    tables = (torch.arange(blocks, device=DEV, dtype=torch.int32) % tail)[None].contiguous()
    dst_tables = torch.full((1, blocks), tail, dtype=torch.int32, device=DEV)
    dst_tables[0, blocks - tail:] = torch.arange(tail, device=DEV)
    kept = torch.arange(MOST, dtype=torch.int32, device=DEV)[None, None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    desc, dst_desc = (pkv.make_desc(num_q_heads=1, num_kv_heads=1, head_dim=64, num_blocks=b, max_blocks_per_seq=blocks,
                                    kv_dtype="fp8_e4m3") for b in (tail, tail + 1))
    pkv.pkv_evict_compact(desc, src[0], src[1], tables, kept, lens, dst_desc=dst_desc, k_dst=dst[0], v_dst=dst[1],
                          dst_tables=dst_tables)
    assert pkv.pkv_device_errors() == 0
    rows = n - (blocks - tail) * 16  # of the last eight blocks
    for a, b in zip(src, dst):
        a, b = a.reshape(-1, 64), b.reshape(-1, 64)[:tail * 16]
        assert torch.equal(b[:rows], a[:rows]) and not b[rows:].any()
