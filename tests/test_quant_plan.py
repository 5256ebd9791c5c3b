"""The quantised decode's plan, on the host: pkv_decode_plan of a quantised desc."""
import math

import pytest

import paged_kv_attention_21_gb300 as pkv
from paged_kv_attention_21_gb300 import build as libbuild

SMS = 152


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return pkv.load_library()


def desc(fmt="fp4", hkv=8, group=4, d=128, blocks=1 << 20, ring=0):
    return pkv.make_desc(num_q_heads=hkv * group, num_kv_heads=hkv, head_dim=d, num_blocks=10,
                         max_blocks_per_seq=blocks, kv_dtype=fmt, ring_blocks=ring)


def test_plan_of_a_quantised_pool():
    """The measured plans: the rules' own examples, by (pairs, blocks)."""
    for fmt in ("int8", "fp4"):
        one = desc(fmt, hkv=1, group=8)
        assert pkv.pkv_decode_plan(one, 960, 2048 * 16, -1, SMS) == (256, 8)
        assert pkv.pkv_decode_plan(one, 512, 128 * 16, -1, SMS) == (128, 1)  # the pairs fill the GPU
        assert pkv.pkv_decode_plan(one, 2, 256 * 16, -1, SMS) == (8, 32)
        assert pkv.pkv_decode_plan(one, 8, 2048 * 16, -1, SMS) == (32, 64)
        assert pkv.pkv_decode_plan(one, 32, 256 * 16, -1, SMS) == (32, 8)    # one cluster of 8
        assert pkv.pkv_decode_plan(one, 128, 128 * 16, 128, SMS) == (9, 1)   # what a window can touch
        with pytest.raises(pkv.PkvError):
            pkv.pkv_decode_plan(one, 1, 0, -1, SMS)


def test_plan_covers_the_context():
    for hkv, n, ctx in ((8, 1, 1), (2, 64, 4096), (8, 120, 32768), (3, 17, 1000)):
        chunk, splits = pkv.pkv_decode_plan(desc(hkv=hkv), n, ctx, -1, SMS)
        assert 1 <= chunk <= 512 and splits == math.ceil(math.ceil(ctx / 16) / chunk) <= 256
