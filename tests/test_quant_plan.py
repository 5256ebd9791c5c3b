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


# the contract: chunks of at most 512 blocks, at most 256 of them a context
MOST_BLOCKS = 256 * 512


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d,group", [(64, 1), (64, 16), (128, 1), (128, 16)])
def test_every_length_of_the_contract_is_planned(fmt, d, group):
    lengths = sorted({min(MOST_BLOCKS, max(1, int(2 ** (i / 4)) + j)) for i in range(69) for j in (-1, 0, 1)})
    assert lengths[-1] == MOST_BLOCKS
    for hkv, seqs in [(1, n) for n in range(1, 66)] + [(8, n) for n in (9, 16, 33, 64, 76, 128, 200, 1000, 8191)]:
        dd = desc(fmt, hkv=hkv, group=group, d=d)
        for blocks in lengths:
            chunk, splits = pkv.pkv_decode_plan(dd, seqs, 16 * blocks, -1, SMS)
            assert 1 <= chunk <= 512 and splits == -(-blocks // chunk) <= 256, (hkv, seqs, blocks)
    with pytest.raises(pkv.PkvError, match="%d blocks .* 256 chunks of 512" % (MOST_BLOCKS + 1)):
        pkv.pkv_decode_plan(desc(fmt, group=group, d=d), 4, 16 * MOST_BLOCKS + 1, -1, SMS)


@pytest.mark.parametrize("d,group", [(64, 4), (128, 4), (128, 16)])
def test_a_pair_more_changes_the_plan_by_little(d, group):
    """Over the long contexts, from one pair to the next the number of CTAs (or where they
    shrink together with the chunks, their blocks) changes by less than 2.5 times."""
    for blocks in (1025, 2048, 4096, 8192, 8193, 32768, 32769, MOST_BLOCKS):
        last = None
        for pairs in range(1, 400):
            chunk, _ = pkv.pkv_decode_plan(desc(hkv=1, group=group, d=d), pairs, 16 * blocks, -1, SMS)
            if last:
                assert chunk <= 2.5 * last and last <= 2.5 * chunk, (blocks, pairs, last, chunk)
            last = chunk


def test_long_contexts_of_few_pairs_are_cut_into_many_chunks():
    """From a sixteenth to a thirty-second of the GPU's CTAs full, at 2048 blocks and more: the
    chunks of one wave, not eight of a cluster."""
    one = desc(hkv=1, group=8)
    for pairs in (20, 32, 38):
        for blocks, most in ((2048, 96), (4096, 128), (8192, 128), (MOST_BLOCKS, 512)):
            chunk, _ = pkv.pkv_decode_plan(one, pairs, 16 * blocks, -1, SMS)
            assert chunk <= most, (pairs, blocks, chunk)
