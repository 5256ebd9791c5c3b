"""Calls of the weights and of eviction that are refused without a GPU."""
import ctypes

import pytest
import torch

import paged_kv_attention_21_gb300 as pkv
from paged_kv_attention_21_gb300 import build as libbuild
from test_score_abi import P, P2, call_compact, call_mass, call_select, desc, refused, rule


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


def at(address, words=0):
    return ctypes.c_void_p(address + 4 * words)


FAR = 0x10000000


@pytest.mark.parametrize("name,size,out,width", [("mass", 700, "kept", 60), ("mass", 700, "kl", 2), ("lens", 2, "kept", 60),
                                                 ("lens", 2, "kl", 2), ("kept", 60, "kl", 2)])
def test_select_refuses_outputs_over_its_inputs(lib, name, size, out, width):
    """A row that does not fit shared memory is read again while others are written.  2 x 3 rows of
    at most 100 of 120 weights, of 10 kept."""
    kw = dict(mass=at(0x20000000), lens=at(0x30000000), kept=at(0x40000000), kl=at(0x50000000), stride=120)
    for word in (size - 1, 0, 1 - width):
        refused(call_select(lib, **dict(kw, **{name: at(FAR), out: at(FAR, word)})), 1, "overlaps")


def test_select_takes_neighbours(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    call_select(lib, mass=at(FAR), lens=at(FAR, 700), kept=at(FAR, 702), kl=at(FAR, 762), stride=120)
    assert "overlaps" not in pkv.pkv_last_error()  # on to the device, which is not there


def test_compact_refuses_weights_over_its_inputs(lib):
    kw = dict(ms=10, mos=9, top=8, ks=8, mass=at(FAR), mo=at(0x20000000))  # one sequence, two heads
    for moved in (1, -1, 19, -16):
        refused(call_compact(lib, **dict(kw, mo=at(FAR, moved))), 1, "mass_out overlaps mass")
    for name, word in (("kept", "kept"), ("kl", "kept_lens"), ("bt", "block_tables"), ("dt", "dst_tables")):
        refused(call_compact(lib, **dict(kw, **{name: at(0x20000000, 16)})), 1, "overlaps " + word)
    # in place: the same weights or others, not some of the same
    here = dict(dt=P, kd=P, vd=P2, ms=9, mos=9, mo=at(FAR, 9))
    refused(call_compact(lib, **dict(kw, **here)), 1, "mass_out overlaps mass")


def test_weights_refuse_to_be_written_over_what_they_read(lib):
    kw = dict(mass=at(FAR), stride=20, top=16)  # one sequence, two heads
    for name, word in (("lse", "lse"), ("lens", "kv_lens"), ("qo", "qo_indptr"), ("bt", "block_tables")):
        refused(call_mass(lib, **dict(kw, **{name: at(FAR, 35)})), 1, "mass overlaps " + word)
    refused(call_mass(lib, rule(slopes=FAR + 4), **kw), 1, "mass overlaps slopes")
    refused(call_mass(lib, rule(prefix_lens=FAR + 140), **kw), 1, "mass overlaps prefix_lens")


def test_a_window_past_32_bits_is_refused():
    for window in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="window"):
            pkv.make_score(0.1, window=window)
    assert pkv.make_score(0.1, window=2 ** 31 - 1).window == 2 ** 31 - 1
    assert pkv.make_score(0.1, window=-1).window == -1
