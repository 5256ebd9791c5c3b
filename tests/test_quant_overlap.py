"""The quantising append's refusal of a q_out over k_new or v_new, on the host: only calls that
are refused are made."""
import ctypes

import pytest

import paged_kv_attention_21_gb300 as pkv
from paged_kv_attention_21_gb300 import build as libbuild

P = ctypes.c_void_p(1 << 20)
HQ, HKV, D = 8, 2, 64  # rows of 512 and 128 elements


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkv.load_library()


@pytest.mark.parametrize("n,new,qs,q,k,v,name", [
    (1, 128, 512, 4096, 4096, 9000, "k_new"),         # the same start
    (1, 128, 512, 4096, 4600, 9000, "k_new"),         # the row's last elements
    (1, 128, 512, 4096, 9000, 4096 - 120, "v_new"),   # its first
    (4, 768, 768, 0, 504, 640, "k_new"),              # packed, k eight elements early
    (4, 768, 768, 128, 0, 768 + 8, "v_new"),          # v's rows reach into the next token's q
    (4, 768, 768, 768 * 3, 640, 768 * 3 - 120, "v_new"),
    (4, 768, 768, 768 * 3 + 8, 768 * 3 + 512, 0, "k_new"),
    (7, 128, 512, 512, 0, 1 << 20, "k_new")])        # other strides, extents that meet
@pytest.mark.parametrize("in_place", [False, True])
def test_q_out_over_new_rows_is_refused(lib, n, new, qs, q, k, v, name, in_place):
    d = pkv.make_desc(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, num_blocks=4, max_blocks_per_seq=4,
                      kv_dtype="int8")
    rope = pkv.Rope(1 << 20, D, 0, 16, 0)
    at = lambda e: ctypes.c_void_p((1 << 30) + 2 * e)  # noqa: E731
    st = lib.pkv_quant_append(ctypes.byref(d), ctypes.byref(rope), P, P, None, None, P, 1, P, P, n, at(k), at(v), new,
                              at(q) if in_place else ctypes.c_void_p(1 << 40), at(q), qs, qs, None)
    assert st == 1 and "q_out overlaps %s" % name in pkv.pkv_last_error()
