"""Windows, lengths and tables at the ends of 32 bits, on the host: the planners, the
ring's check and the workspace sizes.  Refusals return before any CUDA call."""
import ctypes

import pytest

import paged_kv_attention_21_gb300 as pkv
from paged_kv_attention_21_gb300 import build as libbuild

SMS, MOST = 152, 2 ** 31 - 1
P = ctypes.c_void_p(0x1000)  # non-null, aligned; no refused call touches it
DTYPES = [pkv.KV_BF16, pkv.KV_FP8_E4M3, pkv.KV_INT8, pkv.KV_FP4]


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkv.load_library()


def desc(kv_dtype, **kw):
    a = dict(num_q_heads=8, num_kv_heads=2, head_dim=64, num_blocks=10, max_blocks_per_seq=4096)
    a.update(kw)
    return pkv.make_desc(kv_dtype=kv_dtype, **a)


@pytest.mark.parametrize("kv_dtype", DTYPES)
@pytest.mark.parametrize("window", [65536, MOST - 30, MOST - 14, MOST - 13, MOST - 1, MOST])
def test_a_window_beyond_the_context_plans_as_none(lib, kv_dtype, window):
    for n, ctx in ((1, 1), (3, 100), (8, 65536), (200, 4096)):
        d = desc(kv_dtype)
        assert pkv.pkv_decode_plan(d, n, ctx, window, SMS) == pkv.pkv_decode_plan(d, n, ctx, -1, SMS)


@pytest.mark.parametrize("kv_dtype", DTYPES)
@pytest.mark.parametrize("ctx", [MOST - 15, MOST - 14, MOST])
def test_a_ring_plans_the_longest_context_by_its_window(lib, kv_dtype, ctx):
    d = desc(kv_dtype, ring_blocks=9)
    assert pkv.pkv_decode_plan(d, 4, ctx, 128, SMS) == pkv.pkv_decode_plan(d, 4, 100000, 128, SMS)


def decode(lib, d, ctx, window, sm_scale=0.0):
    """A call that is refused for its sm_scale, if not before."""
    byref = ctypes.byref(d)
    if d.kv_dtype in (pkv.KV_INT8, pkv.KV_FP4):
        s = P if d.kv_dtype == pkv.KV_FP4 else None
        st = lib.pkv_quant_decode(byref, P, P, P, s, s, P, P, 1, ctx, sm_scale, window, None, 0, P, None, P,
                                  1 << 20, None)
    else:
        st = lib.pkv_decode_attention(byref, P, P, P, P, P, P, P, 1, ctx, sm_scale, window, None, 0, P, None, P,
                                      1 << 20, None)
    assert st == 1
    return pkv.pkv_last_error()


@pytest.mark.parametrize("kv_dtype", DTYPES)
def test_a_ring_refuses_every_window_it_does_not_hold(lib, kv_dtype):
    d = desc(kv_dtype, ring_blocks=9)
    assert "sm_scale" in decode(lib, d, 1000, 9 * 16 - 15)  # the most it holds
    for window in (9 * 16 - 14, 10 ** 6, MOST - 15, MOST - 14, MOST):
        assert "ring_blocks" in decode(lib, d, 1000, window), window
    assert "sm_scale" in decode(lib, d, MOST, 9 * 16 - 15)


@pytest.mark.parametrize("kv_dtype", DTYPES)
@pytest.mark.parametrize("blocks", [1 << 27, (1 << 27) + 1, 1 << 28, MOST])
def test_tables_that_cover_more_than_32_bits_of_tokens(lib, kv_dtype, blocks):
    d = desc(kv_dtype, max_blocks_per_seq=blocks)
    for ctx in (1, 64, MOST):
        assert "sm_scale" in decode(lib, d, ctx, -1)


def test_ring_prefill_workspace_of_a_window_near_32_bits(lib):
    d = desc(pkv.KV_BF16, ring_blocks=9)
    for window in (10 ** 6, MOST - 32, MOST):
        cap = (window - 1 + 16 + 15) // 16 + 1
        block = 2 * 16 * 64 * 2  # bytes of K, and of V, in a staging block
        a256 = lambda x: (x + 255) // 256 * 256  # noqa: E731
        assert lib.pkv_prefill_ring_workspace_size(ctypes.byref(d), 3, window, 16) == \
            a256(3 * cap * 4) + 256 + 2 * a256(3 * cap * block)
