"""The rotary and quantised-pool entry points without a GPU: formats, refusals,
scaled tables.  Refusals return before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import _quant as Q
import paged_kv_attention_21_gb300 as pkv
from paged_kv_attention_21_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkv.load_library()


def desc(**kw):
    a = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, num_blocks=10, max_blocks_per_seq=4,
             kv_dtype="int8")
    a.update(kw)
    return pkv.make_desc(**a)


P = ctypes.c_void_p(0x1000)  # a non-null, aligned address that no refused call touches
ODD = ctypes.c_void_p(0x1008)


def status(lib, st, word):
    assert st != 0
    assert word in pkv.pkv_last_error(), pkv.pkv_last_error()
    return st


@pytest.mark.parametrize("fmt,d,record", [("int8", 64, 1088), ("int8", 128, 2112), ("fp4", 64, 576),
                                          ("fp4", 128, 1152)])
def test_pool_bytes(lib, fmt, d, record):
    dd = desc(kv_dtype=fmt, head_dim=d, num_blocks=1 << 24, num_kv_heads=8, num_q_heads=64)
    assert Q.record_bytes(fmt, d) == record == pkv.pkv_quant_record_bytes(dd)
    assert pkv.pkv_quant_cache_bytes(dd) == record * 8 << 24  # past 32 bits
    assert pkv.pkv_cache_bytes(dd) == 0
    assert pkv.pkv_quant_cache_bytes(desc(kv_dtype="bf16")) == 0


@pytest.mark.parametrize("fmt,d", [("int8", 64), ("int8", 128), ("fp4", 64), ("fp4", 128)])
def test_code_offsets_are_a_permutation(fmt, d):
    rb = Q.row_bytes(fmt, d)
    at = sorted(Q.code_offset(fmt, d, r, j) for r in range(16) for j in range(rb))
    assert at == list(range(16 * rb))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_reference_quantiser_is_within_half_a_step(fmt):
    rng = np.random.default_rng(3)
    for value in (1e-3, 1.0, 50.0):
        x = (value * rng.standard_normal(128)).astype(np.float32)
        g = value * 4 / 2688
        y = Q.row_values(fmt, *Q.quantise(fmt, x, g), g)
        if fmt == "int8":
            assert np.abs(y - x).max() <= np.abs(x).max() / 127 * 0.5001
        else:  # a step of e2m1 is at most 2 of 6, the e4m3 scale off by 2^-4
            assert np.abs(y - x).max() <= np.abs(x).max() / 6 * (1 + 2.0 ** -4) * 1.0001


def test_the_other_entry_points_refuse_quantised_pools(lib):
    for fmt in ("int8", "fp4"):
        d = ctypes.byref(desc(kv_dtype=fmt))
        assert lib.pkv_append_rope(d, P, P, P, P, P, 1, P, P, 1, P, P, None, None, 0, None) == 2
        assert lib.pkv_gather_kv(d, P, P, P, P, 1, 16, P, None) == 2
        assert lib.pkv_decode_attention(d, P, P, P, P, P, P, P, 1, 16, 1.0, -1, None, 0, P, None, P,
                                        1 << 20, None) == 2
        assert "pkv_quant_" in pkv.pkv_last_error()


def rows(**kw):
    a = dict(in_=0x1000, out=0x100000, in_token_stride=256, in_head_stride=64, out_token_stride=256,
             out_head_stride=64, num_heads=4, reserved=0)
    a.update(kw)
    return pkv.Rows(**a)


def rope(**kw):
    a = dict(cos_sin=0x1000, rotary_dim=64, layout=0, max_pos=16, flags=0)
    a.update(kw)
    return pkv.Rope(**a)


def test_rope_refusals(lib):
    def call(r=None, q=None, k=None, dtype=0, tokens=3, dim=64, pos=P):
        return lib.pkv_rope_rotate(ctypes.byref(r or rope()), dtype, pos, tokens, dim,
                                   ctypes.byref(q or rows()), None if k is None else ctypes.byref(k), None)
    assert status(lib, call(dtype=3), "dtype") == 2
    assert status(lib, call(dim=63), "head_dim") == 2
    assert status(lib, call(dim=514), "head_dim") == 2
    assert status(lib, call(r=rope(rotary_dim=66)), "rotary_dim") == 1
    assert status(lib, call(r=rope(rotary_dim=7)), "rotary_dim") == 1
    assert status(lib, call(r=rope(rotary_dim=0)), "rotary_dim") == 1
    assert status(lib, call(r=rope(layout=2)), "layout") == 1
    assert status(lib, call(r=rope(max_pos=0)), "max_pos") == 1
    assert status(lib, call(r=rope(flags=2)), "flags") == 1
    assert status(lib, call(r=rope(cos_sin=None)), "cos_sin") == 1
    assert status(lib, call(r=rope(cos_sin=0x1004)), "aligned") == 1
    assert status(lib, call(tokens=-1), "num_tokens") == 1
    assert status(lib, call(pos=None), "null") == 1
    assert status(lib, call(q=rows(in_=None)), "null") == 1
    assert status(lib, call(q=rows(in_=0x1001)), "aligned") == 1
    assert status(lib, call(q=rows(in_token_stride=-1)), "stride") == 1
    assert status(lib, call(q=rows(out_token_stride=0)), "overlap") == 1
    assert status(lib, call(q=rows(out_head_stride=63)), "overlap") == 1
    assert status(lib, call(q=rows(out_token_stride=255)), "overlap") == 1
    assert status(lib, call(q=rows(out=0x1000, out_token_stride=512)), "overlaps in") == 1
    assert status(lib, call(q=rows(out=0x1040)), "overlaps in") == 1
    # strides whose extents would not fit 64 bits
    assert status(lib, call(q=rows(in_token_stride=1 << 46), tokens=2 ** 31 - 1), "stride") == 1
    assert status(lib, call(q=rows(out_token_stride=2 ** 63 - 1)), "stride") == 1
    assert status(lib, call(q=rows(in_head_stride=1 << 62)), "stride") == 1
    assert status(lib, call(k=rows(num_heads=-1)), "num_heads") == 1
    assert call(tokens=0) == 0
    assert call(q=rows(num_heads=0)) == 0


def test_append_refusals(lib):
    ok = dict(d=desc(), r=rope(rotary_dim=128), kp=P, vp=P, ks=None, vs=None, bt=P, seqs=1, tts=P,
              pos=P, n=1, k=P, v=P, stride=256, q=P, qo=P, qs=1024, qos=1024)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.pkv_quant_append(ctypes.byref(a["d"]), None if a["r"] is None else ctypes.byref(a["r"]),
                                    a["kp"], a["vp"], a["ks"], a["vs"], a["bt"], a["seqs"], a["tts"],
                                    a["pos"], a["n"], a["k"], a["v"], a["stride"], a["q"], a["qo"],
                                    a["qs"], a["qos"], None)
    assert status(lib, call(d=desc(kv_dtype="bf16")), "quantised") == 2
    assert status(lib, call(d=desc(head_dim=96)), "head_dim") == 2
    assert status(lib, call(d=desc(num_q_heads=34)), "group size") == 2
    assert status(lib, call(ks=P, vs=P), "must be NULL") == 1
    assert status(lib, call(d=desc(kv_dtype="fp4")), "k_scale") == 1
    assert status(lib, call(n=-1), "negative") == 1
    for name in ("kp", "vp", "bt", "tts", "pos", "k", "v", "qo"):
        assert status(lib, call(**{name: None}), "null") == 1
    for name in ("kp", "vp", "k", "v", "q", "qo"):
        assert status(lib, call(**{name: ODD}), "aligned") == 1
    assert status(lib, call(r=None), "rotation") == 1
    assert status(lib, call(stride=248), "stride") == 1
    assert status(lib, call(stride=260), "stride") == 1
    assert status(lib, call(qs=1000), "stride") == 1
    assert status(lib, call(qs=2048), "in place") == 1
    # q_out partly on q: a shifted row, a row of the next token, other strides
    assert status(lib, call(qo=P.value + 16), "q_out overlaps q") == 1
    assert status(lib, call(qo=P.value + 2 * 1024 - 16), "q_out overlaps q") == 1
    assert status(lib, call(qo=P.value + 2 * 1032, qs=2048, qos=2048, n=3, q=P.value + 4096), "q_out overlaps q") == 1
    assert status(lib, call(qo=P.value + 2 * 4096, qs=2048, qos=4096, n=5), "q_out overlaps q") == 1
    assert call(n=0) == 0


def test_read_load_and_decode_refusals(lib):
    d = desc()

    def read(d=d, kp=P, vp=P, ks=None, n=1, dt=0, k=P, v=P, bt=P):
        return lib.pkv_quant_read(ctypes.byref(d), kp, vp, ks, ks, bt, 1, P, P, n, dt, k, v, None)
    assert status(lib, read(d=desc(kv_dtype=1)), "quantised") == 2
    assert status(lib, read(dt=1), "out_dtype") == 2
    assert status(lib, read(n=-1), "negative") == 1
    assert status(lib, read(k=None, v=None), "null") == 1
    assert status(lib, read(kp=None), "null") == 1
    assert status(lib, read(bt=None), "null") == 1
    assert status(lib, read(k=ODD), "aligned") == 1
    assert read(n=0) == 0

    def load(d=d, n=1, dst=4, k=P, src=P):
        return lib.pkv_quant_load_blocks(ctypes.byref(d), P, P, None, None, src, P, n, dst, k, P, None)
    assert status(lib, load(n=-1), "num_pairs") == 1
    assert status(lib, load(dst=0), "dst_num_blocks") == 1
    assert status(lib, load(k=None), "null") == 1
    assert status(lib, load(src=None), "null") == 1
    assert status(lib, load(k=ODD), "aligned") == 1
    assert load(n=0) == 0

    def decode(d=d, q=P, n=1, ctx=64, sm=1.0, window=-1, chunk=0, ws=P, out=P, lens=P):
        return lib.pkv_quant_decode(ctypes.byref(d), q, P, P, None, None, P, lens, n, ctx, sm, window,
                                    None, chunk, out, None, ws, 1 << 20, None)
    assert status(lib, decode(d=desc(kv_dtype=0)), "quantised") == 2
    assert status(lib, decode(n=65536), "num_seqs") == 1
    assert status(lib, decode(ctx=65), "max_context_len") == 1
    assert status(lib, decode(ctx=0), "max_context_len") == 1
    assert status(lib, decode(sm=0.0), "sm_scale") == 1
    assert status(lib, decode(sm=float("nan")), "sm_scale") == 1
    assert status(lib, decode(chunk=513), "chunk_blocks") == 1
    assert status(lib, decode(chunk=-1), "chunk_blocks") == 1
    assert status(lib, decode(q=None), "null") == 1
    assert status(lib, decode(out=ODD), "aligned") == 1
    assert status(lib, decode(d=desc(ring_blocks=2)), "ring") == 1
    assert status(lib, decode(d=desc(ring_blocks=2), window=18), "ring_blocks") == 1
    assert decode(n=0) == 0


def test_binding_refuses_wrong_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="device"):
        pkv.make_rope(z(4, 32, 2))
    with pytest.raises(ValueError, match="dtype"):
        pkv.make_rope(z(4, 32, 2, dtype=torch.float64))
    with pytest.raises(ValueError, match="pairs"):
        pkv.make_rope(z(4, 32, 2), rotary_dim=32)
    with pytest.raises(ValueError, match="layout"):
        pkv.make_rope(z(4, 32, 2), layout="swapped")
    d = desc()
    pool = z(10, 2, 2112, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_pool.*device"):
        pkv.pkv_quant_read(d, pool, pool, z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32),
                           z(1, dtype=torch.int32), z(1, 2, 128))
    with pytest.raises(ValueError, match="k_pool.*dtype"):
        pkv.pkv_quant_decode(d, z(1, 8, 128), pool.float(), pool, z(1, 4), z(1, dtype=torch.int32), 64,
                             1.0, z(1, 8, 128))


# ------------------------------------------------------------ scaled tables --

def table64(theta, r, n, kind, factor=1.0, L=0, low=1.0, high=4.0, attention=1.0):
    """The same frequencies from the formulas, pair by pair, in numpy doubles."""
    j = np.arange(r // 2, dtype=np.float64)
    f = theta ** (-2 * j / r)
    if kind == "linear":
        f = f / factor
    elif kind == "ntk":
        f = (theta * factor ** (r / (r - 2))) ** (-2 * j / r)
    elif kind == "banded":
        wave = 2 * np.pi / f
        mid = (L / wave - low) / (high - low)
        f = np.where(wave < L / high, f, np.where(wave > L / low, f / factor, (1 - mid) * f / factor + mid * f))
    elif kind == "yarn":
        at = lambda turns: r * np.log(L / (2 * np.pi * turns)) / (2 * np.log(theta))  # noqa: E731
        lo, hi = (float(np.clip(v, 0, r - 1)) for v in (np.floor(at(high)), np.ceil(at(low))))
        g = 1 - np.clip((j - lo) / ((hi - lo) or 0.001), 0, 1)
        f = (1 - g) * f / factor + g * f
    ang = np.arange(n, dtype=np.float64)[:, None] * f
    return np.stack((np.cos(ang), np.sin(ang)), -1) * attention


@pytest.mark.parametrize("kind,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
    ("banded", dict(factor=8.0, L=512, low=1.0, high=4.0)),
    ("yarn", dict(factor=16.0, L=512, low=1.0, high=32.0, attention=0.1 * np.log(16) + 1)),
    ("yarn", dict(factor=2.0, L=4, low=1.0, high=32.0))])
@pytest.mark.parametrize("theta,r", [(1e4, 64), (5e5, 128), (1e4, 18)])
def test_scaled_table(lib, kind, kw, theta, r):
    n = 3000
    c = {"L": "original_max_pos", "low": "low_freq", "high": "high_freq"}
    got = pkv.pkv_rope_scaled_table(theta, r, n, kind=kind, **{c.get(k, k): v for k, v in kw.items()})
    ref = table64(theta, r, n, kind, **kw)
    # half a step of fp32 (2^-24 of a value below 2), and the doubles' angle: n
    # times a frequency that two libms have 2^-50 apart
    assert got.shape == ref.shape
    assert np.abs(got - ref).max() <= 2.0 ** -24 * np.abs(ref).max() + n * 2.0 ** -50
    if kind == "none":
        assert np.array_equal(got, pkv.pkv_rope_cos_sin_table(theta, r, n))


def test_scaled_table_refusals(lib):
    bad = [dict(kind="linear", factor=0.5), dict(kind="linear", factor=float("inf")),
           dict(kind="banded", factor=2.0), dict(kind="yarn", factor=2.0, original_max_pos=64, low_freq=4.0,
                                                 high_freq=4.0),
           dict(kind="none", attention=0.0)]
    for kw in bad:
        with pytest.raises(pkv.PkvError):
            pkv.pkv_rope_scaled_table(1e4, 64, 8, **kw)
    with pytest.raises(pkv.PkvError):
        pkv.pkv_rope_scaled_table(1e4, 63, 8)
    with pytest.raises(pkv.PkvError):
        pkv.pkv_rope_scaled_table(1.0, 64, 8)
    with pytest.raises(pkv.PkvError):
        pkv.pkv_rope_scaled_table(1e4, 2, 8, kind="ntk", factor=2.0)
    with pytest.raises(ValueError):
        pkv.pkv_rope_scaled_table(1e4, 64, 8, kind="dynamic")
