"""The score rules', weights' and eviction's entry points without a GPU: refusals, which
return before any CUDA call, and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import _score as S
import paged_kv_attention_21_gb300 as pkv
from paged_kv_attention_21_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkv.load_library()


P, ODD2, ODD8 = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002), ctypes.c_void_p(0x1008)
P2, P3 = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)


def desc(**kw):
    a = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, num_blocks=10, max_blocks_per_seq=4)
    a.update(kw)
    return pkv.make_desc(**a)


def rule(**kw):
    a = dict(sm_scale=0.1, cap=0.0, window=0, reserved=0, slopes=None, sinks=None, prefix_lens=None)
    a.update(kw)
    return pkv.Score(**a)


def refused(st, code, word):
    assert st == code, (st, pkv.pkv_last_error())
    assert word in pkv.pkv_last_error(), pkv.pkv_last_error()


def ref(x):
    return None if x is None else ctypes.byref(x)


BAD_RULES = [(dict(sm_scale=0.0), "sm_scale"), (dict(sm_scale=-1.0), "sm_scale"), (dict(sm_scale=float("nan")), "sm_scale"),
             (dict(sm_scale=float("inf")), "sm_scale"), (dict(cap=-1.0), "cap"), (dict(cap=float("nan")), "cap"),
             (dict(cap=float("inf")), "cap"), (dict(cap=3e38), "cap"), (dict(cap=1e-45), "cap"),
             (dict(sm_scale=1e-30, cap=1e20), "cap"), (dict(reserved=1), "reserved"), (dict(slopes=0x1002), "aligned"),
             (dict(sinks=0x1001), "aligned"), (dict(prefix_lens=0x1002), "aligned")]


def call_decode(lib, r=rule(), d=None, **kw):
    a = dict(q=P, k=P, v=P, ks=None, vs=None, bt=P, lens=P, n=1, top=16, chunk=0, out=P2, lse=None, ws=None, size=0)
    a.update(kw)
    return lib.pkv_score_decode(ref(d or desc()), ref(r), a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["lens"],
                                a["n"], a["top"], a["chunk"], a["out"], a["lse"], a["ws"], a["size"], None)


def call_prefill(lib, r=rule(), d=None, **kw):
    a = dict(q=P, qo=P, k=P, v=P, ks=None, vs=None, bt=P, lens=P, n=1, total=4, qh=None, kh=None, causal=1, out=P2,
             lse=None)
    a.update(kw)
    host = lambda x: None if x is None else np.asarray(x, np.int32).ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    keep = [None if x is None else np.asarray(x, np.int32) for x in (a["qh"], a["kh"])]
    qh, kh = (None if x is None else x.ctypes.data_as(ctypes.c_void_p) for x in keep)
    return lib.pkv_score_prefill(ref(d or desc()), ref(r), a["q"], a["qo"], a["k"], a["v"], a["ks"], a["vs"], a["bt"],
                                 a["lens"], a["n"], a["total"], qh, kh, a["causal"], a["out"], a["lse"], None)


def call_mass(lib, r=rule(), d=None, **kw):
    a = dict(q=P, qo=P, k=P, ks=None, bt=P, lens=P, n=1, total=4, max_q=4, top=16, causal=1, lse=P, keep=1.0, mass=P2,
             stride=16)
    a.update(kw)
    return lib.pkv_score_mass(ref(d or desc()), ref(r), a["q"], a["qo"], a["k"], a["ks"], a["bt"], a["lens"], a["n"],
                              a["total"], a["max_q"], a["top"], a["causal"], a["lse"], a["keep"], a["mass"], a["stride"],
                              None)


@pytest.mark.parametrize("call", [call_decode, call_prefill, call_mass])
def test_score_rules_are_checked(lib, call):
    for kw, word in BAD_RULES:
        refused(call(lib, rule(**kw)), 1, word)
    refused(call(lib, None), 1, "score")
    refused(call(lib, d=desc(kv_dtype="int8")), 2, "pkv_quant_")
    refused(call(lib, d=desc(head_dim=96)), 2, "head_dim")
    refused(call(lib, d=desc(num_q_heads=34)), 2, "group")
    refused(call(lib, d=desc(kv_dtype="fp8_e4m3")), 1, "e4m3")
    refused(call(lib, n=-1), 1, "num_seqs")
    refused(call(lib, n=65536), 1, "num_seqs")
    refused(call(lib, q=ODD8), 1, "aligned")
    refused(call(lib, k=ODD8), 1, "aligned")
    for name in ("k", "bt", "lens"):
        refused(call(lib, **{name: None}), 1, "null")


def test_decode_refusals(lib):
    refused(call_decode(lib, top=0), 1, "max_context_len")
    refused(call_decode(lib, top=65), 1, "max_context_len")
    refused(call_decode(lib, chunk=257), 1, "chunk_blocks") if torch.cuda.is_available() else None
    refused(call_decode(lib, d=desc(ring_blocks=2)), 1, "window")
    refused(call_decode(lib, rule(window=100), d=desc(ring_blocks=2)), 1, "window")
    assert call_decode(lib, n=0) == 0


def test_prefill_refusals(lib):
    refused(call_prefill(lib, d=desc(ring_blocks=2)), 2, "ring")
    refused(call_prefill(lib, total=-1), 1, "total_q")
    refused(call_prefill(lib, qh=[0, 3]), 1, "qo_indptr_host")
    refused(call_prefill(lib, qh=[0, 4], kh=[3]), 1, "kv_len")
    refused(call_prefill(lib, qh=[0, 4], kh=[65]), 1, "kv_len")
    refused(call_prefill(lib, n=2, qh=[0, 5, 4], kh=[9, 9]), 1, "decreases")
    assert call_prefill(lib, total=0) == 0 and call_prefill(lib, n=0) == 0


def test_mass_refusals(lib):
    refused(call_mass(lib, d=desc(ring_blocks=2)), 2, "ring")
    refused(call_mass(lib, top=0), 1, "max_kv_len")
    refused(call_mass(lib, top=65, stride=100), 1, "max_kv_len")
    refused(call_mass(lib, top=17), 1, "max_kv_len")
    refused(call_mass(lib, max_q=-1), 1, "max_q_len")
    refused(call_mass(lib, total=-1), 1, "total_q")
    refused(call_mass(lib, qo=None), 1, "one query per sequence")
    refused(call_mass(lib, qo=None, total=1, max_q=2), 1, "one query per sequence")
    for keep in (-0.5, float("nan"), float("inf")):
        refused(call_mass(lib, keep=keep), 1, "keep")
    for name in ("q", "lse", "mass"):
        refused(call_mass(lib, **{name: None}), 1, "null")
    refused(call_mass(lib, mass=ODD2), 1, "aligned")
    refused(call_mass(lib, lse=ODD2), 1, "aligned")
    assert call_mass(lib, n=0, total=0) == 0


def call_select(lib, **kw):
    a = dict(mass=P, stride=100, lens=P, n=2, h=3, top=100, budget=10, first=2, recent=3, kept=P2, ks=10, kl=P3)
    a.update(kw)
    return lib.pkv_evict_select(a["mass"], a["stride"], a["lens"], a["n"], a["h"], a["top"], a["budget"], a["first"],
                                a["recent"], a["kept"], a["ks"], a["kl"], None)


def test_select_refusals(lib):
    for kw, word in ((dict(n=-1), "num_seqs"), (dict(n=65536), "num_seqs"), (dict(h=0), "num_kv_heads"),
                     (dict(top=0), "max_kv_len"), (dict(top=101), "max_kv_len"), (dict(budget=0), "budget"),
                     (dict(first=-1), "first"), (dict(recent=-1), "recent"), (dict(first=8), "budget"),
                     (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), "budget"), (dict(ks=9), "kept_stride"),
                     (dict(budget=2 ** 31 - 1, ks=99), "kept_stride"), (dict(mass=None), "null"), (dict(lens=None), "null"),
                     (dict(kept=None), "null"), (dict(kl=None), "null"), (dict(mass=ODD2), "aligned")):
        refused(call_select(lib, **kw), 1, word)
    assert call_select(lib, n=0) == 0


@pytest.mark.parametrize("at,n", [(0, 2), (4, 2), (-4, 2), (0, 1), (-4 * 65534, 65535), (4 * 65534, 65535)])
def test_select_refuses_lengths_written_over_those_it_reads(lib, at, n):
    lens = 0x500000
    refused(call_select(lib, n=n, lens=ctypes.c_void_p(lens), kl=ctypes.c_void_p(lens + at)), 1, "overlaps")


def call_compact(lib, d=None, dd=None, **kw):
    a = dict(k=P, v=P2, bt=P, kept=P, ks=8, kl=P, n=1, top=8, kd=ctypes.c_void_p(0x300000), vd=ctypes.c_void_p(0x400000),
             dt=P3, mass=None, ms=0, mo=None, mos=0)
    a.update(kw)
    return lib.pkv_evict_compact(ref(d or desc()), a["k"], a["v"], a["bt"], a["kept"], a["ks"], a["kl"], a["n"], a["top"],
                                 ref(dd or desc()), a["kd"], a["vd"], a["dt"], a["mass"], a["ms"], a["mo"], a["mos"], None)


def test_compact_refusals(lib):
    refused(call_compact(lib, d=desc(kv_dtype="fp4")), 2, "pkv_quant_")
    refused(call_compact(lib, dd=desc(kv_dtype="int8")), 2, "pkv_quant_")
    refused(call_compact(lib, d=desc(ring_blocks=1)), 2, "ring")
    refused(call_compact(lib, dd=desc(ring_blocks=1)), 2, "ring")
    for kw in (dict(num_kv_heads=4), dict(head_dim=64), dict(kv_dtype="fp8_e4m3")):
        refused(call_compact(lib, dd=desc(**kw)), 1, "differ")
    refused(call_compact(lib, top=9), 1, "max_kept")
    refused(call_compact(lib, top=-1), 1, "max_kept")
    refused(call_compact(lib, top=65, ks=100), 1, "max_kept")
    refused(call_compact(lib, mass=P), 1, "both or neither")
    refused(call_compact(lib, mass=P, mo=P2, ms=10, mos=7), 1, "mass_out_stride")
    refused(call_compact(lib, mass=P, mo=P2, ms=0, mos=8), 1, "mass_stride")
    refused(call_compact(lib, mass=P, mo=P, ms=8, mos=8), 1, "in place")
    for name in ("k", "v", "bt", "kept", "kl", "kd", "vd", "dt"):
        refused(call_compact(lib, **{name: None}), 1, "null")
    for name in ("k", "v", "kd", "vd"):
        refused(call_compact(lib, **{name: ODD8}), 1, "aligned")
    refused(call_compact(lib, kept=ODD2), 1, "aligned")
    # half in place: the same tables with other pools, or the pools crossed
    refused(call_compact(lib, dt=P), 1, "in place")
    refused(call_compact(lib, dt=P, kd=P, vd=P2, dd=desc(max_blocks_per_seq=5)), 1, "in place")
    refused(call_compact(lib, kd=P2), 1, "share")
    refused(call_compact(lib, vd=P), 1, "share")
    assert call_compact(lib, n=0) == 0 and call_compact(lib, top=0) == 0


def test_binding_refusals():
    with pytest.raises(ValueError, match="slopes"):
        pkv.make_score(0.1, slopes=torch.zeros(2, 3))
    with pytest.raises(ValueError, match="sinks"):
        pkv.make_score(0.1, sinks=torch.zeros(3, dtype=torch.float64))
    with pytest.raises(ValueError, match="prefix_lens"):
        pkv.make_score(0.1, prefix_lens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="on cpu"):
        pkv.make_score(0.1, slopes=torch.zeros(3))
    d, lens = desc(), torch.zeros(1, dtype=torch.int32)
    s = rule()
    s.tensors = (torch.zeros(8), None, None)  # not on the current device: held to it on every call
    args = (torch.zeros(1, 8, 128).bfloat16(), torch.zeros(10, 2, 16, 128).bfloat16(), None, None, lens, 16, None)
    with pytest.raises(ValueError, match="slopes: on cpu"):
        pkv.pkv_score_decode(d, s, *args)
    s.tensors = (None, None)
    with pytest.raises(ValueError, match="tensors"):
        pkv.pkv_score_decode(d, s, *args)
    with pytest.raises(ValueError, match="q: on cpu"):
        pkv.pkv_score_decode(d, rule(), *args)
    with pytest.raises(ValueError, match="all of them, or none"):
        pkv.pkv_evict_compact(d, None, None, None, None, lens, k_dst=torch.zeros(1))
    with pytest.raises(ValueError, match="mass is None"):
        pkv.pkv_evict_select(None, lens, 1, 1, 0, 0, None, None)


def test_plain_selection():
    w = np.array([5, 1, np.nan, 3, 3, -np.inf, 3, 9], np.float32)
    assert S.select(w, 8, 4, 1, 1).tolist() == [0, 3, 4, 7]
    assert S.select(w, 8, 6, 0, 0).tolist() == [0, 1, 3, 4, 6, 7]
    assert S.select(w, 8, 7, 0, 0).tolist() == [0, 1, 3, 4, 5, 6, 7]
    assert S.select(w, 3, 4, 0, 0).tolist() == [0, 1, 2]
    assert S.select(w, -1, 4, 0, 0).tolist() == []


def test_bounds_see_a_wrong_key():
    """What one key too many or too few changes lies far outside the bounds."""
    class Q:
        pass
    rng = np.random.default_rng(0)
    p = Q()
    p.hq, p.hkv, p.d, p.kv = 2, 1, 64, "bf16"
    p.k, p.v = [rng.standard_normal((40, 1, 64))], [rng.standard_normal((40, 1, 64))]
    r = S.Rule.__new__(S.Rule)
    r.scale, r.cap, r.window, r.causal, r.slopes, r.sinks, r.prefix = 0.125, 5.0, 0, True, None, None, None
    q = rng.standard_normal((1, 2, 64))
    o, lse, bo, bl = r.attend(p, 0, q, [39])
    o2, lse2, _, _ = r.attend(p, 0, q, [38])
    assert (np.abs(lse - lse2) > 100 * bl).all() and (np.abs(o - o2) > bo).mean() > 0.3
    m, bm = r.mass(p, 0, q, [39], lse)
    m2, _ = r.mass(p, 0, q, [38], lse)
    assert abs(m.sum() - 2) < 1e-9 and m2[0, 39] == 0 and m[0, 39] > 1e3 * bm[0, 39]
