"""Quantised decode where magnitudes lie far apart: scales whose product leaves fp32's range."""
import numpy as np
import pytest

import _quant as Q
import _quant_bound as B
import paged_kv_attention_21_gb300 as pkv
from test_gpu_quant_long import decode, within

pytestmark = pytest.mark.gpu


def check(fmt, p, q, tables, lens, o, lse, sm_scale, chunk=512, heads=None):
    for s, n in enumerate(lens):
        ro, rl, tol, ltol = B.attention(fmt, q[s].astype(np.float64), p.rows(0, tables[s], 0, n),
                                        p.rows(1, tables[s], 0, n), np.float64(np.float32(sm_scale)), chunk,
                                        p.units(tables[s], 0, n))
        at = slice(None) if heads is None else heads
        within(o[s][at], ro[at], tol[at], "o of sequence %d" % s)
        within(lse[s][at], rl[at], ltol[at], "lse of sequence %d" % s)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qvalue,sm_scale", [(1e-36, 1e-3), (1e-37, 1e-30), (1.0, 1e-38)])
def test_logits_below_all_numbers_weigh_alike(fmt, d, qvalue, sm_scale):
    """Scales whose product is no number of 32 bits: every visible key has the same weight,
    and none behind the end has any."""
    rng = np.random.default_rng(d)
    p = B.Pools(rng, fmt, 24, 2, d)
    lens = [1, 5, 17, 100, 150]
    tables = np.array([rng.permutation(24)[:10] for _ in lens], np.int32)
    q = Q.bf16(qvalue * rng.standard_normal((5, 6, d)))
    o, lse = decode(p, q, tables, lens, sm_scale=sm_scale)
    check(fmt, p, q, tables, lens, o, lse, sm_scale)
    assert pkv.pkv_device_errors() == 0
