"""Quantised decode where magnitudes lie far apart: scales whose product leaves fp32's range,
logits beyond 2^28, query heads of one group, V rows of one
sequence."""
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


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [4, 13])
@pytest.mark.parametrize("power", [20, 28, 40, 90])
def test_logits_whose_step_passes_one_leave_one_key(fmt, d, hq, power):
    """Logits of up to 2^93, steps of 2^70 apart: the largest one's row is the output wherever
    the second is further below than the logits' own rounding."""
    rng = np.random.default_rng(hq + power)
    p = B.Pools(rng, fmt, 60, 1, d)
    lens = [900, 33, 1]
    tables = np.array([rng.permutation(60)[:57] for _ in lens], np.int32)
    q = Q.bf16(rng.standard_normal((3, hq, d)) * 2.0 ** power)
    o, lse = decode(p, q, tables, lens)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse))
    clear = 0
    for s, n in enumerate(lens):
        k, v = p.rows(0, tables[s], 0, n)[:, 0], p.rows(1, tables[s], 0, n)[:, 0]
        x = np.float64(np.float32(d ** -0.5)) * (q[s].astype(np.float64) @ k.T)
        err = (d + 16) * 2.0 ** -23 * d ** -0.5 * (np.abs(q[s].astype(np.float64)) @ np.abs(k).T).max(1)
        at = x.argmax(1)
        within(lse[s], x.max(1), err + 2.0 ** -22 * np.abs(x.max(1)) + np.log(n), "lse of sequence %d" % s)
        for h in range(hq):
            rest = np.delete(x[h], at[h])
            if n == 1 or x[h].max() - rest.max() > 2 * err[h] + 40:
                # bf16's half a step, 2^-8 of the result; int8: the weight 1 x row scale is rounded
                # to f16 before it, 2^-11 of the value; the products and sums in fp32, some 2^-20
                tol = (2.0 ** -8 * (1 + 2.0 ** -10) + 2.0 ** -11 * (fmt == "int8") + 2.0 ** -20) * np.abs(v[at[h]])
                within(o[s, h], v[at[h]], tol + 2.0 ** -120, "o of head %d" % h)
                clear += 1
    assert clear > hq


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [4, 8, 13])
@pytest.mark.parametrize("power", [22, 40, 100, -22, -40, -90])
def test_a_query_head_far_from_the_others_of_its_group_spoils_none(fmt, d, hq, power):
    rng = np.random.default_rng(hq)
    p = B.Pools(rng, fmt, 60, 1, d)
    lens = [900, 33]
    tables = np.array([rng.permutation(60)[:57] for _ in lens], np.int32)
    q = Q.bf16(rng.standard_normal((2, hq, d)))
    q[:, hq - 2] *= np.float32(2.0 ** power)
    o, lse = decode(p, q, tables, lens)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse))
    check(fmt, p, q, tables, lens, o, lse, d ** -0.5,
          heads=[h for h in range(hq) if h != hq - 2 or power < 0])


def outlier_case(rng, d, hq, n, at, logit, power):
    """An int8 pool in which the rows `at` have a V scale 2^power above the others' and
    a K row that gives every head, whose queries share a direction, about `logit`."""
    p = B.Pools(rng, "int8", (n + 15) // 16 + 2, 1, d)
    table = rng.permutation(p.nb)[:(n + 15) // 16].astype(np.int32)
    base = rng.standard_normal(d)
    q = Q.bf16((base + 0.1 * rng.standard_normal((1, hq, d))))
    kcode = np.rint(127 * base / np.abs(base).max()).astype(np.int64)
    kscale = np.float32(logit * d ** 0.5 / float(kcode @ base))
    for t in at:
        b, r = table[t // 16], t % 16
        codes = (kcode if kscale > 0 else -kcode) + 128
        _, vscale = Q.get_row("int8", d, p.raw[1][b, 0], r)
        vcodes, _ = Q.get_row("int8", d, p.raw[1][b, 0], r)
        Q.put_row("int8", d, p.raw[0][b, 0], r, codes.astype(np.uint8),
                  np.frombuffer(np.abs(kscale).tobytes(), np.uint8))
        big = np.float32(np.frombuffer(vscale.tobytes(), np.float32)[0] * np.float32(2.0 ** power))
        Q.put_row("int8", d, p.raw[1][b, 0], r, vcodes, np.frombuffer(big.tobytes(), np.uint8))
        p.v_unit[b, 0, r] = big
    one = np.ones(1)
    p.values = [Q.pool_values("int8", d, raw, one) for raw in p.raw]
    return p, q, table[None]


@pytest.mark.parametrize("d,hq", [(64, 5), (128, 4), (64, 12), (128, 16)])
@pytest.mark.parametrize("power", [10, 24, 60, -24, -60])
@pytest.mark.parametrize("where", ["first", "last", "spread"])
@pytest.mark.parametrize("chunk", [512, 8])
def test_a_v_row_of_little_weight_spoils_none_by_its_scale(d, hq, power, where, chunk):
    """Rows with almost no weight under V scales far above the others' (the others keep their
    bits), or with almost all of it under scales far below."""
    rng = np.random.default_rng(hq + power if power > 0 else 1000 - power)
    n = 700
    at = {"first": [0], "last": [n - 1], "spread": [3, 90, 91, 300, 511, 640]}[where]
    p, q, tables = outlier_case(rng, d, hq, n, at, -120.0 if power > 0 else 25.0, power)
    o, lse = decode(p, q, tables, [n], chunk=chunk)
    check("int8", p, q, tables, [n], o, lse, d ** -0.5, chunk)


@pytest.mark.parametrize("d,hq", [(64, 5), (128, 16)])
def test_v_scales_that_rise_and_fall_with_the_weights(d, hq):
    """Logits that rise by 60 over the context while the V scales fall by 2^70, and the other way:
    early products that later ones leave far behind, and products that keep growing."""
    rng = np.random.default_rng(d)
    n = 1040
    for up in (1, -1):
        p = B.Pools(rng, "int8", n // 16, 1, d)
        table = rng.permutation(p.nb).astype(np.int32)
        base = rng.standard_normal(d)
        q = Q.bf16((base + 0.05 * rng.standard_normal((1, hq, d))))
        code = np.rint(127 * base / np.abs(base).max()).astype(np.int64) + 128
        for t in range(n):
            b, r = table[t // 16], t % 16
            part = (t if up > 0 else n - t) / n
            ks = np.float32(60 * part * d ** 0.5 / float((code - 128) @ base))
            vs = np.float32(2.0 ** (20 - 70 * part) * (1 + rng.random()))
            Q.put_row("int8", d, p.raw[0][b, 0], r, code.astype(np.uint8), np.frombuffer(ks.tobytes(), np.uint8))
            vcodes, _ = Q.get_row("int8", d, p.raw[1][b, 0], r)
            Q.put_row("int8", d, p.raw[1][b, 0], r, vcodes, np.frombuffer(vs.tobytes(), np.uint8))
            p.v_unit[b, 0, r] = vs
        p.values = [Q.pool_values("int8", d, raw, np.ones(1)) for raw in p.raw]
        for chunk in (512, 3):
            o, lse = decode(p, q, table[None], [n], chunk=chunk)
            check("int8", p, q, table[None], [n], o, lse, d ** -0.5, chunk)


def test_v_rows_that_are_all_zero():
    """Zero V scales, at first and throughout: nothing but zeros until the first number."""
    rng = np.random.default_rng(0)
    p = B.Pools(rng, "int8", 40, 1, 64)
    tables = np.arange(40, dtype=np.int32)[None]
    tail = p.raw[1][..., 16 * 64:].copy().view(np.float32)
    tail[:35] = 0
    p.raw[1][..., 16 * 64:] = tail.view(np.uint8)
    p.values[1] = Q.pool_values("int8", 64, p.raw[1], np.ones(1))
    p.v_unit[:35] = 0
    q = Q.bf16(rng.standard_normal((1, 4, 64)))
    for n in (16, 560, 640):
        o, lse = decode(p, q, tables, [n])
        check("int8", p, q, tables, [n], o, lse, 0.125)
        if n <= 560:
            assert not np.any(o)
