"""Decode over quantised pools in 64 bits with an error bound that a wrong block passes at no
tested length, and pools whose rows are all different.

The bound on one output element, term by term (w_i the key's share of the softmax, v_i its
value, x_i its logit, A_i = sm_scale sum_d |q_d k_id|):
  * logits: D + 8 roundings of 2^-23 of A_i (the products are exact), 2^-21 |x_i| for the
    scaling and exp2.  A logit off by dx_i moves o by at most w_i dx_i (|v_i| + |o|).
  * the weights' rounding to f16: half a step, 2^-11 of the weight, below f16's normal range
    2^-25 of the unit, and never more than the weight itself.  4-bit: the unit is at most the
    largest weight of the head.  int8: what is rounded is weight x row scale, normalised
    so that the largest of a head is at least 2^4 units.  Roundings of different keys are
    independent: by Hoeffding's inequality their sum is beyond 7 sqrt(sum a_i^2), a_i the
    largest single one, with a probability of 2 exp(-24.5) = 5e-11 an element.  Copies of a
    row (`copies` of them) round alike: their a_i add up first.
  * sums in fp32: a lane adds two weights a block and a warp takes every fourth of a chunk's
    blocks; then 3 + 4 + 13 additions join lanes, warps and chunks.  As many MMAs add to an
    element of O.  2^-23 each (an MMA may cut off where an addition rounds).
  * the result's rounding to bf16: half a step, 2^-8."""
from __future__ import annotations

import numpy as np

import _quant as Q


def attention(fmt, q, keys, vals, sm_scale, chunk, v_unit=None, copies=None, sinks=None):
    """q [Hq][D]; keys, vals [T][Hkv][D]; v_unit [T][Hkv]: int8 V row scales; copies [T].
    Returns o, lse and the bounds on |o - kernel's| and |lse - kernel's|."""
    hq, d = q.shape
    n, hkv = keys.shape[:2]
    o, lse = np.zeros((hq, d)), np.full(hq, -np.inf)
    tol, ltol = np.zeros((hq, d)), np.zeros(hq)
    c = np.ones(n) if copies is None else np.asarray(copies, np.float64)
    steps = 2 * (-(-chunk // 4)) + 20
    for h in range(hq):
        k, v = keys[:, h * hkv // hq], vals[:, h * hkv // hq]
        x = sm_scale * (k @ q[h])
        sink = -np.inf if sinks is None else sinks[h]
        m = max(x.max(initial=-np.inf), sink)
        if m == -np.inf:
            continue
        e = np.exp(x - m)
        total = (c * e).sum() + np.exp(sink - m)
        lse[h] = m + np.log(total)
        w = e / total  # of one copy
        o[h] = (c * w) @ v
        dx = (d + 8) * 2.0 ** -23 * sm_scale * (np.abs(k) @ np.abs(q[h])) + 2.0 ** -21 * np.abs(x)
        av = np.abs(v)
        if fmt == "int8":
            unit = v_unit[:, h * hkv // hq]
            p, code = w * unit, av / np.where(unit > 0, unit, 1)[:, None]
            a = np.maximum(2.0 ** -11 * p, np.minimum(p, 2.0 ** -29 * p.max(initial=0.0)))[:, None] * code
        else:
            a = np.maximum(2.0 ** -11 * w, np.minimum(w, 2.0 ** -25 * w.max(initial=0.0)))[:, None] * av
        mass = (c * w) @ av
        sums = steps * 2.0 ** -23
        lerr = ((c * w) @ dx + 2.0 ** -21 * np.abs(sink if np.isfinite(sink) else 0.0) + sums)
        tol[h] = ((c * w * dx) @ av + np.abs(o[h]) * lerr + 7 * np.sqrt(((c[:, None] * a) ** 2).sum(0)) + sums * mass)
        tol[h] = tol[h] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o[h]) + 2.0 ** -120
        ltol[h] = lerr + 2.0 ** -21 * (1 + np.abs(lse[h]))
    return o, lse, tol, ltol


class Pools:
    """K and V pools [nb][Hkv][record] of random rows, no two alike, of about N(0, 1) values."""

    def __init__(self, rng, fmt, nb, hkv, d):
        self.fmt, self.nb, self.hkv, self.d = fmt, nb, hkv, d
        rb = Q.row_bytes(fmt, d)
        self.raw, self.values, self.scales = [], [], [None, None]
        for which in range(2):
            if fmt == "int8":
                codes = rng.integers(1, 256, (nb, hkv, 16 * rb), dtype=np.uint8)
                unit = ((0.5 + rng.random((nb, hkv, 16))) / 73).astype(np.float32)
                tail = unit.view(np.uint8).reshape(nb, hkv, -1)
                g = np.ones(hkv)
            else:
                codes = rng.integers(0, 256, (nb, hkv, 16 * rb), dtype=np.uint8)
                tail = rng.integers(0x30, 0x40, (nb, hkv, d), dtype=np.uint8)  # e4m3 0.5 .. 1.875
                g = self.scales[which] = ((0.8 + 0.4 * rng.random(hkv)) / 3.5).astype(np.float32)
            pool = np.concatenate((codes, tail), -1)
            self.raw.append(pool)
            self.values.append(Q.pool_values(fmt, d, pool, g))  # [nb][Hkv][16][D]
            if fmt == "int8" and which == 1:
                self.v_unit = unit.astype(np.float64)

    def rows(self, which, table, lo, hi):
        """fp64 [hi - lo][Hkv][D] of positions lo .. hi - 1 under a table of block ids."""
        t = np.arange(lo, hi)
        return self.values[which][table[t // 16], :, t % 16]

    def units(self, table, lo, hi):
        t = np.arange(lo, hi)
        return self.v_unit[table[t // 16], :, t % 16] if self.fmt == "int8" else None
