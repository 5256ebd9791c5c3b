"""The error bound of the long quantised decodes on the CPU: at every length that a GPU test
holds to it, one wrong 16-token block of V or K lies beyond."""
import numpy as np
import pytest

import _quant as Q
import _quant_bound as B


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,chunk", [(700, 512), (2100, 129), (4000, 256), (9000, 512)])
def test_one_wrong_block_is_beyond_the_bound(fmt, d, n, chunk):
    rng = np.random.default_rng(n + d)
    p = B.Pools(rng, fmt, (n + 15) // 16 + 1, 1, d)
    table = rng.permutation(p.nb)[:(n + 15) // 16]
    q = Q.bf16(rng.standard_normal((2, d))).astype(np.float64)
    k, v, u = p.rows(0, table, 0, n), p.rows(1, table, 0, n), p.units(table, 0, n)
    sm = np.float64(np.float32(d ** -0.5))
    o, lse, tol, ltol = B.attention(fmt, q, k, v, sm, chunk, u)
    assert np.all(tol > 2.0 ** -8 * np.abs(o))  # no smaller than the result's own rounding
    for at in (0, n // 2 // 16 * 16, (n - 32) // 16 * 16):
        here = slice(at, at + 16)
        other = (at + n // 3) // 16 * 16 % (n - 16)
        for wrong in (np.zeros_like(v[here]), v[other:other + 16]):
            w = v.copy()
            w[here] = wrong
            bad = B.attention(fmt, q, k, w, sm, chunk, u)[0]
            assert (np.abs(bad - o) / tol).max(1).min() > 2, at  # in every head
        w = k.copy()
        w[here] = k[other:other + 16]
        bad, badl = B.attention(fmt, q, w, v, sm, chunk, u)[:2]
        assert (np.abs(bad - o) / tol).max(1).min() > 2, at


def test_the_bound_covers_a_rounded_decode():
    """A decode in the kernel's own steps -- f16 weights, fp32 sums, a bf16 result -- of random
    rows, and with one row of a far larger scale and little weight, stays within it."""
    rng = np.random.default_rng(5)
    for fmt in ("int8", "fp4"):
        for far in (False, True):
            p = B.Pools(rng, fmt, 130, 1, 64)
            table = rng.permutation(130)
            k, v, u = p.rows(0, table, 0, 2080), p.rows(1, table, 0, 2080), p.units(table, 0, 2080)
            q = Q.bf16(rng.standard_normal((1, 64))).astype(np.float64)
            x = 0.125 * (k[:, 0] @ q[0])
            if far:
                k[7, 0] = -40 * q[0] / 0.125 / (q[0] @ q[0])
                x[7] = -40
                if fmt == "int8":
                    u[7] *= 2.0 ** 20
                v[7] *= 2.0 ** 20
            w = np.exp2(np.float32(x / np.log(2) - np.ceil(x.max() / np.log(2))).astype(np.float32))
            total = w.astype(np.float64).sum()
            unit = u[:, 0] if fmt == "int8" else np.ones(2080)
            scale = 2.0 ** (4 - np.floor(np.log2((w * unit).max()))) if fmt == "int8" else 1.0
            f16 = (w * unit * scale).astype(np.float16).astype(np.float64) / scale
            o = Q.bf16(((f16[:, None] * (v[:, 0] / unit[:, None])).sum(0) / total).astype(np.float32))
            ro, rl, tol, ltol = B.attention(fmt, q, k, v, 0.125, 512, u)
            assert np.all(np.abs(o - ro[0]) <= tol[0]), (fmt, far)
