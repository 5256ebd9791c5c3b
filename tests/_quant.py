"""Plain numpy forms of the quantised pools and the rotary positions, written
from the format's definition, and the error bounds the tests hold kernels to."""
from __future__ import annotations

import numpy as np
import torch

BS = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(fmt, d):
    return d if fmt == "int8" else d // 2


def record_bytes(fmt, d):
    return 16 * d + 64 if fmt == "int8" else 8 * d + d


def code_offset(fmt, d, r, j):
    """Offset in a record of byte j of row r's codes."""
    rb = row_bytes(fmt, d)
    return r * rb + 16 * ((j // 16) ^ ((r * rb // 128) % (rb // 16))) + j % 16


def bf16(x):
    """fp32 array rounded to bf16 by torch, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().float().numpy()


def e4m3_bytes(x):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_values(b):
    t = torch.from_numpy(np.ascontiguousarray(b, np.uint8)).view(torch.float8_e4m3fn)
    return t.float().numpy()


def quantise(fmt, x, g):
    """One fp32 row [D] -> (code bytes [row_bytes], scale bytes)."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        mag = np.where(np.isfinite(x), np.abs(x), np.float32(0))
        if fmt == "int8":
            s = np.float32(mag.max() / np.float32(127))
            if not s > 0:
                y = np.zeros_like(x)
            else:
                y = (x / s).astype(np.float32)
            y = np.where(np.isnan(y), np.float32(0), y)
            c = np.clip(np.rint(y), -127, 127).astype(np.int64) + 128
            return c.astype(np.uint8), np.frombuffer(s.tobytes(), np.uint8)
        g = np.float32(g)
        b = x.reshape(-1, 16)
        e = np.minimum(mag.reshape(-1, 16).max(1) / np.float32(np.float32(6) * g), np.float32(448))
        sb = e4m3_bytes(e)
        t = (e4m3_values(sb) * g).astype(np.float32)[:, None]
        y = np.where(t > 0, (b / np.where(t > 0, t, 1)).astype(np.float32), np.float32(0))
        y = np.where(np.isnan(y), np.float32(0), y).reshape(-1)
        code = np.zeros(y.size, np.uint8)
        for i, v in enumerate(np.abs(y)):
            dist = np.abs(E2M1 - np.float64(min(v, 6.0)))
            best = np.flatnonzero(dist == dist.min())
            code[i] = best[0] if len(best) == 1 else best[best % 2 == 0][0]  # ties to the even code
        code |= (np.signbit(y).astype(np.uint8) << 3)
        return code[0::2] | (code[1::2] << 4), sb


def row_values(fmt, codes, scales, g):
    """Code and scale bytes of a row -> fp64 values (g included)."""
    if fmt == "int8":
        s = np.frombuffer(np.ascontiguousarray(scales).tobytes(), np.float32)[0]
        return (codes.astype(np.float64) - 128) * np.float64(s)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(-1)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(e4m3_values(scales).astype(np.float64), 16) * np.float64(np.float32(g))


def put_row(fmt, d, record, r, codes, scales):
    rb = row_bytes(fmt, d)
    for j in range(rb):
        record[code_offset(fmt, d, r, j)] = codes[j]
    sb = len(scales)
    record[16 * rb + r * sb:16 * rb + (r + 1) * sb] = scales


def get_row(fmt, d, record, r):
    rb = row_bytes(fmt, d)
    sb = 4 if fmt == "int8" else d // 16
    at = [code_offset(fmt, d, r, j) for j in range(rb)]
    return record[at], record[16 * rb + r * sb:16 * rb + (r + 1) * sb]


def pool_values(fmt, d, pool, g):
    """A pool [nb][Hkv][record] -> fp64 [nb][Hkv][16][D]; vectorised get_row."""
    rb = row_bytes(fmt, d)
    at = np.array([[code_offset(fmt, d, r, j) for j in range(rb)] for r in range(16)])
    codes = pool[..., at]
    if fmt == "int8":
        s = np.ascontiguousarray(pool[..., 16 * rb:]).view(np.float32)
        s = np.where(np.isnan(s), np.float32(np.nan), s)  # quiet: random bytes may be a signalling NaN
        return (codes.astype(np.float64) - 128) * s[..., None].astype(np.float64)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (d,))
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = e4m3_values(pool[..., 16 * rb:]).astype(np.float64).reshape(codes.shape[:-1] + (d // 16,))
    return v * np.repeat(s, 16, -1) * np.asarray(g, np.float32).astype(np.float64)[None, :, None, None]


def rotate(x, cs, layout, steps=np.float64, inverse=False):
    """Rows [..., D] turned by cs [r/2][2]; `steps` float32 rounds every op."""
    n = cs.shape[0]
    y = np.array(x, steps)
    c, s = cs[:, 0].astype(steps), cs[:, 1].astype(steps) * steps(-1 if inverse else 1)
    i0, i1 = ((np.arange(n), np.arange(n) + n) if layout == "half"
              else (2 * np.arange(n), 2 * np.arange(n) + 1))
    a, b = y[..., i0].copy(), y[..., i1].copy()
    y[..., i0] = a * c - b * s
    y[..., i1] = b * c + a * s
    return y


def attention(q, keys, vals, sm_scale, sinks=None):
    """fp64 decode of one sequence: q [Hq][D], keys / vals [T][Hkv][D].  Returns
    (o, lse, bound on |o - ref| of a bf16 result, bound on |lse - ref|).

    The bounds, term by term:
      * logits: D + 8 roundings of fp32 accumulation, each 2^-23 of sum |q||k|
        sm_scale (the products are exact), and 2^-21 |x| for the scaling and exp2;
        a logit off by dx moves a weight by a factor e^dx: 2 dx of sum w |v|;
      * a weight rounded to f16: 2^-11 of it, or 2^-25 below f16's normal range
        (relative to a weight >= 1, of n keys; int8 weights carry the row scale
        normalised to [1/64, 64] of the largest, hence 64 times that);
      * sums of n weights in fp32: at most n / 16 + 64 roundings of 2^-24;
      * the bf16 result: half a step, 2^-8."""
    hq, d = q.shape
    hkv = keys.shape[1]
    n = keys.shape[0]
    g = hq // hkv
    o = np.zeros((hq, d))
    lse = np.full(hq, -np.inf)
    bound, lbound = np.zeros((hq, d)), np.zeros(hq)
    for h in range(hq):
        k, v = keys[:, h // g], vals[:, h // g]
        x = sm_scale * (k @ q[h]) if n else np.zeros(0)
        every = np.append(x, sinks[h]) if sinks is not None else x
        if every.size == 0:
            continue
        m = every.max()
        total = np.exp(every - m).sum() if m > -np.inf else 0.0
        lse[h] = m + np.log(total) if total else -np.inf
        w = np.exp(x - lse[h])
        o[h] = w @ v if n else 0.0
        mass = w @ np.abs(v) if n else np.zeros(d)
        dx = ((d + 8) * 2.0 ** -23 * sm_scale * (np.abs(k) @ np.abs(q[h])).max() if n else 0.0)
        dx += 2.0 ** -21 * np.abs(every[np.isfinite(every)]).max(initial=0.0)  # a -inf sink adds nothing
        sums = (n / 16 + 64) * 2.0 ** -24
        bound[h] = (2.0 ** -8 * np.abs(o[h]) + mass * (2.0 ** -11 + 2 * dx + 2 * sums)
                    + (64 * n * 2.0 ** -25 * np.abs(v).max() if n else 0.0) + 2.0 ** -120)
        lbound[h] = dx + sums + 2.0 ** -21 * (1 + abs(lse[h]))
    return o, lse, bound, lbound


class QuantCase:
    """A quantised pool pair filled with rows of a given value scale, through
    scattered tables, with NaN scales in every slot that no sequence uses."""

    def __init__(self, rng, fmt, lens, hq, hkv, d, ring=0, value=1.0, extra=2, poison=True):
        self.fmt, self.hq, self.hkv, self.d, self.ring = fmt, hq, hkv, d, ring
        self.lens = np.asarray(lens, np.int32)
        nblk = np.minimum((self.lens + 15) // 16, ring) if ring else (self.lens + 15) // 16
        self.nb = int(nblk.sum()) + extra
        perm = rng.permutation(self.nb)
        self.mbps = max(1, int(nblk.max()) if len(nblk) else 1, ring)
        self.tables = np.full((len(lens), self.mbps), -1, np.int32)
        at = 0
        for s, k in enumerate(nblk):
            self.tables[s, :k] = perm[at:at + k]
            at += k
        self.k_scale = self.v_scale = None
        if fmt == "fp4":
            self.k_scale = (value * (3.5 + rng.random(hkv)) / 2688).astype(np.float32)
            self.v_scale = (value * (3.5 + rng.random(hkv)) / 2688).astype(np.float32)
        rec = record_bytes(fmt, d)
        self.pools = []
        for g in (self.k_scale, self.v_scale):
            bank = [quantise(fmt, value * rng.standard_normal(d).astype(np.float32),
                             1.0 if g is None else g[0]) for _ in range(64)]
            rb = row_bytes(fmt, d)
            at = np.array([[code_offset(fmt, d, r, j) for j in range(rb)] for r in range(16)])
            pick = rng.integers(0, 64, (self.nb, hkv, 16))
            pool = np.zeros((self.nb, hkv, rec), np.uint8)
            pool[..., at] = np.stack([c for c, _ in bank])[pick]
            sc = np.stack([s for _, s in bank])[pick]
            if poison:
                used = np.zeros((self.nb, 16), bool)
                for s, n in enumerate(self.lens):
                    for t in range(max(0, n - 16 * ring + 16) if ring else 0, n):
                        b = t // 16 % ring if ring else t // 16
                        used[self.tables[s, b], t % 16] = True
                bad = (np.frombuffer(np.float32(np.nan).tobytes(), np.uint8) if fmt == "int8"
                       else np.uint8(0x7F))
                sc = np.where(used[:, None, :, None], sc, bad)
            pool[..., 16 * rb:] = sc.reshape(self.nb, hkv, -1)
            self.pools.append(pool)
        self.q = bf16(rng.standard_normal((len(lens), hq, d)))

    def rows(self, which, s, lo, hi):
        """fp64 [hi - lo][Hkv][D] of sequence s."""
        g = (self.k_scale, self.v_scale)[which]
        vals = pool_values(self.fmt, self.d, self.pools[which], np.ones(self.hkv) if g is None else g)
        t = np.arange(lo, hi)
        b = t // 16 % self.ring if self.ring else t // 16
        return vals[self.tables[s, b], :, t % 16]
