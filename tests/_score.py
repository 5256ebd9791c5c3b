"""Plain numpy forms, in 64 bits, of attention under a score rule, of the weight that each
key receives, and of the choice of keys to keep; and bounds on what rounding may add."""
import numpy as np
import torch

import paged_kv_attention_21_gb300 as pkv

U_BF16, U_F16, U_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24  # half a step, relative to the value


class Paged:
    """K and V of sequences of the given lengths in scattered blocks of a pool whose unused
    slots hold NaN (bf16) or NaN codes (e4m3); k[s], v[s]: [len][Hkv][D] in 64 bits."""

    def __init__(self, lens, hq, hkv, d, kv="bf16", seed=0, spare=3, ring=0, window=0, device="cuda"):
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.kv, self.rng = list(lens), hq, hkv, d, kv, rng
        per = [(n + 15) // 16 if not ring else min(ring, (n + 15) // 16) for n in lens]
        nb = sum(per) + spare
        self.nb, self.ring = nb, ring
        perm = rng.permutation(nb)
        self.mbps = max(1, max(per, default=1), ring) + 1
        self.tables = np.full((len(lens), self.mbps), -1, np.int32)
        at = 0
        for s, n in enumerate(per):
            self.tables[s, :n] = perm[at:at + n]
            at += n
        self.k, self.v = [], []
        scales = [None, None]
        if kv != "bf16":
            scales = [(0.007 + 0.004 * rng.random(hkv)).astype(np.float32) for _ in range(2)]
        pools = []
        for which in range(2):
            pool = np.full((nb, hkv, 16, d), np.nan, np.float32)
            values = []
            for s, n in enumerate(lens):
                x = torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32))
                if kv == "bf16":
                    x = x.bfloat16().float().numpy()
                    values.append(x.astype(np.float64))
                else:
                    x = (x / torch.from_numpy(scales[which])[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
                    values.append(x.astype(np.float64) * scales[which].astype(np.float64)[:, None])
                lo = max(0, n - window) if ring else 0
                for t in range(lo, n):
                    b = t // 16 % ring if ring else t // 16
                    pool[self.tables[s, b], :, t % 16] = x[t]
            (self.k, self.v)[which].extend(values)
            pool = torch.from_numpy(pool)
            pools.append(pool.bfloat16() if kv == "bf16" else pool.to(torch.float8_e4m3fn).view(torch.uint8))
        self.k_pool, self.v_pool = (p.to(device) for p in pools)
        self.scales = dict(k_scale=None, v_scale=None) if kv == "bf16" else {
            n: torch.from_numpy(x).to(device) for n, x in zip(("k_scale", "v_scale"), scales)}
        self.desc = self.make_desc()
        self.t = torch.from_numpy(self.tables).to(device)
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.device = device

    def make_desc(self, **kw):
        a = dict(num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.d, num_blocks=self.nb,
                 max_blocks_per_seq=self.mbps, kv_dtype="bf16" if self.kv == "bf16" else "fp8_e4m3",
                 ring_blocks=self.ring)
        a.update(kw)
        return pkv.make_desc(**a)

    def queries(self, rows, scale=1.5):
        q = torch.from_numpy((scale * self.rng.standard_normal((rows, self.hq, self.d))).astype(np.float32)).bfloat16()
        return q.to(self.device), q.float().numpy().astype(np.float64)


class Rule:
    def __init__(self, d, hq, seqs, cap=0.0, slopes=None, sinks=False, window=0, prefix=None, causal=True, seed=0,
                 device="cuda"):
        rng = np.random.default_rng(seed + 77)
        self.scale, self.cap, self.window, self.causal = 1.0 / np.sqrt(d), cap, window, causal
        self.slopes = None if slopes is None else (slopes * 2.0 ** (-8.0 * (1 + np.arange(hq)) / hq)).astype(np.float32)
        self.sinks = rng.standard_normal(hq).astype(np.float32) if sinks else None
        self.prefix = None if prefix is None else np.asarray(prefix, np.int32)
        put = lambda x: None if x is None else torch.from_numpy(x).to(device)  # noqa: E731
        self.score = pkv.make_score(self.scale, cap=cap, slopes=put(self.slopes), sinks=put(self.sinks),
                                    window=window, prefix_lens=put(self.prefix))
        self.scale = float(np.float32(self.scale))

    def logits(self, p, s, q, pos):
        """[Hq][queries][keys], -inf where not seen, and a bound on an fp32 evaluation's error."""
        k = np.repeat(p.k[s], p.hq // p.hkv, 1).transpose(1, 2, 0)
        x = self.scale * (q.transpose(1, 0, 2) @ k)
        # a k-step of 16 dims at a time into an fp32 accumulator: two half steps for each
        err = self.scale * (np.abs(q).transpose(1, 0, 2) @ np.abs(k)) * (p.d / 16) * 4 * U_F32
        if p.kv != "bf16":  # q in f16: exact from 2^-14 on, else off by at most 2^-25
            err += self.scale * 2.0 ** -25 * np.abs(k).sum(1, keepdims=True)
        err += 4 * U_F32 * np.abs(x)  # the scale's factors and their products
        if self.cap:
            x = self.cap * np.tanh(x / self.cap)
            err += 3e-7 * self.cap * np.minimum(1, np.abs(x) / (0.2 * self.cap)) + 4 * U_F32 * np.abs(x)
        t, pos = np.arange(k.shape[2]), np.asarray(pos)[:, None]
        if self.slopes is not None:
            fall = self.slopes.astype(np.float64)[:, None, None] * np.abs(pos - t)
            x = x - fall
            err += 3 * U_F32 * np.abs(fall)
        err += 2 * U_F32 * np.abs(x)
        hi = np.full_like(pos, k.shape[2] - 1)
        if self.causal:
            hi = pos
            if self.prefix is not None:
                hi = np.where(pos < self.prefix[s], np.maximum(pos, self.prefix[s] - 1), pos)
        seen = (t <= hi) & ((t > pos - self.window) if self.window > 0 else True)
        return np.where(seen, x, -np.inf), err

    def attend(self, p, s, q, pos):
        """o [queries][Hq][D], lse, and bounds on both."""
        x, err = self.logits(p, s, q, pos)
        n = x.shape[2]
        err = np.where(x > -np.inf, err, 0).max(-1, initial=0.0)  # one factor of e^err on each weight
        top = x.max(-1, initial=-np.inf)
        if self.sinks is not None:
            top = np.maximum(top, self.sinks.astype(np.float64)[:, None])
        top = np.where(top == -np.inf, 0.0, top)
        w = np.exp(x - top[..., None])
        total = w.sum(-1)
        if self.sinks is not None:
            total = total + np.exp(self.sinks.astype(np.float64)[:, None] - top)
        with np.errstate(divide="ignore"):
            lse = top + np.log(total)
        w = w / np.where(total > 0, total, 1.0)[..., None]
        v = np.repeat(p.v[s], p.hq // p.hkv, 1).transpose(1, 0, 2)
        o = (w @ v).transpose(1, 0, 2)
        u = U_BF16 if p.kv == "bf16" else U_F16
        vmax = np.abs(v).max(initial=0.0)
        # weights: one rounding, e^err on numerator and denominator, exp2 and the sums 2^-20; f16
        # weights lose up to 2^-25 each against a largest of at least 2^-8; one rounding of o
        bound = (w @ np.abs(v)) * (u + 2 * err + 2.0 ** -20)[..., None] + n * vmax * 2.0 ** -17 * U_F32 * 2.0 ** 7 * (p.kv != "bf16")
        bound = bound.transpose(1, 0, 2) + U_BF16 * np.abs(o) + 1e-30
        lse_bound = err + 2.0 ** -20 + 6 * U_F32 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
        return o, lse.T, bound, lse_bound.T

    def mass(self, p, s, q, pos, lse, rows=None):
        """[Hkv][keys]: the weights' sums, and a bound; lse as given."""
        x, err = self.logits(p, s, q, pos)
        z = lse.astype(np.float64).T[..., None]
        with np.errstate(invalid="ignore"):
            w = np.where((x > -np.inf) & (z > -np.inf), np.exp(x - z), 0.0)
        zf = np.where(np.isfinite(z), np.abs(z), 0.0)
        # x - lse and its two factors of log2(e): three half steps of each; exp2 2^-22; the sum
        rel = err + 4 * U_F32 * (zf + np.abs(np.where(x > -np.inf, x, 0.0))) + 2.0 ** -20
        g = p.hq // p.hkv
        fold = lambda y: y.sum(1).reshape(p.hkv, g, -1).sum(1)  # noqa: E731
        return fold(w), fold(w * rel)


def close(got, want, bound, what=""):
    got = got.float().cpu().numpy().astype(np.float64) if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isinf(want) & (got == want))
    off = np.where(same, 0.0, np.abs(got - np.where(np.isinf(want), 0.0, want)))
    assert not np.isnan(got).any(), "%s: NaN" % what
    assert (np.isinf(want) == np.isinf(got)).all(), "%s: infinities differ" % what
    worst = (off - bound).argmax() if off.size else 0
    assert (off <= bound).all(), "%s: off by %g, bound %g, value %g" % (
        what, off.flat[worst], np.broadcast_to(bound, off.shape).flat[worst], want.flat[worst])


def select(mass, n, budget, first, recent):
    """The kept positions of one row of weights, ascending."""
    if n <= budget:
        return np.arange(max(n, 0))
    lo, hi = first, n - recent
    w = np.where(np.isnan(mass[lo:hi]), -np.inf, mass[lo:hi]).astype(np.float64)
    nan = np.isnan(mass[lo:hi])
    # a NaN is below -inf: sort by (is a number, value), the largest first, ties by position
    order = np.lexsort((np.arange(hi - lo), -w, nan))[:budget - first - recent]
    return np.concatenate([np.arange(lo), np.sort(order) + lo, np.arange(hi, n)])
