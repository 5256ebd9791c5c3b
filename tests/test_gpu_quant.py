"""The quantised pools on the GPU: append and read-back bit for bit, widening,
decode attention against 64 bits, and a sequence served through all of them."""
import numpy as np
import pytest
import torch

import _quant as Q
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().to(DEV)


def desc_of(fmt, hq, hkv, d, nb, mbps, ring=0):
    return pkv.make_desc(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, num_blocks=nb,
                         max_blocks_per_seq=mbps, kv_dtype=fmt, ring_blocks=ring)


# ------------------------------------------------------------ append, read --

def expected_append(fmt, d, pools, tables, ring, tts, pos, k, v, scales, cs, layout):
    """The pools after the append, from the definition, row by row."""
    out = [p.copy() for p in pools]
    for i, (s, p) in enumerate(zip(tts, pos)):
        if s < 0:
            continue
        b = p // 16 % ring if ring else p // 16
        kr = Q.rotate(k[i], cs[p], layout, np.float32) if cs is not None else k[i]
        for which, rows in ((0, kr), (1, v[i])):
            for h in range(rows.shape[0]):
                g = 1.0 if scales[which] is None else scales[which][h]
                Q.put_row(fmt, d, out[which][tables[s, b], h], p % 16, *Q.quantise(fmt, rows[h], g))
    return out


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hq,hkv,d,r,layout,packed,ring", [
    (8, 2, 64, 64, "half", False, 0), (16, 2, 128, 128, "half", True, 0), (5, 5, 128, 64, "interleaved", True, 0),
    (16, 1, 64, 18, "half", False, 3), (3, 3, 128, 0, "half", True, 0), (4, 4, 64, 32, "interleaved", False, 0)])
def test_append_is_the_definition_bit_for_bit(fmt, hq, hkv, d, r, layout, packed, ring):
    rng = np.random.default_rng(hq * d + r)
    lens = [1, 16, 17, 40, 3]
    n = sum(lens)
    nb, mbps = 16, max(3, ring)
    tables = np.full((len(lens), mbps), -1, np.int32)
    perm = iter(rng.permutation(nb))
    for s, ln in enumerate(lens):
        for b in range((ln + 15) // 16):
            tables[s, b] = next(perm)
    tts = np.repeat(np.arange(len(lens)), lens).astype(np.int32)
    pos = np.concatenate([np.arange(ln) for ln in lens]).astype(np.int32)
    if ring:  # far positions, each slot still its own
        pos = pos + 16 * ring * 5
    order = rng.permutation(n)
    tts, pos = tts[order], pos[order]
    tts[2] = -1  # padding
    qkv = Q.bf16(rng.standard_normal((n, hq + 2 * hkv, d)) * np.exp(rng.standard_normal((n, hq + 2 * hkv, 1))))
    qkv[0, hq] = 0.0            # a zero row
    qkv[1, hq + hkv, :16] = 0.0  # a zero block of a row
    qkv[3, hq, 5] = 1e-30
    k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    scales = ((0.0017 * (1 + rng.random(hkv))).astype(np.float32),
              (0.0017 * (1 + rng.random(hkv))).astype(np.float32)) if fmt == "fp4" else (None, None)
    rec = Q.record_bytes(fmt, d)
    pools = [rng.integers(0, 256, (nb, hkv, rec)).astype(np.uint8) for _ in range(2)]
    cs = pkv.pkv_rope_scaled_table(1e4, r, 400, kind="yarn", factor=4.0, original_max_pos=100,
                                   attention=1.1) if r else None
    rope = pkv.make_rope(dev(cs), layout=layout) if r else None
    buf = bf(qkv)
    qd, kd, vd = buf[:, :hq], buf[:, hq:hq + hkv], buf[:, hq + hkv:]
    if not packed:
        qd, kd, vd = qd.contiguous(), kd.contiguous(), vd.contiguous()
    gp = [dev(p) for p in pools]
    qo = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    dd = desc_of(fmt, hq, hkv, d, nb, mbps, ring)
    ks, vs = (dev(s) for s in scales)
    pkv.pkv_quant_append(dd, gp[0], gp[1], dev(tables), dev(tts), dev(pos), kd, vd,
                         q=qd if r else None, q_out=qo if r else None, rope=rope, k_scale=ks, v_scale=vs)
    ref = expected_append(fmt, d, pools, tables, ring, tts, pos, k, v, scales, cs, layout)
    assert pkv.pkv_device_errors() == 0
    for which in (0, 1):
        assert np.array_equal(gp[which].cpu().numpy(), ref[which]), "pool %d" % which
    if r:
        want = np.stack([Q.rotate(qkv[i, :hq], cs[p], layout, np.float32) for i, p in enumerate(pos)])
        want = torch.from_numpy(want).bfloat16()
        want[2] = 7.0
        assert torch.equal(qo.cpu(), want)
        pkv.pkv_quant_append(dd, gp[0], gp[1], dev(tables), dev(tts), dev(pos), kd, vd, q=qd, rope=rope,
                             k_scale=ks, v_scale=vs)  # q in place, the same bits
        want[2] = torch.from_numpy(qkv[2, :hq]).bfloat16()
        assert torch.equal(qd.cpu(), want)
    # read back, both types, and one of the two alone
    for dtype in (torch.float32, torch.bfloat16):
        outs = [torch.full((n, hkv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
        pkv.pkv_quant_read(dd, gp[0], gp[1], dev(tables), dev(tts), dev(pos), outs[0], outs[1],
                           k_scale=ks, v_scale=vs)
        alone = torch.empty_like(outs[1])
        alone.fill_(7.0)
        pkv.pkv_quant_read(dd, gp[0], gp[1], dev(tables), dev(tts), dev(pos), v_out=alone, k_scale=ks,
                           v_scale=vs)
        assert torch.equal(alone, outs[1])
        for which in (0, 1):
            vals = Q.pool_values(fmt, d, ref[which], np.ones(hkv) if scales[which] is None else scales[which])
            b = pos // 16 % ring if ring else pos // 16
            want = vals[tables[tts, b], :, pos % 16].astype(np.float32)  # the fp64 product, rounded once
            want[2] = 7.0
            assert torch.equal(outs[which].cpu(), torch.from_numpy(want).to(dtype))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_append_rounds_quotients_at_the_borders(fmt):
    """K rows of chosen fp32 values -- k = 1 rotated by (cos, sin) = (value, 0) -- that
    sit on, and a few steps beside, the borders between codes, under scales of random
    significands and exponents: every quotient must round as the division does."""
    rng = np.random.default_rng(12)
    d, n = 128, 512
    half = d // 2
    mids = (np.arange(127) + 0.5) if fmt == "int8" else np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    cs = np.zeros((n, half, 2), np.float32)
    g = np.ones(1, np.float32) * np.float32(1.2345e-3)
    for i in range(n):
        if i % 2 and fmt == "fp4":  # all-ones and near-power-of-two significands too
            g_amax = np.float32(2.0 ** rng.integers(-6, 6) * (2 - 2.0 ** -23 * rng.integers(0, 4)))
        else:
            g_amax = np.float32(2.0 ** rng.integers(-6, 6) * (1 + rng.random()))
        row = np.empty(half, np.float32)
        for b in range(0, half, 16):
            # the scale that this amax gives, then values at its borders
            _, sc = Q.quantise(fmt, np.concatenate(([g_amax], np.zeros(half - 1))).astype(np.float32), g[0])
            t = (np.frombuffer(sc.tobytes(), np.float32)[0] if fmt == "int8"
                 else np.float32(Q.e4m3_values(sc[:1])[0] * g[0]))
            v = (rng.choice(mids, 16).astype(np.float64) * np.float64(t)).astype(np.float32)
            v = (v.view(np.int32) + rng.integers(-2, 3, 16).astype(np.int32)).view(np.float32)
            v = np.clip(v * rng.choice([-1, 1], 16), -g_amax, g_amax).astype(np.float32)
            v[0] = g_amax
            row[b:b + 16] = v
        cs[i, :, 0] = row
    k = np.zeros((n, 1, d), np.float32)
    k[..., :half] = 1.0
    k[:, :, half:][..., ::7] = -0.0
    v = Q.bf16(rng.standard_normal((n, 1, d)))
    tables = np.arange(n // 16, dtype=np.int32)[None]
    tts, pos = np.zeros(n, np.int32), np.arange(n, dtype=np.int32)
    scale = g if fmt == "fp4" else None
    pools = [np.zeros((n // 16, 1, Q.record_bytes(fmt, d)), np.uint8) for _ in range(2)]
    gp = [dev(p) for p in pools]
    pkv.pkv_quant_append(desc_of(fmt, 1, 1, d, n // 16, n // 16), gp[0], gp[1], dev(tables), dev(tts), dev(pos),
                         bf(k), bf(v), rope=pkv.make_rope(dev(cs)), q=bf(k), q_out=bf(k), k_scale=dev(scale),
                         v_scale=dev(scale))
    ref = expected_append(fmt, d, pools, tables, 0, tts, pos, k, v, (scale, scale), cs, "half")
    for which in (0, 1):
        assert np.array_equal(gp[which].cpu().numpy(), ref[which])


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_append_of_values_that_are_not_finite_and_of_extremes(fmt):
    d, nb = 64, 2
    rows = np.zeros((12, d), np.float32)
    rng = np.random.default_rng(1)
    rows[:] = rng.standard_normal((12, d))
    rows[0, 3] = np.nan
    rows[1, 4], rows[1, 20] = np.inf, -np.inf
    rows[2] = np.nan
    rows[3] = np.inf
    rows[4] = 3e38
    rows[5] = 1e-38
    rows[6] = 1e-40 * np.arange(d)
    rows[7] = 0.0
    rows[8] = -0.0
    rows[9, 0] = 3.3e38
    rows[10] *= 1e-20
    rows[11] *= 1e20
    rows = Q.bf16(rows)
    tables = np.array([[1]], np.int32)
    g = np.array([4 / 2688], np.float32) if fmt == "fp4" else None
    pools = [np.zeros((nb, 1, Q.record_bytes(fmt, d)), np.uint8) for _ in range(2)]
    tts, pos = np.zeros(12, np.int32), np.arange(12, dtype=np.int32)
    gp = [dev(p) for p in pools]
    pkv.pkv_quant_append(desc_of(fmt, 1, 1, d, nb, 1), gp[0], gp[1], dev(tables), dev(tts), dev(pos),
                         bf(rows[:, None]), bf(rows[:, None]), k_scale=dev(g), v_scale=dev(g))
    ref = expected_append(fmt, d, pools, tables, 0, tts, pos, rows[:, None], rows[:, None], (g, g), None, "half")
    for which in (0, 1):
        assert np.array_equal(gp[which].cpu().numpy(), ref[which])


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_bad_tokens_are_flagged_and_skipped(fmt):
    d, hkv, nb = 128, 2, 3
    dd = desc_of(fmt, 4, hkv, d, nb, 2)
    tables = dev(np.array([[0, 5], [-1, 2]], np.int32))
    tts = dev(np.array([2, 0, 0, 0, 1, -1, 1], np.int32))
    pos = dev(np.array([0, 32, -1, 16, 0, 999, 17], np.int32))
    x = torch.randn(7, hkv, d, device=DEV).bfloat16()
    g = torch.full((hkv,), 0.002, device=DEV) if fmt == "fp4" else None
    pools = [torch.zeros(nb, hkv, Q.record_bytes(fmt, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    pkv.pkv_quant_append(dd, pools[0], pools[1], tables, tts, pos, x, x, k_scale=g, v_scale=g)
    assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION | pkv.DEVERR_BLOCK_ID
    for p in pools:
        used = p.view(nb, -1).ne(0).any(1).tolist()
        assert used == [False, False, True]
    out = torch.full((7, hkv, d), 7.0, device=DEV)
    pkv.pkv_quant_read(dd, pools[0], pools[1], tables, tts, pos, out, k_scale=g, v_scale=g)
    assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION | pkv.DEVERR_BLOCK_ID
    assert torch.all(out[:6] == 7) and not torch.any(out[6] == 7)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hkv,d", [(1, 64), (8, 64), (3, 128), (8, 128)])
def test_load_blocks_and_copy_blocks(fmt, hkv, d):
    rng = np.random.default_rng(hkv + d)
    c = Q.QuantCase(rng, fmt, [16 * 5], hkv, hkv, d, extra=3, poison=False)
    dd = desc_of(fmt, hkv, hkv, d, c.nb, c.mbps)
    gp = [dev(p) for p in c.pools]
    src = np.array([4, 0, 7, c.nb, 2], np.int32)
    dst = np.array([1, 3, 0, 2, 9], np.int32)
    outs = [torch.full((6, hkv, 16, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.pkv_quant_load_blocks(dd, gp[0], gp[1], dev(src), dev(dst), outs[0], outs[1],
                              k_scale=dev(c.k_scale), v_scale=dev(c.v_scale))
    assert pkv.pkv_device_errors() == pkv.DEVERR_BLOCK_ID
    for which, g in ((0, c.k_scale), (1, c.v_scale)):
        vals = Q.pool_values(fmt, d, c.pools[which], np.ones(hkv) if g is None else g)
        want = torch.full((6, hkv, 16, d), 7.0, dtype=torch.bfloat16)
        for s, t in ((4, 1), (0, 3), (7, 0)):
            want[t] = torch.from_numpy(vals[s].astype(np.float32)).bfloat16()
        assert torch.equal(outs[which].cpu(), want)
    pkv.pkv_copy_blocks(dd, gp[0], gp[1], dev(np.array([4, 2], np.int32)), dev(np.array([0, 6], np.int32)))
    for which in (0, 1):
        want = c.pools[which].copy()
        want[0], want[6] = want[4], want[2]
        assert np.array_equal(gp[which].cpu().numpy(), want)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hq,hkv,d,r,layout,where", [
    (8, 2, 64, 64, "half", "packed"), (8, 2, 64, 32, "half", "in place"), (12, 3, 128, 128, "half", "in place"),
    (5, 1, 128, 48, "interleaved", "packed"), (6, 6, 64, 64, "interleaved", "in place"),
    (16, 1, 128, 96, "half", "alternating"), (6, 2, 128, 18, "half", "in place"),
    (5, 1, 64, 16, "half", "packed"), (9, 3, 64, 50, "half", "alternating"), (6, 2, 128, 22, "interleaved", "in place")])
def test_append_of_many_tokens_is_the_append_of_few(fmt, hq, hkv, d, r, layout, where):
    """One call of so many tokens that q gets blocks of its own, against calls of 500:
    the same bits in pools and q_out, padding, bad positions, bad blocks and a ring
    included (a bad block keeps its token's q)."""
    rng = np.random.default_rng(hq * d + r)
    n = (3 << 16) // ((hq + 2 * hkv) * (d // 16)) + 777
    seqs, ring = 37, 0 if where == "packed" else 8
    mbps = ((n // seqs + 16) // 16 if not ring else ring) + 1
    pos = (np.arange(n) // seqs).astype(np.int32)
    if ring:  # the last rounds of the ring: every slot its own
        pos = pos % (16 * ring) + 16 * ring * 3
    tts = (np.arange(n) % seqs).astype(np.int32)
    if ring:
        tts[seqs * 16 * ring:] = -1  # further tokens would meet the first ones' slots
    nb = seqs * mbps
    tables = rng.permutation(nb).astype(np.int32).reshape(seqs, mbps)
    tables[3, 0], tables[5, 0] = nb, -1
    tts[[7, n // 2, n - 2]] = -1
    tts[100], pos[200], pos[300] = seqs, -5, 10 ** 6
    cs = pkv.pkv_rope_scaled_table(1e4, r, 16 * ring * 4 if ring else n // seqs + 1)
    rope = pkv.make_rope(dev(cs), layout=layout, inverse=where == "alternating")
    buf = torch.randn(n, hq + 2 * hkv, d, device=DEV).bfloat16()
    k, v = buf[:, hq:hq + hkv], buf[:, hq + hkv:]
    g = dev(np.full(hkv, 4 / 2688, np.float32)) if fmt == "fp4" else None
    dd = desc_of(fmt, hq, hkv, d, nb, mbps, ring)
    td, sd, pd = dev(tables), dev(tts), dev(pos)

    def run(step):
        pools = [torch.full((nb, hkv, Q.record_bytes(fmt, d)), 77, dtype=torch.uint8, device=DEV) for _ in range(2)]
        if where == "alternating":  # q and q_out rows in turn in one buffer
            both = torch.full((n, 2, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
            both[:, 0] = buf[:, :hq]
            q, qo = both[:, 0], both[:, 1]
        elif where == "packed":
            q, qo = buf[:, :hq], torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        else:
            q, qo = buf[:, :hq].clone(), None
        for i in range(0, n, step):
            at = slice(i, i + step)
            pkv.pkv_quant_append(dd, pools[0], pools[1], td, sd[at], pd[at], k[at], v[at], q=q[at],
                                 q_out=None if qo is None else qo[at], rope=rope, k_scale=g, v_scale=g)
        assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION | pkv.DEVERR_BLOCK_ID
        return pools + [q, q if qo is None else qo]
    many, few = run(n), run(500)
    for a, b in zip(many, few):
        assert torch.equal(a, b)
    # the rotation itself, bit for bit
    x = buf[:, :hq].float().cpu().numpy()
    got = many[3].cpu()
    for i in list(range(0, n, 97)) + [3, 5, 7, 100, 200, 300]:
        bad = tts[i] < 0 or tts[i] >= seqs or pos[i] < 0 or pos[i] >= len(cs)
        if bad:
            want = torch.from_numpy(x[i]).bfloat16() if where == "in place" else torch.full((hq, d), 7.0).bfloat16()
        else:
            want = torch.from_numpy(Q.rotate(x[i], cs[pos[i]], layout, np.float32,
                                             inverse=where == "alternating")).bfloat16()
        assert torch.equal(got[i], want), i


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hkv,d", [(3, 128), (8, 64), (5, 64)])
def test_load_of_many_blocks_is_the_load_of_few(fmt, hkv, d):
    """So many pairs that a CTA takes four heads (groups of four left incomplete too)."""
    rec, pairs = Q.record_bytes(fmt, d), 16 * 152 * 512 // (2 * d * hkv) + 11
    gen = torch.Generator().manual_seed(d)
    nb = 97
    pools = [torch.randint(0, 256, (nb, hkv, rec), generator=gen, dtype=torch.uint8) for _ in range(2)]
    for p in pools:  # scales that are numbers
        at = p[..., 16 * Q.row_bytes(fmt, d):]
        at.copy_(torch.rand(nb, hkv, 16, generator=gen).view(torch.uint8) if fmt == "int8" else at % 0x7F)
    pools = [p.to(DEV) for p in pools]
    src = torch.randint(0, nb, (pairs,), generator=gen).int()
    dst = torch.randperm(pairs, generator=gen).int()
    src[5], dst[9] = nb, -1
    src, dst = src.to(DEV), dst.to(DEV)
    g = torch.rand(hkv, generator=gen).to(DEV) + 0.01 if fmt == "fp4" else None
    dd = desc_of(fmt, hkv, hkv, d, nb, 4)

    def run(step):
        outs = [torch.full((pairs, hkv, 16, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        for i in range(0, pairs, step):
            pkv.pkv_quant_load_blocks(dd, pools[0], pools[1], src[i:i + step], dst[i:i + step], outs[0], outs[1],
                                      k_scale=g, v_scale=g)
        assert pkv.pkv_device_errors() == pkv.DEVERR_BLOCK_ID
        return outs
    for a, b in zip(run(pairs), run(50)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hkv,d,out", [(3, 128, torch.float32), (8, 64, torch.bfloat16), (5, 128, torch.bfloat16)])
def test_read_of_many_rows_is_the_read_of_few(fmt, hkv, d, out):
    """So many rows that a thread takes four heads (groups of four left incomplete too),
    the same row twice, padding, bad positions and blocks among them."""
    gen = torch.Generator().manual_seed(d + hkv)
    n, nb, mbps, seqs = 4 * 152 * 512 // (hkv * d // 8) + 13, 61, 7, 9
    pools = [torch.randint(0, 256, (nb, hkv, Q.record_bytes(fmt, d)), generator=gen, dtype=torch.uint8) for _ in range(2)]
    for p in pools:  # scales that are numbers
        at = p[..., 16 * Q.row_bytes(fmt, d):]
        at.copy_(torch.rand(nb, hkv, 16, generator=gen).view(torch.uint8) if fmt == "int8" else at % 0x7F)
    pools = [p.to(DEV) for p in pools]
    tables = torch.randint(0, nb, (seqs, mbps), generator=gen).int()
    tables[2, 3], tables[4, 0] = nb, -1
    tts = torch.randint(0, seqs, (n,), generator=gen).int()
    pos = torch.randint(0, 16 * mbps, (n,), generator=gen).int()
    tts[[3, n // 2]], tts[9], pos[11], pos[n - 1] = -1, seqs, -4, 16 * mbps
    tables, tts, pos = tables.to(DEV), tts.to(DEV), pos.to(DEV)
    g = torch.rand(hkv, generator=gen).to(DEV) + 0.01 if fmt == "fp4" else None
    dd = desc_of(fmt, hkv, hkv, d, nb, mbps)

    def run(step, which=(0, 1)):
        outs = [torch.full((n, hkv, d), 7.0, dtype=out, device=DEV) for _ in range(2)]
        for i in range(0, n, step):
            at = slice(i, i + step)
            pkv.pkv_quant_read(dd, pools[0] if 0 in which else None, pools[1] if 1 in which else None, tables, tts[at],
                               pos[at], outs[0][at] if 0 in which else None, outs[1][at] if 1 in which else None,
                               k_scale=g, v_scale=g)
        assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION | pkv.DEVERR_BLOCK_ID
        return outs
    few = run(300)
    many = run(n)
    assert torch.equal(many[0], few[0]) and torch.equal(many[1], few[1])
    assert torch.all(few[0][torch.tensor([3, 9, 11, n // 2, n - 1], device=DEV)] == 7)
    assert torch.equal(run(n, (1,))[1], few[1]) and torch.equal(run(n, (0,))[0], few[0])


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_the_binding_refuses_tensors_that_do_not_fit(fmt):
    hq, hkv, d, nb, mbps, n = 8, 2, 64, 4, 2, 3
    dd = desc_of(fmt, hq, hkv, d, nb, mbps)
    i32 = dict(dtype=torch.int32, device=DEV)
    ok = dict(k_pool=torch.zeros(nb, hkv, Q.record_bytes(fmt, d), dtype=torch.uint8, device=DEV),
              block_tables=torch.zeros(1, mbps, **i32), token_to_seq=torch.full((n,), -1, **i32),
              positions=torch.zeros(n, **i32))
    ok["v_pool"] = ok["k_pool"].clone()
    if fmt == "fp4":
        ok.update(k_scale=torch.ones(hkv, device=DEV), v_scale=torch.ones(hkv, device=DEV))
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    x, q = torch.zeros(n, hkv, d, **bf16), torch.zeros(n, hq, d, **bf16)
    rope = pkv.make_rope(torch.zeros(8, d // 2, 2, device=DEV))

    def refused(fn, error, text, base, **kw):
        with pytest.raises(error, match=text):
            fn(desc=dd, **dict(base, **kw))
    app = dict(ok, k_new=x, v_new=x, q=q, rope=rope)
    pkv.pkv_quant_append(desc=dd, **app)  # all padding: nothing is written
    assert not torch.any(ok["k_pool"]) and not torch.any(ok["v_pool"])
    f = pkv.pkv_quant_append
    refused(f, TypeError, "k_new: expected a tensor", app, k_new=[1.0])
    refused(f, ValueError, "k_new is None", app, k_new=None)
    refused(f, ValueError, "k_new: dtype", app, k_new=x.float())
    refused(f, ValueError, "k_new: shape", app, k_new=x[:2])
    refused(f, ValueError, "heads must be contiguous", app, k_new=torch.zeros(n, d, hkv, **bf16).transpose(1, 2))
    refused(f, ValueError, "strides .* differ", app, k_new=torch.zeros(n, 2 * hkv, d, **bf16)[:, :hkv])
    refused(f, ValueError, "q: shape", app, q=x)
    refused(f, ValueError, "q_out: dtype", app, q_out=q.half())
    refused(f, ValueError, "k_pool: dtype", app, k_pool=ok["k_pool"].to(torch.int8))
    refused(f, ValueError, "v_pool: shape", app, v_pool=ok["v_pool"][..., 1:])
    refused(f, ValueError, "v_pool: .*contiguous", app,
            v_pool=torch.zeros(hkv, nb, ok["k_pool"].shape[2], dtype=torch.uint8, device=DEV).transpose(0, 1))
    refused(f, ValueError, "positions: dtype", app, positions=ok["positions"].long())
    refused(f, ValueError, "token_to_seq: shape", app, token_to_seq=ok["token_to_seq"][:1])
    refused(f, ValueError, "block_tables: shape", app, block_tables=torch.zeros(1, mbps + 1, **i32))
    refused(f, ValueError, "positions: on cpu", app, positions=ok["positions"].cpu())
    refused(f, TypeError, "bytes-like", app, rope=3)
    refused(f, pkv.PkvError, "without a rotation", app, rope=None)
    refused(f, pkv.PkvError, "rotary_dim", app, rope=pkv.make_rope(torch.zeros(8, d, 2, device=DEV)))
    scales = dict(k_scale=None) if fmt == "fp4" else dict(k_scale=torch.ones(hkv, device=DEV))
    refused(f, pkv.PkvError, "k_scale", app, **scales)
    refused(f, ValueError, "v_scale: shape", app, v_scale=torch.ones(hkv + 1, device=DEV))
    flat = torch.zeros(n * hkv * d + 8, **bf16)
    refused(f, pkv.PkvError, "aligned", app, k_new=flat[1:1 + x.numel()].view(x.shape))
    read = dict(ok, k_out=x.clone(), v_out=x.clone())
    f = pkv.pkv_quant_read
    refused(f, ValueError, "k_out or v_out", read, k_out=None, v_out=None)
    refused(f, ValueError, "dtype", read, k_out=x.half(), v_out=x.half())
    refused(f, ValueError, "v_out: dtype", read, v_out=x.float())
    refused(f, ValueError, "k_out: shape", read, k_out=q)
    bases = {k: ok[k] for k in ("k_pool", "v_pool", "k_scale", "v_scale") if k in ok}
    cache = torch.zeros(5, hkv, 16, d, **bf16)
    load = dict(bases, src_blocks=torch.zeros(2, **i32), dst_blocks=torch.zeros(2, **i32), k_cache=cache,
                v_cache=cache.clone())
    f = pkv.pkv_quant_load_blocks
    refused(f, ValueError, "dst_blocks: shape", load, dst_blocks=torch.zeros(3, **i32))
    refused(f, ValueError, "v_cache: shape", load, v_cache=cache[:4])
    refused(f, ValueError, "k_cache: dtype", load, k_cache=cache.half())
    qd = torch.zeros(2, hq, d, **bf16)
    dec = dict(bases, q=qd, block_tables=torch.zeros(2, mbps, **i32), context_lens=torch.zeros(2, **i32),
               max_context_len=32, sm_scale=1.0, out=torch.empty_like(qd))
    f = pkv.pkv_quant_decode
    refused(f, ValueError, "q: shape", dec, q=q)
    refused(f, ValueError, "lse: dtype", dec, lse=torch.zeros(2, hq, dtype=torch.float64, device=DEV))
    refused(f, ValueError, "sinks: shape", dec, sinks=torch.zeros(hkv, device=DEV))
    refused(f, ValueError, "does not fit", dec, max_context_len=1 << 40)
    refused(f, TypeError, "real number|float", dec, sm_scale="1")
    refused(f, TypeError, "integer", dec, window=1.5)
    f = pkv.pkv_rope_rotate
    for bad, error, text in ((dict(q=q.double()), ValueError, "q: dtype"), (dict(q=q[0]), ValueError, "q: expected"),
                             (dict(q=q.transpose(1, 2)), ValueError, "contiguous dims"),
                             (dict(k=x[:2]), ValueError, "k: 2 tokens"), (dict(k=x.half()), ValueError, "k: dtype"),
                             (dict(q_out=q[..., :32]), ValueError, "q_out: shape"),
                             (dict(k=x[..., :32]), ValueError, "head_dim")):
        with pytest.raises(error, match=text):
            f(**dict(dict(rope=rope, positions=ok["positions"], q=q), **bad))
    # calls without tokens or sequences do nothing
    none = torch.zeros(0, **i32)
    pkv.pkv_quant_append(desc=dd, **dict(app, token_to_seq=none, positions=none, k_new=x[:0], v_new=x[:0], q=q[:0]))
    pkv.pkv_quant_read(desc=dd, **dict(read, token_to_seq=none, positions=none, k_out=x[:0], v_out=None))
    pkv.pkv_quant_load_blocks(desc=dd, **dict(load, src_blocks=none, dst_blocks=none))
    pkv.pkv_quant_decode(desc=dd, **dict(dec, q=qd[:0], out=qd[:0], context_lens=none,
                                         block_tables=torch.zeros(0, mbps, **i32)))
    pkv.pkv_rope_rotate(rope, none, q[:0])
    assert pkv.pkv_device_errors() == 0


# ---------------------------------------------------------------- decode --

def run_decode(c, sm_scale=None, window=-1, chunk=0, sinks=None, max_len=None, ws=None, lens=None):
    dd = desc_of(c.fmt, c.hq, c.hkv, c.d, c.nb, c.mbps, c.ring)
    lens = c.lens if lens is None else lens
    max_len = max(1, int(lens.max())) if max_len is None else max_len
    sm_scale = c.d ** -0.5 if sm_scale is None else sm_scale
    if ws is None:
        need = pkv.pkv_quant_decode_workspace_size(dd, len(lens), max_len, window, chunk)
        ws = torch.zeros(max(256, need), dtype=torch.uint8, device=DEV)
    q = bf(c.q)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    pkv.pkv_quant_decode(dd, q, dev(c.pools[0]), dev(c.pools[1]), dev(c.tables), dev(lens), max_len,
                         sm_scale, out, lse, ws, window=window, chunk_blocks=chunk, k_scale=dev(c.k_scale),
                         v_scale=dev(c.v_scale), sinks=dev(sinks))
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def check_decode(c, got, window=-1, sinks=None, sm_scale=None, seqs=None):
    o, lse = got
    sm_scale = c.d ** -0.5 if sm_scale is None else sm_scale
    for s in range(len(c.lens)) if seqs is None else seqs:
        n = int(c.lens[s])
        lo = max(0, n - window) if window > 0 else 0
        ro, rl, tol, ltol = Q.attention(c.q[s].astype(np.float64), c.rows(0, s, lo, n), c.rows(1, s, lo, n),
                                        np.float64(np.float32(sm_scale)), sinks)
        assert np.all(np.isfinite(o[s])), s
        err = np.abs(o[s] - ro)  # an empty row's bound is 0: it is exactly 0
        assert np.all(err <= tol), "sequence %d (length %d): %.3g of the bound" % (s, n, (err / (tol + 1e-300)).max())
        fin = np.isfinite(rl)
        assert np.array_equal(fin, np.isfinite(lse[s]))
        assert np.all(np.abs(lse[s][fin] - rl[fin]) <= ltol[fin]), s


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (7, 1), (16, 2), (9, 1), (16, 1), (24, 8), (30, 2)])
def test_decode_lengths_and_groups(fmt, d, hq, hkv):
    rng = np.random.default_rng(hq * 131 + d)
    c = Q.QuantCase(rng, fmt, [1, 0, 16, 17, 31, 100, 255, 33, 640], hq, hkv, d)
    check_decode(c, run_decode(c))
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (16, 1, 128), (4, 4, 128)])
@pytest.mark.parametrize("chunk", [1, 2, 3, 5, 8, 40])
def test_decode_splits(fmt, hq, hkv, d, chunk):
    """1 .. 64 chunks a sequence, a last chunk of one key, empty sequences beside
    long ones; the same workspace for every call, whatever the last one left in it."""
    rng = np.random.default_rng(chunk)
    c = Q.QuantCase(rng, fmt, [1009, 0, 16 * chunk, 16 * chunk + 1, 5, 320], hq, hkv, d)
    dd = desc_of(fmt, hq, hkv, d, c.nb, c.mbps)
    ws = torch.zeros(max(256, pkv.pkv_quant_decode_workspace_size(dd, 6, 1009, -1, chunk)), dtype=torch.uint8,
                     device=DEV)
    first = run_decode(c, chunk=chunk, ws=ws)
    check_decode(c, first)
    again = run_decode(c, chunk=chunk, ws=ws)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
@pytest.mark.parametrize("chunk", [0, 2])
def test_decode_windows_and_sinks(fmt, window, chunk):
    rng = np.random.default_rng(window)
    hq, hkv, d = 12, 3, 64
    c = Q.QuantCase(rng, fmt, [1, 15, 16, 17, 64, 301, 0, 700], hq, hkv, d)
    sinks = rng.standard_normal(hq).astype(np.float32)
    sinks[0], sinks[1], sinks[2] = 30.0, -30.0, -np.inf
    check_decode(c, run_decode(c, window=window, chunk=chunk), window)
    o, lse = run_decode(c, window=window, chunk=chunk, sinks=sinks)
    check_decode(c, (o, lse), window, sinks)
    assert np.all(o[6] == 0) and np.array_equal(lse[6], sinks.astype(np.float64))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_ring(fmt, d):
    rng = np.random.default_rng(9)
    for window, ring in ((128, 9), (16, 2), (33, 4), (600, 40)):
        c = Q.QuantCase(rng, fmt, [1, window, window + 1, 977, 16 * ring * 3], 8, 2, d, ring=ring)
        check_decode(c, run_decode(c, window=window), window)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("value,qvalue", [(1e-3, 1.0), (30.0, 1.0), (1.0, 1e-6), (1.0, 3e5), (1.0, 40.0)])
def test_decode_magnitudes(fmt, value, qvalue):
    """Small and large caches; q below f16's normal range and beyond its largest;
    logits that concentrate the softmax on one key."""
    rng = np.random.default_rng(4)
    c = Q.QuantCase(rng, fmt, [300, 17, 900], 8, 2, 128, value=value)
    c.q = Q.bf16(c.q * qvalue)
    sm = 128 ** -0.5 / (1.0 if qvalue < 100 else qvalue)
    check_decode(c, run_decode(c, sm_scale=sm), sm_scale=sm)


def test_decode_rows_of_very_different_scales():
    """int8 rows whose scales span 2^-8 .. 2^8, largest first, last and in between."""
    rng = np.random.default_rng(8)
    for order in (1, -1, 0):
        c = Q.QuantCase(rng, "int8", [320], 4, 2, 64)
        at = 16 * 64
        for which in (0, 1):
            sc = np.ascontiguousarray(c.pools[which][..., at:]).view(np.float32)
            t = np.arange(320)
            f = 2.0 ** (8 - 16 * t / 319) if order == 1 else 2.0 ** (-8 + 16 * t / 319) if order == -1 else \
                2.0 ** rng.integers(-8, 9, 320)
            if which == 0:
                f = np.sqrt(np.sqrt(f))
            for i in range(320):
                sc[c.tables[0, i // 16], :, i % 16] *= f[i]
            c.pools[which][..., at:] = sc.view(np.uint8).reshape(c.pools[which][..., at:].shape)
        check_decode(c, run_decode(c, sm_scale=0.01), sm_scale=0.01)


def test_decode_bad_blocks_and_lengths_are_flagged():
    rng = np.random.default_rng(2)
    c = Q.QuantCase(rng, "fp4", [100, 50], 8, 2, 64, poison=False)
    c.tables[0, 3] = c.nb
    run_decode(c)
    assert pkv.pkv_device_errors() == pkv.DEVERR_BLOCK_ID
    c.tables[0, 3] = -5
    run_decode(c, chunk=2)
    assert pkv.pkv_device_errors() == pkv.DEVERR_BLOCK_ID
    c.tables[0, 3] = 0
    o, lse = run_decode(c, max_len=64)  # sequence 0 is cut at the bound, sequence 1 is whole
    assert pkv.pkv_device_errors() == pkv.DEVERR_LENGTH
    check_decode(c, (o, lse), seqs=[1])
    full = c.lens.copy()
    c.lens = np.array([64, 50], np.int32)
    check_decode(c, (o, lse))
    c.lens = full


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 64), (7, 1, 128), (12, 1, 128), (5, 1, 64), (18, 2, 64)])
def test_decode_many_sequences_merge_in_wide_ctas(fmt, hq, hkv, d):
    """More rows than the narrow merge takes (152 * 16): several heads a CTA, groups that
    fill no whole number of CTAs, empty and one-chunk sequences in between."""
    rng = np.random.default_rng(hq + d)
    n = 2432 // hq + 9
    lens = rng.integers(0, 60, n)
    c = Q.QuantCase(rng, fmt, lens, hq, hkv, d)
    check_decode(c, run_decode(c, chunk=1), seqs=range(0, n, 3))
    sinks = rng.standard_normal(hq).astype(np.float32)
    check_decode(c, run_decode(c, chunk=1, window=20, sinks=sinks), 20, sinks, seqs=range(1, n, 5))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (9, 1, 64)])
def test_decode_most_chunks(fmt, hq, hkv, d):
    """256 chunks are the most; a bound that needs one more is refused."""
    rng = np.random.default_rng(3)
    c = Q.QuantCase(rng, fmt, [4096, 4081, 17], hq, hkv, d)
    check_decode(c, run_decode(c, chunk=1))
    c = Q.QuantCase(rng, fmt, [4097], hq, hkv, d)
    with pytest.raises(pkv.PkvError, match="chunks"):
        run_decode(c, chunk=1)
    check_decode(c, run_decode(c, chunk=2))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("chunk", [0, 1])
def test_decode_most_sequences(fmt, chunk):
    """65535 sequences share the blocks of a few; their neighbours' lengths differ, some are
    empty or below zero (taken as empty)."""
    rng = np.random.default_rng(1)
    hq, hkv, d, n = 3, 1, 64, 65535
    c = Q.QuantCase(rng, fmt, [32, 32, 27, 16, 1, 0], hq, hkv, d, poison=False)
    pick = rng.integers(0, 6, n)
    q = rng.standard_normal((64, hq, d))
    c.q = Q.bf16(q)[rng.integers(0, 64, n)]
    c.tables, c.lens = c.tables[pick], c.lens[pick]
    c.lens[7], c.lens[n - 1] = -1, -2 ** 31
    got = run_decode(c, chunk=chunk, max_len=32)
    for s in (7, n - 1):
        assert not np.any(got[0][s]) and np.all(np.isneginf(got[1][s]))
    check_decode(c, got, seqs=[s for s in list(range(0, n, 1009)) + [1, 2, 3, n - 2] if c.lens[s] >= 0])
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (11, 1)])
def test_decode_a_query_head_that_is_not_finite_spoils_no_other(fmt, bad, hq, hkv):
    """The group's heads share q's power of two: an infinity must not set it (the others,
    beyond f16's range here, would overflow)."""
    rng = np.random.default_rng(5)
    c = Q.QuantCase(rng, fmt, [300, 40], hq, hkv, 64)
    c.q = Q.bf16(c.q * 3e5)
    whole = c.q.copy()
    c.q[0, 1, 7] = bad
    o, lse = run_decode(c, sm_scale=1e-6)
    assert not np.any(np.isfinite(o[0, 1]))
    c.q = whole
    o2, lse2 = run_decode(c, sm_scale=1e-6)
    o[0, 1], lse[0, 1] = o2[0, 1], lse2[0, 1]
    check_decode(c, (o, lse), sm_scale=1e-6)


def test_decode_two_streams_two_workspaces_and_graphs():
    rng = np.random.default_rng(6)
    cases = [Q.QuantCase(rng, fmt, [900, 33, 500, 1], 16, 2, 128) for fmt in ("int8", "fp4")]
    runs = []
    for c in cases:
        dd = desc_of(c.fmt, c.hq, c.hkv, c.d, c.nb, c.mbps)
        t = dict(desc=dd, q=bf(c.q), k_pool=dev(c.pools[0]), v_pool=dev(c.pools[1]), block_tables=dev(c.tables),
                 context_lens=dev(c.lens), max_context_len=900, sm_scale=c.d ** -0.5,
                 out=torch.zeros(4, 16, 128, dtype=torch.bfloat16, device=DEV),
                 lse=torch.zeros(4, 16, device=DEV), chunk_blocks=4,
                 workspace=torch.zeros(max(256, pkv.pkv_quant_decode_workspace_size(dd, 4, 900, -1, 4)),
                                       dtype=torch.uint8, device=DEV),
                 k_scale=dev(c.k_scale), v_scale=dev(c.v_scale))
        runs.append(t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(20):
        for t, s in zip(runs, streams):
            pkv.pkv_quant_decode(stream=s, **t)
    torch.cuda.synchronize()
    for c, t in zip(cases, runs):
        check_decode(c, (t["out"].double().cpu().numpy(), t["lse"].double().cpu().numpy()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for t in runs:
            pkv.pkv_quant_decode(**t)
    for c, t in zip(cases, runs):  # other queries and lengths in the same buffers
        c.q = Q.bf16(rng.standard_normal(c.q.shape))
        c.lens = np.array([17, 33, 499, 1], np.int32)
        t["q"].copy_(bf(c.q))
        t["context_lens"].copy_(dev(c.lens))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for c, t in zip(cases, runs):
        check_decode(c, (t["out"].double().cpu().numpy(), t["lse"].double().cpu().numpy()))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_pool_offsets_past_32_bits(fmt):
    """The last blocks of a pool of more than 2^32 bytes: append, read, widen, decode."""
    hq, hkv, d = 8, 8, 128
    rec = Q.record_bytes(fmt, d)
    nb = (1 << 32) // (hkv * rec) + 40
    pools = [torch.empty(nb, hkv, rec, dtype=torch.uint8, device=DEV) for _ in range(2)]
    n = 70
    tables = torch.arange(nb - 5, nb, dtype=torch.int32, device=DEV)[None]
    dd = desc_of(fmt, hq, hkv, d, nb, 5)
    g = torch.full((hkv,), 4.0 / 2688, device=DEV) if fmt == "fp4" else None
    k, v = (torch.randn(n, hkv, d, device=DEV).bfloat16() for _ in range(2))
    tts, pos = torch.zeros(n, dtype=torch.int32, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    pkv.pkv_quant_append(dd, pools[0], pools[1], tables, tts, pos, k, v, k_scale=g, v_scale=g)
    ko, vo = (torch.empty(n, hkv, d, device=DEV) for _ in range(2))
    pkv.pkv_quant_read(dd, pools[0], pools[1], tables, tts, pos, ko, vo, k_scale=g, v_scale=g)
    kb, vb = (torch.zeros(5, hkv, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pkv.pkv_quant_load_blocks(dd, pools[0], pools[1], tables[0], torch.arange(5, dtype=torch.int32, device=DEV),
                              kb, vb, k_scale=g, v_scale=g)
    assert torch.equal(kb.transpose(1, 2).reshape(80, hkv, d)[:n], ko.bfloat16())
    assert torch.equal(vb.transpose(1, 2).reshape(80, hkv, d)[:n], vo.bfloat16())
    q = torch.randn(1, hq, d, device=DEV).bfloat16()
    out = torch.empty_like(q)
    ws = torch.zeros(max(256, pkv.pkv_quant_decode_workspace_size(dd, 1, n)), dtype=torch.uint8, device=DEV)
    pkv.pkv_quant_decode(dd, q, pools[0], pools[1], tables, torch.tensor([n], dtype=torch.int32, device=DEV), n,
                         d ** -0.5, out, None, ws, k_scale=g, v_scale=g)
    ro, _, tol, _ = Q.attention(q[0].double().cpu().numpy(), ko.double().cpu().numpy(), vo.double().cpu().numpy(),
                                np.float64(np.float32(d ** -0.5)))
    # the rows read back were rounded to fp32: 2^-24 more on each product
    assert np.all(np.abs(out[0].double().cpu().numpy() - ro) <= tol * 1.001)
    assert pkv.pkv_device_errors() == 0
    # and the values are the rows' own, within half a step.  int8: amax / 254.  4-bit,
    # t the 16 dims' scale: half a step is at most t, t <= amax / 6 (1 + 2^-4) with
    # e4m3's rounding, a scale rounded down clips at most amax 2^-4, and one beyond
    # 448 g = 4 / 6 clips amax - 4
    for x, src in ((ko, k), (vo, v)):
        amax = float(src.float().abs().max())
        bound = amax / 254 if fmt == "int8" else max(amax / 6 * (1 + 2.0 ** -4), amax - 4.0)
        assert float((x - src.float()).abs().max()) <= bound * 1.0001


# ------------------------------------------------- a sequence, end to end --

@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("layout,r", [("half", 128), ("interleaved", 64)])
def test_a_batch_served_through_the_quantised_cache(fmt, layout, r):
    """A prompt in two chunks (append, widen, ragged prefill), then four decode
    steps (append with the rotation of q, decode), against 64-bit attention over
    the definition's rows; YaRN positions, q and k in one packed buffer."""
    rng = np.random.default_rng(77)
    hq, hkv, d, steps = 8, 2, 128, 4
    prompts = [53, 7, 96]
    b = len(prompts)
    total = [p + steps for p in prompts]
    mbps = max((t + 15) // 16 for t in total)
    nb = sum((t + 15) // 16 for t in total) + 2
    perm = list(rng.permutation(nb))
    tables = np.full((b, mbps), -1, np.int32)
    for s, t in enumerate(total):
        for i in range((t + 15) // 16):
            tables[s, i] = perm.pop()
    cs = pkv.pkv_rope_scaled_table(1e4, r, 200, kind="yarn", factor=4.0, original_max_pos=50, attention=1.1386)
    rope = pkv.make_rope(dev(cs), layout=layout)
    dd = desc_of(fmt, hq, hkv, d, nb, mbps)
    g = np.full(hkv, 5.0 / 2688, np.float32) if fmt == "fp4" else None
    gd = dev(g)
    pools = [torch.zeros(nb, hkv, Q.record_bytes(fmt, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    qkv = [Q.bf16(rng.standard_normal((t, hq + 2 * hkv, d))) for t in total]
    sm = np.float64(np.float32(d ** -0.5))

    # the definition's rows of every sequence
    def stored(x, rotated):
        rows = np.empty((len(x), hkv, d))
        for p in range(len(x)):
            y = Q.rotate(x[p], cs[p], layout, np.float32) if rotated else x[p]
            for h in range(hkv):
                gh = 1.0 if g is None else g[h]
                rows[p, h] = Q.row_values(fmt, *Q.quantise(fmt, y[h], gh), gh)
        return rows
    keys = [stored(x[:, hq:hq + hkv], True) for x in qkv]
    vals = [stored(x[:, hq + hkv:], False) for x in qkv]
    turned = [Q.bf16(np.stack([Q.rotate(x[p, :hq], cs[p], layout, np.float32) for p in range(len(x))])) for x in qkv]

    # prompt chunks
    cuts = [(0, [20, 5, 48]), ([20, 5, 48], prompts)]
    staged = [torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    bdesc = pkv.make_desc(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, num_blocks=nb, max_blocks_per_seq=mbps)
    for lo, hi in cuts:
        lo = [0] * b if lo == 0 else lo
        rows = bf(np.concatenate([x[a:e] for x, a, e in zip(qkv, lo, hi)]))
        tts = np.repeat(np.arange(b), [e - a for a, e in zip(lo, hi)]).astype(np.int32)
        pos = np.concatenate([np.arange(a, e) for a, e in zip(lo, hi)]).astype(np.int32)
        q = torch.empty(len(pos), hq, d, dtype=torch.bfloat16, device=DEV)
        pkv.pkv_quant_append(dd, pools[0], pools[1], dev(tables), dev(tts), dev(pos), rows[:, hq:hq + hkv],
                             rows[:, hq + hkv:], q=rows[:, :hq], q_out=q, rope=rope, k_scale=gd, v_scale=gd)
        ids = np.unique(np.concatenate([tables[s, :(e + 15) // 16] for s, e in enumerate(hi)])).astype(np.int32)
        pkv.pkv_quant_load_blocks(dd, pools[0], pools[1], dev(ids), dev(ids), staged[0], staged[1], k_scale=gd,
                                  v_scale=gd)
        qo = np.concatenate(([0], np.cumsum([e - a for a, e in zip(lo, hi)]))).astype(np.int32)
        lens = np.array(hi, np.int32)
        out = torch.empty_like(q)
        pkv.pkv_prefill_attention_ragged(bdesc, q, dev(qo), staged[0], staged[1], dev(tables), dev(lens), float(sm),
                                         out, qo_indptr_host=qo, kv_lens_host=lens)
        got = out.double().cpu().numpy()
        for i, (s, p) in enumerate(zip(tts, pos)):
            # the widened rows are the values rounded to bf16, which is what the prefill attends
            ro, _, tol, _ = Q.attention(turned[s][p].astype(np.float64), Q.bf16(keys[s][:p + 1]).astype(np.float64),
                                        Q.bf16(vals[s][:p + 1]).astype(np.float64), sm)
            # and its weights are bf16: 2^-8 of sum w |v| <= max |v| in the bound's place of f16's 2^-11
            tol = tol + 2.0 ** -8 * np.abs(vals[s][:p + 1]).max()
            assert np.all(np.abs(got[i] - ro) <= tol), (i, s, p)

    # decode steps
    ws = torch.zeros(max(256, pkv.pkv_quant_decode_workspace_size(dd, b, max(total), -1, 2)), dtype=torch.uint8,
                     device=DEV)
    tts = dev(np.arange(b, dtype=np.int32))
    for step in range(steps):
        pos = np.array(prompts, np.int32) + step
        rows = bf(np.stack([x[p] for x, p in zip(qkv, pos)]))
        q = torch.empty(b, hq, d, dtype=torch.bfloat16, device=DEV)
        pkv.pkv_quant_append(dd, pools[0], pools[1], dev(tables), tts, dev(pos), rows[:, hq:hq + hkv],
                             rows[:, hq + hkv:], q=rows[:, :hq], q_out=q, rope=rope, k_scale=gd, v_scale=gd)
        out = torch.empty_like(q)
        lse = torch.empty(b, hq, device=DEV)
        pkv.pkv_quant_decode(dd, q, pools[0], pools[1], dev(tables), dev(pos + 1), max(total), float(sm), out, lse,
                             ws, chunk_blocks=2, k_scale=gd, v_scale=gd)
        for s, p in enumerate(pos):
            assert np.array_equal(q[s].float().cpu().numpy(), turned[s][p])
            ro, rl, tol, ltol = Q.attention(turned[s][p].astype(np.float64), keys[s][:p + 1], vals[s][:p + 1], sm)
            assert np.all(np.abs(out[s].double().cpu().numpy() - ro) <= tol)
            assert np.all(np.abs(lse[s].double().cpu().numpy() - rl) <= ltol)
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_captured_serving_steps_are_the_eager_ones(fmt):
    """Append (q in place) then decode, the launches overlapping as they do in a stream:
    40 steps without a synchronisation, and the same steps as replays of one graph whose
    positions and lengths move on the device, give the same bits as one step at a time."""
    hq, hkv, d, b, steps = 16, 2, 128, 5, 40
    start = torch.tensor([0, 15, 250, 31, 700], dtype=torch.int32, device=DEV)
    mbps = (700 + steps) // 16 + 1
    nb = b * mbps
    gen = torch.Generator().manual_seed(2)
    tables = torch.randperm(nb, generator=gen).int().view(b, mbps).to(DEV)
    dd = desc_of(fmt, hq, hkv, d, nb, mbps)
    g = torch.full((hkv,), 4 / 2688, device=DEV) if fmt == "fp4" else None
    rope = pkv.make_rope(dev(pkv.pkv_rope_scaled_table(1e4, d, 800)))
    tts = torch.arange(b, dtype=torch.int32, device=DEV)
    rows = torch.randn(steps, b, hq + 2 * hkv, d, generator=gen).bfloat16().to(DEV)
    old = torch.randn(700, hkv, d, generator=gen).bfloat16().to(DEV)
    ws = torch.zeros(max(256, pkv.pkv_quant_decode_workspace_size(dd, b, 740, -1, 4)), dtype=torch.uint8, device=DEV)

    def fresh():
        pools = [torch.zeros(nb, hkv, Q.record_bytes(fmt, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
        for s, n in enumerate(start.tolist()):
            at = torch.arange(n, dtype=torch.int32, device=DEV)
            pkv.pkv_quant_append(dd, pools[0], pools[1], tables, torch.full_like(at, s), at, old[:n], old[:n],
                                 k_scale=g, v_scale=g)
        return pools

    def step(pools, buf, pos, lens, out):
        pkv.pkv_quant_append(dd, pools[0], pools[1], tables, tts, pos, buf[:, hq:hq + hkv], buf[:, hq + hkv:],
                             q=buf[:, :hq], q_out=out, rope=rope, k_scale=g, v_scale=g)
        pkv.pkv_quant_decode(dd, out, pools[0], pools[1], tables, lens, 740, d ** -0.5, out, None, ws,
                             chunk_blocks=4, k_scale=g, v_scale=g)

    results = []
    for wait in (True, False):
        pools = fresh()
        pos = [start + i for i in range(steps)]
        lens = [p + 1 for p in pos]
        outs = torch.zeros(steps, b, hq, d, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        for i in range(steps):
            step(pools, rows[i], pos[i], lens[i], outs[i])
            if wait:
                torch.cuda.synchronize()
        results.append(pools + [outs])
    pools, outs = fresh(), torch.zeros(steps, b, hq, d, dtype=torch.bfloat16, device=DEV)
    buf, pos, lens = rows[0].clone(), start.clone(), start + 1
    out = torch.zeros(b, hq, d, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pools, buf, pos, lens, out)
        pos += 1
        lens += 1
    for i in range(steps):
        buf.copy_(rows[i])
        graph.replay()
        outs[i].copy_(out)
    torch.cuda.synchronize()
    results.append(pools + [outs])
    assert pkv.pkv_device_errors() == 0
    for other in results[1:]:
        for a, c in zip(results[0], other):
            assert torch.equal(a, c)
