"""Quantised decode over long contexts and long chunks, against 64 bits within a bound that
a wrong block exceeds (test_quant_bound.py)."""
import numpy as np
import pytest
import torch

import _quant as Q
import _quant_bound as B
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def decode(p, q, tables, lens, window=-1, chunk=0, ring=0, max_len=None, sinks=None, sm_scale=None):
    """out, lse as fp64 arrays; the planned call where chunk is 0."""
    b, hq, d = q.shape
    dd = pkv.make_desc(num_q_heads=hq, num_kv_heads=p.hkv, head_dim=d, num_blocks=p.nb,
                       max_blocks_per_seq=tables.shape[1], kv_dtype=p.fmt, ring_blocks=ring)
    max_len = int(max(lens)) if max_len is None else max_len
    need = pkv.pkv_quant_decode_workspace_size(dd, b, max_len, window, chunk)
    ws = torch.zeros(max(256, need), dtype=torch.uint8, device=DEV)
    qd = torch.from_numpy(q).bfloat16().to(DEV)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    pkv.pkv_quant_decode(dd, qd, dev(p.raw[0]), dev(p.raw[1]), dev(tables), dev(np.asarray(lens, np.int32)), max_len,
                         d ** -0.5 if sm_scale is None else sm_scale, out, lse, ws, window=window, chunk_blocks=chunk,
                         k_scale=dev(p.scales[0]), v_scale=dev(p.scales[1]), sinks=dev(sinks))
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def within(got, ref, tol, what):
    err = np.abs(got - ref)
    assert np.all(err <= tol), "%s: %.3g of the bound" % (what, (err / tol).max())


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("b,hkv,group,d,ctx", [(4, 8, 2, 64, 70000), (3, 8, 2, 128, 70000), (15, 1, 12, 128, 131072),
                                               (1, 1, 4, 64, 600000), (2, 2, 3, 128, 600000)])
def test_planned_decode_of_long_contexts(fmt, b, hkv, group, d, ctx):
    """Contexts past 65536 and 524288 tokens with default arguments.  Tables repeat a few
    blocks, so that the pool stays small: a row counts as often as it stands in the context."""
    rng = np.random.default_rng(ctx + b)
    p = B.Pools(rng, fmt, 40, hkv, d)
    tables = rng.integers(0, p.nb, (b, (ctx + 15) // 16)).astype(np.int32)
    lens = [int(x) for x in rng.integers(ctx // 2, ctx, b)]
    lens[0] = ctx - 7
    q = Q.bf16(rng.standard_normal((b, hkv * group, d)))
    o, lse = decode(p, q, tables, lens, max_len=ctx)
    every = np.arange(p.nb)
    for s in range(b) if b < 5 else (0, 7, b - 1):
        n = lens[s]
        copies = np.zeros((p.nb, 16))
        np.add.at(copies, tables[s, :n // 16], 1)
        copies[tables[s, n // 16], :n % 16] += 1
        ro, rl, tol, ltol = B.attention(fmt, q[s].astype(np.float64), p.rows(0, every, 0, 16 * p.nb),
                                        p.rows(1, every, 0, 16 * p.nb), np.float64(np.float32(d ** -0.5)), 512,
                                        p.units(every, 0, 16 * p.nb), copies.reshape(-1))
        within(o[s], ro, tol, "o of sequence %d" % s)
        within(lse[s], rl, ltol, "lse of sequence %d" % s)
    assert pkv.pkv_device_errors() == 0


def check(p, q, tables, lens, got, chunk, window=-1, ring=0, sinks=None):
    d = q.shape[2]
    for s, n in enumerate(lens):
        lo = max(0, n - window) if window > 0 else 0
        t = np.arange((n + 15) // 16)
        line = tables[s][t % ring] if ring else tables[s]
        ro, rl, tol, ltol = B.attention(p.fmt, q[s].astype(np.float64), p.rows(0, line, lo, n), p.rows(1, line, lo, n),
                                        np.float64(np.float32(d ** -0.5)), chunk, p.units(line, lo, n), sinks=sinks)
        within(got[0][s], ro, tol, "o of sequence %d" % s)
        within(got[1][s], rl, ltol, "lse of sequence %d" % s)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 4, 1), (64, 13, 1), (128, 32, 2)])
@pytest.mark.parametrize("chunk", [129, 200, 256, 512])
def test_chunks_of_more_blocks_than_a_warp_holds_ids(fmt, d, hq, hkv, chunk):
    """A warp holds 32 block ids at a time, a chunk's 128: contexts that end on either side of
    the second and later ones, tables scattered."""
    rng = np.random.default_rng(chunk + d)
    lens = [16 * 128, 16 * 128 + 1, 16 * 129 + 5, 16 * chunk - 3, 16 * chunk + 17, 9000, 100]
    n = [(x + 15) // 16 for x in lens]
    p = B.Pools(rng, fmt, sum(n) + 3, hkv, d)
    perm, tables, at = rng.permutation(p.nb).astype(np.int32), np.full((len(lens), max(n)), -1, np.int32), 0
    for s, k in enumerate(n):
        tables[s, :k] = perm[at:at + k]
        at += k
    q = Q.bf16(rng.standard_normal((len(lens), hq, d)))
    sinks = rng.standard_normal(hq).astype(np.float32)
    check(p, q, tables, lens, decode(p, q, tables, lens, chunk=chunk, sinks=sinks), chunk, sinks=sinks)
    window = 16 * 140 + 3  # a window's first block starts a chunk anywhere in the table
    check(p, q, tables, lens, decode(p, q, tables, lens, chunk=chunk, window=window), chunk, window)
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("chunk", [200, 512])
def test_a_ring_that_wraps_within_a_chunk(fmt, d, chunk):
    """Windows of 251 blocks over a ring of 252, at turns that put the ring's end into the first
    ids of a warp, into the second, and between."""
    rng = np.random.default_rng(d)
    window, ring = 16 * 250 - 15, 252
    lens = [4000, 4100, 16 * 252 + 900, 16 * 252 * 2 + 16 * 130, 16 * 252 * 3 - 1, 16 * 252 * 3 + 16 * 128 + 2]
    p = B.Pools(rng, fmt, ring * len(lens), 1, d)
    tables = rng.permutation(p.nb).astype(np.int32).reshape(len(lens), ring)
    q = Q.bf16(rng.standard_normal((len(lens), 5, d)))
    got = decode(p, q, tables, lens, chunk=chunk, window=window, ring=ring)
    check(p, q, tables, lens, got, chunk, window, ring)
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("at", [128, 131, 255, 256, 290])
def test_a_bad_block_id_among_a_warps_later_ones_is_flagged(fmt, at):
    """And one behind the end is not looked at."""
    rng = np.random.default_rng(at)
    p = B.Pools(rng, fmt, 300, 1, 64)
    tables = rng.permutation(300).astype(np.int32)[None]
    q = Q.bf16(rng.standard_normal((1, 3, 64)))
    for bad in (p.nb, -1, 2 ** 31 - 1, -2 ** 31):
        tables[0, at] = bad
        o, lse = decode(p, q, tables, [16 * (at + 1)], chunk=512, max_len=16 * 300)
        assert pkv.pkv_device_errors() == pkv.DEVERR_BLOCK_ID and np.all(np.isfinite(lse))
        got = decode(p, q, tables, [16 * at], chunk=512, max_len=16 * 300)
        assert pkv.pkv_device_errors() == 0
        check(p, q, tables, [16 * at], got, 512)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_the_longest_context_and_one_key_more(fmt):
    """256 chunks of 512 blocks, over a table of a few blocks again and again."""
    rng = np.random.default_rng(21)
    p = B.Pools(rng, fmt, 40, 1, 64)
    n = 256 * 512 * 16
    tables = rng.integers(0, p.nb, (1, n // 16 + 1)).astype(np.int32)
    q = Q.bf16(rng.standard_normal((1, 2, 64)))
    got = decode(p, q, tables, [n], max_len=n)
    every = np.arange(p.nb)
    copies = np.repeat(np.bincount(tables[0, :n // 16], minlength=p.nb), 16)
    ro, rl, tol, ltol = B.attention(fmt, q[0].astype(np.float64), p.rows(0, every, 0, 16 * p.nb),
                                    p.rows(1, every, 0, 16 * p.nb), np.float64(np.float32(0.125)), 512,
                                    p.units(every, 0, 16 * p.nb), copies)
    within(got[0][0], ro, tol, "o")
    within(got[1][0], rl, ltol, "lse")
    with pytest.raises(pkv.PkvError, match="256 chunks of 512 blocks"):
        decode(p, q, tables, [n], max_len=n + 1)
    assert pkv.pkv_device_errors() == 0
