"""Windows at the end of 32 bits on the GPU: a window that no context fills is none."""
import numpy as np
import pytest
import torch

import _quant as Q
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
MOST = 2 ** 31 - 1
LENS = [1, 700, 16, 333]


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def pools_of(kv_dtype, nb, hkv, d):
    gen = torch.Generator(device=DEV).manual_seed(nb)
    p = [torch.randn(nb, hkv, 16, d, generator=gen, device=DEV) for _ in range(2)]
    if kv_dtype == pkv.KV_FP8_E4M3:
        return [x.to(torch.float8_e4m3fn).view(torch.uint8) for x in p]
    return [x.bfloat16() for x in p]


@pytest.mark.parametrize("kv_dtype", [pkv.KV_BF16, pkv.KV_FP8_E4M3])
def test_decode_and_prefill_with_a_window_near_32_bits(kv_dtype):
    hq, hkv, d, b = 8, 2, 128 if kv_dtype == pkv.KV_BF16 else 64, len(LENS)
    mbps = (max(LENS) + 15) // 16
    nb = b * mbps
    kc, vc = pools_of(kv_dtype, nb, hkv, d)
    scale = torch.ones(hkv, device=DEV) if kv_dtype == pkv.KV_FP8_E4M3 else None
    tables = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).int().view(b, mbps).to(DEV)
    dd = pkv.make_desc(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, num_blocks=nb, max_blocks_per_seq=mbps,
                       kv_dtype=kv_dtype)
    lens = torch.tensor(LENS, dtype=torch.int32, device=DEV)
    for n in (1, 5, 40):  # decode; the short-query and the tile kernels over the last n tokens
        own = [min(n, x) for x in LENS]
        qo = np.concatenate(([0], np.cumsum(own))).astype(np.int32)
        q = torch.randn(int(qo[-1]), hq, d, device=DEV).bfloat16()
        outs = []
        for window in (-1, MOST, MOST - 14):
            out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
            if n == 1:
                ws = torch.zeros(max(256, pkv.pkv_decode_workspace_size(dd, b, 700, window, 0)), dtype=torch.uint8,
                                 device=DEV)
                pkv.pkv_decode_attention(dd, q, kc, vc, tables, lens, 700, d ** -0.5, out, lse, ws, window=window,
                                         k_scale=scale, v_scale=scale)
            else:
                pkv.pkv_prefill_attention_ragged(dd, q, dev(qo), kc, vc, tables, lens, d ** -0.5, out, lse,
                                                 window=window, k_scale=scale, v_scale=scale, qo_indptr_host=qo,
                                                 kv_lens_host=np.array(LENS, np.int32))
            outs.append((out, lse))
        for out, lse in outs[1:]:
            assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1]), n
        assert not torch.any(outs[0][1] == 7)
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hkv,chunk", [(1, 0), (2, 3), (8, 0), (160, 0)])
def test_quantised_decode_with_a_window_near_32_bits(fmt, hkv, chunk):
    """One chunk, clusters and the second launch; so many pairs that no cluster is planned."""
    rng = np.random.default_rng(hkv)
    c = Q.QuantCase(rng, fmt, LENS + [0], 4 * hkv if hkv < 100 else hkv, hkv, 64)
    dd = pkv.make_desc(num_q_heads=c.hq, num_kv_heads=hkv, head_dim=64, num_blocks=c.nb, max_blocks_per_seq=c.mbps,
                       kv_dtype=fmt)
    pools, q = [dev(p) for p in c.pools], torch.from_numpy(c.q).bfloat16().to(DEV)
    outs = []
    for window in (-1, MOST, MOST - 13):
        ws = torch.zeros(max(256, pkv.pkv_quant_decode_workspace_size(dd, 5, 700, window, chunk)), dtype=torch.uint8,
                         device=DEV)
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
        pkv.pkv_quant_decode(dd, q, pools[0], pools[1], dev(c.tables), dev(c.lens), 700, 0.125, out, lse, ws,
                             window=window, chunk_blocks=chunk, k_scale=dev(c.k_scale), v_scale=dev(c.v_scale))
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    assert not torch.any(outs[0][1] == 7) and not torch.any(outs[0][0][4])
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("hq,d", [(4, 64), (12, 64), (4, 128)])
def test_quantised_ring_decode_at_the_longest_contexts(fmt, hq, d):
    """A ring's contexts that end at the last positions of 32 bits: the same keys under a
    window as contexts that lie whole turns of the ring earlier, hence the same bits."""
    rng = np.random.default_rng(hq)
    ring = 16
    near = np.array([MOST, MOST - 1, MOST - 15, MOST - 16, MOST - 17, MOST - 300], np.int32)
    early = (near.astype(np.int64) % (16 * ring) + 16 * ring * 3).astype(np.int32)
    c = Q.QuantCase(rng, fmt, early, hq, 1, d, ring=ring, poison=False)
    for pool in c.pools:  # slots that no window reaches hold no numbers
        at = pool[..., 16 * Q.row_bytes(fmt, d):]
        at = at.view(np.float32) if fmt == "int8" else at.reshape(at.shape[:2] + (16, d // 16))
        for s, n in enumerate(early):
            for t in range(n - 16 * ring, n - 100):
                at[c.tables[s, t // 16 % ring], :, t % 16] = np.nan if fmt == "int8" else 0x7F
    dd = pkv.make_desc(num_q_heads=hq, num_kv_heads=1, head_dim=d, num_blocks=c.nb, max_blocks_per_seq=c.mbps,
                       kv_dtype=fmt, ring_blocks=ring)
    pools, q = [dev(p) for p in c.pools], torch.from_numpy(c.q).bfloat16().to(DEV)
    for chunk in (0, 1, 3):
        outs = []
        for lens in (early, near):
            ws = torch.zeros(max(256, pkv.pkv_quant_decode_workspace_size(dd, 6, MOST, 100, chunk)),
                             dtype=torch.uint8, device=DEV)
            out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
            pkv.pkv_quant_decode(dd, q, pools[0], pools[1], dev(c.tables), dev(lens), MOST, d ** -0.5, out, lse, ws,
                                 window=100, chunk_blocks=chunk, k_scale=dev(c.k_scale), v_scale=dev(c.v_scale))
            outs.append((out, lse))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        assert torch.all(torch.isfinite(outs[0][1])) and torch.all(torch.isfinite(outs[0][0]))
    assert pkv.pkv_device_errors() == 0
