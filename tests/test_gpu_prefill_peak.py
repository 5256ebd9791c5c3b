"""Prefill where one key's logit lies far above all others, in each column of a 128-key tile."""
import numpy as np
import pytest
import torch

import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("peak", [14.0, 100.0])
def test_a_single_peak_in_any_column(kv, d, peak):
    """128 queries behind 256 keys, one key of which has a logit of `peak` and the others of
    about 0: the output is that key's V, and lse the peak."""
    n, m, hq = 384, 128, 2
    rng = np.random.default_rng(3)
    v = torch.from_numpy(rng.standard_normal((n, 1, d)).astype(np.float32)).bfloat16()
    q = torch.zeros(m, hq, d).bfloat16()
    q[..., 0] = 8.0
    scale = torch.ones(1, device=DEV) if kv != "bf16" else None
    tables = torch.arange(n // 16, dtype=torch.int32, device=DEV)[None]
    desc = pkv.make_desc(num_q_heads=hq, num_kv_heads=1, head_dim=d, num_blocks=n // 16, max_blocks_per_seq=n // 16,
                         kv_dtype=kv)
    qo = torch.tensor([0, m], dtype=torch.int32, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    for column in list(range(0, 128, 9)) + list(range(116, 128)):
        for tile in (0, 1):
            k = torch.zeros(n, 1, d)
            k[128 * tile + column, 0, 0] = 1.0
            pools = [x.reshape(n // 16, 16, 1, d).transpose(1, 2).contiguous() for x in (k.bfloat16(), v)]
            if kv != "bf16":
                pools = [x.float().to(torch.float8_e4m3fn).view(torch.uint8) for x in pools]
            pools = [x.to(DEV) for x in pools]
            out, lse = torch.empty(m, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(m, hq, device=DEV)
            pkv.pkv_prefill_attention_ragged(desc, q.to(DEV), qo, pools[0], pools[1], tables, lens, peak / 8.0, out, lse,
                                             k_scale=scale, v_scale=scale)
            values = pools[1].view(torch.float8_e4m3fn) if kv != "bf16" else pools[1]
            values = values.double().cpu().transpose(1, 2).reshape(n, d).numpy()
            for i in (0, 1, 77, 127):
                seen = n - m + i + 1
                w = np.full(seen, np.exp(-peak))
                w[128 * tile + column] = 1.0
                want = w @ values[:seen] / w.sum()
                got = out[i].double().cpu().numpy()
                # weights and the output are each rounded to 16 bits once; f16 weights lose up to 2^-25 each
                bound = 2.0 ** -7 * (w @ np.abs(values[:seen])) / w.sum() + seen * 2.0 ** -17 * np.abs(values).max() * 2.0 ** -8
                assert (np.abs(got - want) <= bound).all(), (column, tile, i)
                assert (np.abs(lse[i].cpu().numpy() - (peak + np.log(w.sum()))) <= 2.0 ** -18 * peak).all(), (column, tile, i)
