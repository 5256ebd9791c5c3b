"""Prefill over a context that ends at the end of 32 bits, on the GPU."""
import numpy as np
import pytest
import torch

from _far import Far, queries
from test_gpu_score import check_prefill, prefill
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("end", [MOST // 16 * 16, MOST // 16 * 16 - 5, MOST - 127, MOST - 128])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("e4m3", 64)])
def test_the_last_keys(kv, d, end):
    """The same bits as over the same keys at the beginning; slots behind the last key hold NaN."""
    f = Far(end, 8, 2, d, kv, seed=43)
    p = f.small
    for m in (4, 90):
        qo, qo_t, q, q64 = queries(p, m)
        for rule in (dict(), dict(cap=3.0), dict(cap=9.0), dict(slopes=0.1), dict(cap=9.0, slopes=0.1, sinks=True)):
            for window in (150, 30):
                r = f.rule(window=window, **rule)
                want = prefill(p, r, q, qo, qo_t)
                check_prefill(p, r, q64, qo, *want)
                out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
                args = (f.desc, r.score, q, qo_t, p.k_pool, p.v_pool, f.table, f.len, out, lse)
                hosts = dict(qo_indptr_host=qo, kv_lens_host=[end])
                pkv.pkv_score_prefill(*args, **hosts, **p.scales)
                assert pkv.pkv_device_errors() == 0
                if m > 16:  # (a few queries: chunks of keys begin elsewhere)
                    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
                check_prefill(p, r, q64, qo, out, lse)
                if not rule:
                    out.zero_()
                    pkv.pkv_prefill_attention_ragged(f.desc, q, qo_t, p.k_pool, p.v_pool, f.table, f.len, r.scale, out, lse,
                                                     window=window, qo_indptr_host=qo,
                                                     kv_lens_host=np.array([end], np.int32), **p.scales)
                    check_prefill(p, r, q64, qo, out, lse)
