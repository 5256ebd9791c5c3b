"""Weights of keys at the end of 32 bits, on the GPU."""
import numpy as np
import pytest
import torch

from _far import Far, queries
from _score import close
from test_gpu_score import prefill
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("end", [MOST, MOST - 15, MOST - 100])
@pytest.mark.parametrize("kv,hq", [("bf16", 4), ("e4m3", 2)])
def test_the_last_keys(kv, hq, end):
    """Both kernels; keys below the windows keep what they had."""
    f = Far(end, hq, 1, 64, kv, seed=41)
    p, n = f.small, f.small.lens[0]
    mass = torch.zeros(1, 1, MOST, device="cuda")
    for m in (1, 5, 70):
        for rule in (dict(window=100), dict(window=100, cap=8.0), dict(window=60, slopes=0.1)):
            r = f.rule(**rule)
            qo, qo_t, q, q64 = queries(p, m)
            _, lse = prefill(p, r, q, qo, qo_t)
            mass.zero_()
            mass[0, 0, f.start - 3:f.start] = 2.0
            pkv.pkv_score_mass(f.desc, r.score, q, qo_t, p.k_pool, f.table, f.len, end, lse, mass, keep=0.5, max_q_len=m,
                               k_scale=p.scales["k_scale"])
            assert pkv.pkv_device_errors() == 0
            want, bound = r.mass(p, 0, q64, np.arange(n - m, n), lse.cpu().numpy())
            close(mass[0, :, f.start:end], want, bound + 2.0 ** -24 * (m + 8) * want + 1e-38, (m, rule))
            assert torch.equal(mass[0, 0, f.start - 3:f.start], torch.ones(3, device="cuda"))
            assert not mass[0, 0, :f.start - 3].any() and not mass[0, 0, end:].any()
