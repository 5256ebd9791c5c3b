"""Weights where a query's lse is -inf, on the GPU: it adds nothing, whatever its row of q holds,
as in a batch padded with rows that nobody wrote."""
import numpy as np
import pytest
import torch

from _score import Paged, Rule
from test_gpu_score import check_mass, mass_of, prefill, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (12, 1, 128)])
@pytest.mark.parametrize("rule", [dict(), dict(cap=8.0), dict(slopes=0.1), dict(cap=8.0, slopes=0.1, window=70),
                                  dict(causal=False)])
@pytest.mark.parametrize("q_lens", [[1, 2, 1], [70, 150, 300]])
def test_rows_that_count_for_nothing(kv, hq, hkv, d, rule, q_lens):
    p = Paged([90, 400, 513], hq, hkv, d, kv, seed=51)
    r = Rule(d, hq, 3, **rule)
    qo, qo_t, q, q64 = problem(p, q_lens)
    _, lse = prefill(p, r, q, qo, qo_t)
    rows = q.shape[0]
    dead = np.zeros((rows, hq), bool)
    dead[0] = dead[-1] = True  # sequence 0 has no row left where it has one
    dead[rows // 2, hq // 2:] = True
    if rows > 100:
        dead[80:122] = True
    lse[torch.from_numpy(dead).to("cuda")] = float("-inf")
    start = torch.rand(3, hkv, 513, device="cuda")
    want = None
    for junk in (0.0, float("nan"), float("inf"), -3e38):
        bad = q.clone()
        bad[torch.from_numpy(dead).to("cuda")] = junk
        got = mass_of(p, r, bad, qo_t, lse, start, 1.0, max(q_lens))
        check_mass(p, r, q64, qo, lse, start, 1.0, got)
        want = got if want is None else want
        assert torch.equal(got, want), junk
