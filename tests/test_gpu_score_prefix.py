"""Prefix lengths at the ends of 32 bits, on the GPU: any value may stand there, of which at most
the sequence's length counts, and none below 1."""
import numpy as np
import pytest
import torch

from _score import Paged, Rule
from test_gpu_score import check_mass, check_prefill, mass_of, prefill, problem

pytestmark = pytest.mark.gpu
LOWEST, MOST = -2 ** 31, 2 ** 31 - 1
LENS = [300, 513, 260, 700, 390, 129]
RULES = [dict(), dict(cap=5.0), dict(slopes=0.2), dict(cap=5.0, slopes=0.2), dict(cap=20.0, window=150)]


def rule_of(d, hq, rule, prefix):
    r = Rule(d, hq, len(LENS), prefix=prefix, **rule)
    r.prefix = np.clip(prefix, 0, LENS)  # what counts of them
    return r


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("q_lens", [[200, 300, 140, 400, 390, 100], [4, 8, 1, 6, 2, 3]])
def test_any_prefix_length_may_stand_there(kv, rule, q_lens):
    """Several key tiles before, across and behind the diagonal; the tile, the short-query and both
    weight kernels."""
    p = Paged(LENS, 8, 2, 64, kv, seed=31)
    for prefix in ([LOWEST, MOST, -1, LOWEST + 1, 0, LOWEST], [MOST, LOWEST, LOWEST, MOST, LOWEST, MOST - 1]):
        r = rule_of(64, 8, rule, prefix)
        qo, qo_t, q, q64 = problem(p, q_lens)
        out, lse = prefill(p, r, q, qo, qo_t)
        check_prefill(p, r, q64, qo, out, lse)
        start = torch.rand(len(LENS), 2, 704, device="cuda")
        check_mass(p, r, q64, qo, lse, start, 1.0, mass_of(p, r, q, qo_t, lse, start, 1.0, max(q_lens)))
