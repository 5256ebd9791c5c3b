"""Attention under a cap repeats its bits, on the GPU: a sequence's output depends on its own
queries and keys, not on its neighbours in the batch nor on what ran before."""
import numpy as np
import pytest
import torch

from _score import Paged, Rule
from test_gpu_score import prefill, problem

pytestmark = pytest.mark.gpu
LENS = [437, 300, 256, 640]


def bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32).clone()


def run(p, r, q, qo, qo_t):
    out, lse = prefill(p, r, q, qo, qo_t)
    return bits(out), bits(lse)


CAPS = [1.0, 2.5, 4.0, 60.0]  # scores past 0.7 of the cap, just below 0.3 and on both sides of it, far below


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 2, 64), (3, 1, 128), (12, 1, 64), (5, 5, 128)])
@pytest.mark.parametrize("cap", CAPS)
def test_neighbours_change_no_bit(kv, hq, hkv, d, cap):
    """The last rows of a sequence's last query tile are the next sequence's queries."""
    n = 48
    q_lens = [37, 11] * (n // 2)  # the first of each pair stays, the other changes
    p = Paged([256 + 5 * s for s in range(n)], hq, hkv, d, kv, seed=hq + d)
    r = Rule(d, hq, n, cap=cap)
    qo, qo_t, q, _ = problem(p, q_lens)
    q = (q.float() * 0.1).bfloat16()  # logits of about 0.15
    stay = torch.from_numpy(np.repeat(np.arange(n) % 2 == 0, q_lens)).to("cuda")
    want = run(p, r, q, qo, qo_t)
    for size in (0.0, 8.0, 200.0):
        other = (q.float() * size).bfloat16()
        other[stay] = q[stay]
        got = run(p, r, other, qo, qo_t)
        assert torch.equal(got[0][stay], want[0][stay]) and torch.equal(got[1][stay], want[1][stay]), size


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(3, 1, 128), (12, 1, 128), (5, 1, 64), (7, 1, 128), (4, 1, 128)])
@pytest.mark.parametrize("cap", CAPS)
def test_what_ran_before_changes_no_bit(kv, hq, hkv, d, cap):
    """Groups that do not divide 128: a query tile's last rows are those of no query, and hold what
    another kernel left in shared memory."""
    p = Paged(LENS, hq, hkv, d, kv, seed=hq + d)
    r = Rule(d, hq, 4, cap=cap)
    qo, qo_t, q, _ = problem(p, [200, 257, 130, 500])
    q = (q.float() * 0.1).bfloat16()
    # a call of 256 sequences that fills each of its query tiles
    n, m = 256, 128
    fill = Paged([m], 4, 1, d, kv, seed=1)
    fill.lens, fill.t = [m] * n, fill.t.repeat(n, 1).contiguous()
    fill.lens_t = torch.full((n,), m, dtype=torch.int32, device="cuda")
    fill_r = Rule(d, 4, n, cap=30.0)
    fill_qo = (m * np.arange(n + 1)).astype(np.int32)
    fill_qo_t = torch.from_numpy(fill_qo).to("cuda")
    rows = torch.randn(n * m, 4, d, device="cuda")
    want = None
    for size in (0.0, 300.0, 1.0, 3e4):
        prefill(fill, fill_r, (rows * size).bfloat16(), fill_qo, fill_qo_t)
        got = run(p, r, q, qo, qo_t)
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), size


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (6, 2), (12, 1)])
@pytest.mark.parametrize("cap,slopes", [(1.0, None), (4.0, None), (60.0, None), (4.0, 0.1)])
def test_alone_and_in_a_batch_the_same_bits(kv, hq, hkv, cap, slopes):
    q_lens = [137, 201, 90, 333]
    p = Paged(LENS, hq, hkv, 128, kv, seed=hq)
    r = Rule(128, hq, 4, cap=cap, slopes=slopes)
    qo, qo_t, q, _ = problem(p, q_lens)
    q = (q.float() * 0.1).bfloat16()
    q[int(qo[1]):int(qo[2])] *= 20
    want = run(p, r, q, qo, qo_t)
    assert all(torch.equal(x, y) for x, y in zip(want, run(p, r, q, qo, qo_t)))
    lens, tables = p.lens, p.t
    for s in range(4):
        a, b = int(qo[s]), int(qo[s + 1])
        p.lens, p.lens_t, p.t = [lens[s]], torch.tensor(lens[s:s + 1], dtype=torch.int32, device="cuda"), tables[s:s + 1]
        one = np.array([0, b - a], np.int32)
        got = run(p, Rule(128, hq, 1, cap=cap, slopes=slopes), q[a:b], one, torch.from_numpy(one).to("cuda"))
        assert torch.equal(got[0], want[0][a:b]) and torch.equal(got[1], want[1][a:b]), s
