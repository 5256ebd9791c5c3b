"""Decode under a score rule with the stream-ordering promises of the descriptor, on the GPU."""
import pytest
import torch

from _score import Paged, Rule
from test_gpu_score import check_decode, decode
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
LENS = [1, 640, 0, 17, 330, 64]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("flags", [1, 3])
@pytest.mark.parametrize("chunk", [0, 20, 4])
def test_promises_change_no_bit(kv, flags, chunk):
    """Behind another call of the library that touches nothing of this one's."""
    p = Paged(LENS, 8, 2, 128, kv, seed=61)
    r = Rule(128, 8, len(LENS), cap=12.0, slopes=0.1, sinks=True)
    q, q64 = p.queries(len(LENS))
    want, want_lse = decode(p, r, q, chunk=chunk)
    other = Paged([900, 30], 8, 2, 128, kv, seed=62)
    rule = Rule(128, 8, 2, cap=12.0)
    q2, _ = other.queries(2)
    p.desc = p.make_desc(flags=flags)
    ws, ws2 = (torch.zeros(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(2))
    out2, lse2 = torch.zeros_like(q2), torch.zeros(2, 8, device="cuda")
    for _ in range(5):
        out, lse = torch.full_like(q, float("nan")), torch.full((len(LENS), 8), float("nan"), device="cuda")
        torch.cuda.synchronize()
        pkv.pkv_score_decode(other.desc, rule.score, q2, other.k_pool, other.v_pool, other.t, other.lens_t, 900, out2, lse2,
                             ws2, **other.scales)
        pkv.pkv_score_decode(p.desc, r.score, q, p.k_pool, p.v_pool, p.t, p.lens_t, 640, out, lse, ws, chunk_blocks=chunk,
                             **p.scales)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check_decode(p, r, q64, out, lse)
