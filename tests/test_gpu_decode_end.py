"""Decode of a context that ends at the end of 32 bits, on the GPU: the bits of the same keys at
the beginning."""
import pytest
import torch

from _far import Far
from test_gpu_score import check_decode, decode
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("end", [MOST, MOST - 1, MOST - 15, MOST - 16])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("e4m3", 64)])
def test_the_last_position(kv, d, end):
    """The slot behind the last key, in its block, holds a NaN."""
    f = Far(end, 8, 2, d, kv, seed=42)
    p = f.small
    q, q64 = p.queries(1)
    for rule in (dict(window=200), dict(window=30, cap=9.0), dict(window=200, slopes=0.1, sinks=True)):
        r = f.rule(**rule)
        want, want_lse = decode(p, r, q)
        check_decode(p, r, q64, want, want_lse)
        ws = torch.zeros(max(256, pkv.pkv_decode_workspace_size(f.desc, 1, end, r.window, 0)), dtype=torch.uint8,
                         device="cuda")
        out, lse = torch.zeros_like(q), torch.zeros_like(want_lse)
        pkv.pkv_score_decode(f.desc, r.score, q, p.k_pool, p.v_pool, f.table, f.len, end, out, lse, ws, **p.scales)
        assert pkv.pkv_device_errors() == 0
        p.lens_t, p.t, p.desc, kept = f.len, f.table, f.desc, (p.lens_t, p.t, p.desc)
        check_decode(p, r, q64, out, lse)
        if rule == dict(window=200):
            out.zero_()
            pkv.pkv_decode_attention(f.desc, q, p.k_pool, p.v_pool, f.table, f.len, end, r.scale, out, lse, ws, window=200,
                                     **p.scales)
            check_decode(p, r, q64, out, lse)
        p.lens_t, p.t, p.desc = kept
