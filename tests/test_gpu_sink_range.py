"""Sinks far above and below every logit, on the GPU: however many chunks a context is cut into,
lse is ln(sum of e^x + e^sink)."""
import numpy as np
import pytest
import torch

from _score import Paged, Rule
from test_gpu_score import check_decode, check_prefill, decode, prefill, problem
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
LENS = [1, 640, 0, 17, 330, 64, 500, 2]
SINKS = [100.0, -100.0, 88.0, 95.0, 400.0, -3e38, 5.0, 3e30]


def rule_of(d, hq, **kw):
    r = Rule(d, hq, len(LENS), sinks=True, **kw)
    r.sinks = np.resize(np.array(SINKS, np.float32), hq)
    r.score = pkv.make_score(r.scale, cap=r.cap, window=r.window, sinks=torch.from_numpy(r.sinks).to("cuda"))
    return r


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (16, 2, 64), (8, 8, 128)])
@pytest.mark.parametrize("chunk", [64, 20, 14, 10, 4, 1])  # one chunk, clusters of 2, 3 and 4, more by tickets
@pytest.mark.parametrize("rule", [dict(), dict(cap=8.0)])
def test_decode(kv, hq, hkv, d, chunk, rule):
    p = Paged(LENS, hq, hkv, d, kv, seed=chunk)
    r = rule_of(d, hq, **rule)
    q, q64 = p.queries(len(LENS))
    check_decode(p, r, q64, *decode(p, r, q, chunk=chunk))
    if rule:
        return
    # the plain decode
    size = pkv.pkv_decode_workspace_size(p.desc, len(LENS), 640, 0, chunk)
    ws = torch.zeros(max(256, size), dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, float("nan")), torch.full((len(LENS), hq), float("nan"), device="cuda")
    pkv.pkv_decode_attention(p.desc, q, p.k_pool, p.v_pool, p.t, p.lens_t, 640, r.scale, out, lse, ws, chunk_blocks=chunk,
                             sinks=torch.from_numpy(r.sinks).to("cuda"), **p.scales)
    check_decode(p, r, q64, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 64), (16, 4, 128)])
@pytest.mark.parametrize("q_lens", [[1, 4, 0, 3, 2, 4, 1, 2], [1, 100, 0, 17, 33, 64, 130, 2]])
def test_prefill_and_few_queries(kv, hq, hkv, d, q_lens):
    p = Paged(LENS, hq, hkv, d, kv, seed=5)
    for rule in (dict(), dict(cap=8.0), dict(window=300)):
        r = rule_of(d, hq, **rule)
        qo, qo_t, q, q64 = problem(p, q_lens)
        check_prefill(p, r, q64, qo, *prefill(p, r, q, qo, qo_t))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_logits_far_below_a_sink(kv):
    """Every logit at -200 or less under sinks of about 0: lse is the sink, the output nothing."""
    p = Paged([640, 100], 8, 2, 64, kv, seed=6)
    p.k_pool.zero_()
    p.k_pool[..., 0] = 16.0 if kv == "bf16" else torch.tensor(16.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    scale = np.ones(2) if kv == "bf16" else p.scales["k_scale"].cpu().double().numpy()
    for s, n in enumerate(p.lens):
        p.k[s] = np.zeros((n, 2, 64))
        p.k[s][..., 0] = 16.0 * scale
    r = Rule(64, 8, 2, sinks=True)
    q = torch.zeros(3, 8, 64, device="cuda").bfloat16()
    q[..., 0] = -128.0 / scale.min()
    q64 = q.double().cpu().numpy()
    for chunk in (64, 20, 10, 2):
        out, lse = decode(p, r, q[:2], chunk=chunk)
        check_decode(p, r, q64[:2], out, lse)
        assert np.array_equal(lse.cpu().numpy(), np.stack([r.sinks] * 2)) and not out.any()
    qo = np.array([0, 2, 3], np.int32)
    out, lse = prefill(p, r, q, qo, torch.from_numpy(qo).to("cuda"))
    check_prefill(p, r, q64, qo, out, lse)
