"""65535 sequences, the most a call takes, on the GPU: weights by both kernels, choice and move."""
import numpy as np
import pytest
import torch

import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
N, HQ, HKV, D, BLOCKS, WIDTH = 65535, 4, 2, 64, 64, 40


def problem(q_len):
    """Every sequence's queries, at most q_len of them, over up to 40 keys in blocks that all share."""
    gen = torch.Generator(device=DEV).manual_seed(q_len)
    rand = lambda lo, hi: torch.randint(lo, hi, (N,), generator=gen, device=DEV, dtype=torch.int32)  # noqa: E731
    lens = rand(0, WIDTH + 1)
    size = torch.minimum(rand(0, q_len + 1), lens)
    qo = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    qo[1:] = torch.cumsum(size, 0)
    pool = torch.randn(BLOCKS, HKV, 16, D, generator=gen, device=DEV).bfloat16()
    tables = torch.randint(0, BLOCKS, (N, 3), generator=gen, device=DEV, dtype=torch.int32)
    q = torch.randn(int(qo[-1]), HQ, D, generator=gen, device=DEV).bfloat16()
    return lens, size, qo, pool, tables, q


@pytest.mark.parametrize("q_len", [3, 20])  # up to 6 and up to 40 query rows
def test_weights(q_len):
    lens, size, qo, pool, tables, q = problem(q_len)
    desc = pkv.make_desc(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, num_blocks=BLOCKS, max_blocks_per_seq=3)
    lse = torch.full((q.shape[0], HQ), 3.0, device=DEV)
    mass = torch.rand(N, HKV, WIDTH, device=DEV)
    got = mass.clone()
    pkv.pkv_score_mass(desc, pkv.make_score(0.125), q, qo, pool, tables, lens, WIDTH, lse, got, keep=0.5, max_q_len=q_len)
    assert pkv.pkv_device_errors() == 0
    t = torch.arange(WIDTH, device=DEV)
    seq = torch.repeat_interleave(torch.arange(N, device=DEV), size.long())
    pos = torch.arange(q.shape[0], device=DEV) - qo[seq] + lens[seq] - size[seq]
    want = 0.5 * mass.double() * (t < (lens - size)[:, None])[:, None]
    for rows in torch.arange(q.shape[0], device=DEV).split(20000):  # (a part at a time: its keys in 64 bits)
        keys = pool[tables[seq[rows]].long()].double().transpose(1, 2).flatten(2, 3)[:, :, :WIDTH]  # [row][Hkv][t][D]
        x = (q[rows].double().unflatten(1, (HKV, 2, 1)) * keys[:, :, None]).sum(-1) * 0.125
        w = torch.exp(x - 3.0).sum(2) * (t <= pos[rows, None])[:, None]
        want.index_add_(0, seq[rows], w)
    want = torch.where((t < lens[:, None])[:, None], want, mass.double())
    # logits up to 8 in fp32 over 64 dims: 64 * 2^-24 * sum |q k| / 8 < 5e-5; the rest is less
    assert ((got - want).abs() <= 1e-4 * want + 1e-30).all()


def test_choice_and_move():
    lens, _, _, pool, tables, _ = problem(1)
    gen = torch.Generator(device=DEV).manual_seed(9)
    mass = torch.rand(N, HKV, WIDTH, generator=gen, device=DEV)
    kept = torch.full((N, HKV, 16), -1, dtype=torch.int32, device=DEV)
    kept_lens = torch.zeros(N, dtype=torch.int32, device=DEV)
    pkv.pkv_evict_select(mass, lens, WIDTH, 16, 1, 2, kept, kept_lens)
    assert torch.equal(kept_lens, lens.clamp(max=16))
    t = torch.arange(WIDTH, device=DEV)
    n = lens[:, None, None]
    ends = (t < 1) | (t >= n - 2)
    score = torch.where(ends, torch.full_like(mass, 9.0), mass).masked_fill(t >= n, -1.0)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :16]
    order = torch.sort(order.masked_fill(torch.arange(16, device=DEV) >= n, 10 ** 6), -1).values
    want = torch.where(order == 10 ** 6, torch.full_like(order, -1), order).int()
    assert torch.equal(kept, want)
    desc, dst_desc = (pkv.make_desc(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, num_blocks=b, max_blocks_per_seq=m)
                      for b, m in ((BLOCKS, 3), (N, 1)))
    k, v = (torch.zeros(N, HKV, 16, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dst = torch.randperm(N, generator=gen, device=DEV).int()[:, None].contiguous()
    out = torch.zeros(N, HKV, 16, device=DEV)
    pkv.pkv_evict_compact(desc, pool, -pool, tables, kept, kept_lens, dst_desc=dst_desc, k_dst=k, v_dst=v, dst_tables=dst,
                          mass=mass, mass_out=out)
    assert pkv.pkv_device_errors() == 0
    at = kept.clamp(min=0).long()
    rows = pool[torch.gather(tables.long()[:, None].expand(N, HKV, 3), 2, at // 16),
                torch.arange(HKV, device=DEV)[:, None], at % 16].masked_fill((kept < 0)[..., None], 0.0)
    assert torch.equal(k[dst[:, 0].long()], rows) and torch.equal(v[dst[:, 0].long()].abs(), rows.abs())
    assert torch.equal(out, torch.gather(mass, 2, at).masked_fill(kept < 0, 0.0))
