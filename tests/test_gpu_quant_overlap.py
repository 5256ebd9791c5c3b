"""The quantising append refuses a q_out that shares bytes with k_new or v_new, and takes every
other layout of one buffer."""
import numpy as np
import pytest
import torch

import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D = 4, 2, 64


def shares(n, a, sa, ra, b, sb, rb):
    one = {a + i * sa + j for i in range(n) for j in range(ra)}
    return any(b + i * sb + j in one for i in range(n) for j in range(rb))


@pytest.mark.parametrize("n", [1, 2, 5])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_of_one_buffer(n, in_place):
    rng = np.random.default_rng(n)
    buf = torch.zeros(8192, dtype=torch.bfloat16, device=DEV)
    d = pkv.make_desc(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, num_blocks=4, max_blocks_per_seq=4, kv_dtype="int8")
    pools = [torch.zeros(4, HKV, pkv.pkv_quant_record_bytes(d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    rope = pkv.make_rope(torch.zeros(8, D // 2, 2, device=DEV))
    i32 = dict(dtype=torch.int32, device=DEV)
    tables, tts, pos = torch.zeros(1, 4, **i32), torch.full((n,), -1, **i32), torch.zeros(n, **i32)  # all padding
    seen = {}
    for turn in range(300):
        qos = int(rng.choice([256, 264, 512, 768]))
        new = int(rng.choice([128, 136, 512, 768])) if rng.random() < 0.5 else max(qos, 128)
        qo, k, v, q = (8 * int(x) for x in rng.integers(0, 300, 4))
        q = qo if in_place else 6000  # apart from all
        rows = lambda at, stride, h: torch.as_strided(buf, (n, h, D), (stride, D, 1), at)  # noqa: E731
        met = [name for name, at in (("k_new", k), ("v_new", v)) if shares(n, qo, qos, HQ * D, at, new, HKV * D)]
        if not met and not in_place and shares(n, qo, qos, HQ * D, q, 256, HQ * D):
            continue
        kw = dict(desc=d, k_pool=pools[0], v_pool=pools[1], block_tables=tables, token_to_seq=tts, positions=pos,
                  k_new=rows(k, new, HKV), v_new=rows(v, new, HKV), q=rows(q, qos if in_place else 256, HQ),
                  q_out=rows(qo, qos, HQ), rope=rope)
        if met:
            with pytest.raises(pkv.PkvError, match="q_out overlaps"):
                pkv.pkv_quant_append(**kw)
        else:
            pkv.pkv_quant_append(**kw)
        seen[bool(met)] = seen.get(bool(met), 0) + 1
    assert min(seen[True], seen[False]) > 20
    torch.cuda.synchronize()
    assert not torch.any(buf) and pkv.pkv_device_errors() == 0


def test_the_packed_projection_is_taken():
    """q, k and v side by side in one token's row, q in place and out."""
    n, heads = 9, HQ + 2 * HKV
    d = pkv.make_desc(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, num_blocks=4, max_blocks_per_seq=4, kv_dtype="int8")
    pools = [torch.zeros(4, HKV, pkv.pkv_quant_record_bytes(d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    rope = pkv.make_rope(torch.from_numpy(pkv.pkv_rope_scaled_table(1e4, D, 16)).to(DEV))
    buf = torch.randn(n, heads, D, device=DEV).bfloat16()
    tables = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    tts, pos = torch.zeros(n, dtype=torch.int32, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    out = torch.empty(n, HQ, D, dtype=torch.bfloat16, device=DEV)
    for order in ((0, HQ, HQ + HKV), (2 * HKV, 0, HKV), (HKV, 0, HKV + HQ)):
        b = buf.clone()
        q, k, v = (b[:, at:at + h] for at, h in zip(order, (HQ, HKV, HKV)))
        pkv.pkv_quant_append(d, pools[0], pools[1], tables, tts, pos, k, v, q=q, q_out=out, rope=rope)
        pkv.pkv_quant_append(d, pools[0], pools[1], tables, tts, pos, k, v, q=q, rope=rope)
        assert torch.equal(q, out)
