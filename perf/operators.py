"""Timing cases for the quantised-cache and rotary operators of the library.

Four operators are exercised, each in a plain form (elementary torch, 32-bit
arithmetic) and through the library's entry points (``own`` true):

* ``rope``   rotary positions on q and k: half-split or interleaved pairs, the
             whole head or its first ``rotary_dim`` dims, rows of a packed QKV
             buffer, bf16 / f16 / f32;
* ``store``  the new tokens' K (rotated) and V quantised as they are written
             into a paged int8 or 4-bit pool, then read back as rows;
* ``load``   whole blocks of a quantised pool widened into a bf16 pool, as for
             a prefill over a cached prefix;
* ``decode`` one query token per sequence over a quantised paged pool.

Pool layout: one record per (block, KV head): the codes of the block's 16
rows, then their scales.  int8: D bytes a row holding code + 128, then 16 fp32
scales (value = code * scale).  4-bit: D / 2 bytes a row (dim 2i in the low
nibble of byte i), then [16][D / 16] e4m3 scales, one per 16 dims (value =
e2m1 * scale * the head's fp32 scale).  Inside the codes, the 16-byte chunk c of
row r sits at chunk c ^ ((r * row_bytes / 128) mod chunks).
"""
import math
import random

import torch

own = False

BLOCK = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the rotation of one decode step of a small batch: latency
        dict(name="rope_step", op="rope", tokens=4, hq=8, hkv=2, d=64, rotary=64, layout="half",
             dtype="bf16", packed=False, max_pos=4096),
        # a mixed step's prompt chunks, q and k inside the packed QKV projection's output
        dict(name="rope_prompt", op="rope", tokens=4096, hq=32, hkv=8, d=128, rotary=128,
             layout="half", dtype="bf16", packed=True, max_pos=32768),
        # interleaved pairs on half of each head, an odd token count, far positions
        dict(name="rope_partial", op="rope", tokens=8191, hq=16, hkv=2, d=128, rotary=64,
             layout="interleaved", dtype="f16", packed=False, max_pos=131072),
        # the KV write of a decode step: one token of each of 256 sequences
        dict(name="store_step_int8", op="store", fmt="int8", seqs=256, chunk=1, ctx=768, hq=32,
             hkv=8, d=128, rotary=128, layout="half", out="bf16"),
        # eight prompt chunks of 512 tokens appended behind their cached prefixes
        dict(name="store_prompt_fp4", op="store", fmt="fp4", seqs=8, chunk=512, ctx=8192, hq=32,
             hkv=8, d=128, rotary=128, layout="half", out="bf16"),
        # small heads, ragged odd chunks, half-rotated interleaved heads
        dict(name="store_odd_fp4", op="store", fmt="fp4", seqs=9, chunk=111, ctx=1024, hq=64,
             hkv=8, d=64, rotary=32, layout="interleaved", out="f32"),
        # the cached prefixes of a prompt batch widened for the prefill
        dict(name="load_prefix_fp4", op="load", fmt="fp4", blocks=4096, hkv=8, d=128),
        # a short prefix of a small-head int8 cache
        dict(name="load_short_int8", op="load", fmt="int8", blocks=333, hkv=8, d=64),
        # the smallest decode: four short ragged sequences
        dict(name="decode_small_int8", op="decode", fmt="int8", seqs=4, lo=17, hi=255, hq=8, hkv=2,
             d=64, window=0, sinks=False),
        # one GPU's batch of a two-KV-head layer
        dict(name="decode_mid_fp4", op="decode", fmt="fp4", seqs=64, lo=256, hi=4096, hq=16, hkv=2,
             d=128, window=0, sinks=False),
        # a wide group over small heads with attention sinks
        dict(name="decode_wide_int8", op="decode", fmt="int8", seqs=128, lo=1024, hi=16384, hq=64,
             hkv=8, d=64, window=0, sinks=True),
        # a long ragged batch, the largest cache read
        dict(name="decode_long_fp4", op="decode", fmt="fp4", seqs=120, lo=1024, hi=32768, hq=32,
             hkv=8, d=128, window=0, sinks=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "store", "load", "decode", "decode"))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 3, 4, 8))
    hq = hkv * rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
    fmt = rng.choice(("int8", "fp4"))
    rotary = rng.choice((d, d, d // 2, d // 4, 18))
    layout = rng.choice(("half", "interleaved"))
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, max(2, 160000 // (hq + hkv))), hq=hq, hkv=hkv, d=d,
                    rotary=rotary, layout=layout, dtype=rng.choice(("bf16", "f16", "f32")),
                    packed=rng.random() < 0.5, max_pos=_log(rng, 64, 131072))
    if op == "store":
        seqs = _log(rng, 1, 64)
        chunk = _log(rng, 1, max(2, 60000 // ((hq + hkv) * seqs)))
        return dict(op=op, fmt=fmt, seqs=seqs, chunk=chunk, ctx=chunk + _log(rng, 1, 2048), hq=hq,
                    hkv=hkv, d=d, rotary=rotary, layout=layout, out=rng.choice(("bf16", "f32")))
    if op == "load":
        return dict(op=op, fmt=fmt, blocks=_log(rng, 1, 30000 // hkv), hkv=hkv, d=d)
    seqs = _log(rng, 1, 128)
    hi = _log(rng, 1, max(2, min(32768, 6000000 // (seqs * hkv))))
    window = rng.choice((0, 0, 0, _log(rng, 1, 512)))
    return dict(op=op, fmt=fmt, seqs=seqs, lo=max(0, hi // rng.choice((1, 4, 16)) - 1), hi=hi, hq=hq,
                hkv=hkv, d=d, window=window, sinks=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs --

def _row_bytes(fmt, d):
    return d if fmt == "int8" else d // 2


def _scale_bytes(fmt, d):
    return 4 if fmt == "int8" else d // BLOCK


def _record(fmt, d):
    return BLOCK * (_row_bytes(fmt, d) + _scale_bytes(fmt, d))


def _code_at(fmt, d, dev):
    """[16][row bytes]: where byte j of row r sits among a record's codes."""
    rb = _row_bytes(fmt, d)
    r = torch.arange(BLOCK, device=dev)[:, None]
    j = torch.arange(rb, device=dev)[None, :]
    return r * rb + (((j // 16) ^ ((r * rb // 128) % (rb // 16))) * 16) + j % 16


def _table(max_pos, rotary, dev, theta=1.0e6):
    """fp32 [max_pos][rotary / 2][2] (cos, sin), angles in 64 bits."""
    j = torch.arange(rotary // 2, dtype=torch.float64, device=dev)
    ang = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * theta ** (-2.0 * j / rotary)
    return torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()


def _pool(fmt, nb, hkv, d, gen, dev):
    """A pool of quantised N(0, 1) rows: each row is one of 8192 quantised ones."""
    bank = torch.randn(8192, d, generator=gen, device=dev)
    if fmt == "int8":
        codes, scales = _quant_int8(bank)
        scales = scales[:, None].contiguous().view(torch.uint8)
    else:
        codes, scales = _quant_fp4(bank, torch.full((1,), 4.5 / 2688.0, device=dev))
    pick = torch.randint(0, 8192, (nb, hkv, BLOCK), generator=gen, device=dev)
    pool = torch.empty(nb, hkv, _record(fmt, d), dtype=torch.uint8, device=dev)
    rb = _row_bytes(fmt, d)
    r = torch.arange(BLOCK, device=dev)[:, None]
    c = torch.arange(rb // 16, device=dev)[None, :] ^ ((r * rb // 128) % (rb // 16))
    step = 8192
    for a in range(0, nb, step):
        p = pick[a:a + step]
        rows = codes[p].view(p.shape[0], hkv, BLOCK, rb // 16, 16)
        pool[a:a + step, :, :BLOCK * rb] = rows[:, :, r, c].reshape(p.shape[0], hkv, -1)
        pool[a:a + step, :, BLOCK * rb:] = scales[p].reshape(p.shape[0], hkv, -1)
    return pool


def _tables(lens, dev, rng):
    """Scattered block tables: every sequence its own blocks, -1 past its end."""
    n = [(x + BLOCK - 1) // BLOCK for x in lens]
    nb = max(1, sum(n))
    perm = list(range(nb))
    rng.shuffle(perm)
    width = max(1, max(n))
    rows, at = [], 0
    for k in n:
        rows.append(perm[at:at + k] + [-1] * (width - k))
        at += k
    return torch.tensor(rows, dtype=torch.int32, device=dev), nb


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case)
    op, d = case["op"], case["d"]
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    if op == "rope":
        t, hq, hkv, dt = case["tokens"], case["hq"], case["hkv"], DTYPES[case["dtype"]]
        if case["packed"]:  # q | k | v of the projection, side by side per token
            qkv = randn(t, hq + 2 * hkv, d).to(dt)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = randn(t, hq, d).to(dt), randn(t, hkv, d).to(dt)
        s["q_out"], s["k_out"] = (torch.empty(t, h, d, dtype=dt, device=dev) for h in (hq, hkv))
        s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=gen, device=dev).int()
        s["table"] = _table(case["max_pos"], case["rotary"], dev)
        if own:
            s["rope"] = _lib().make_rope(s["table"], layout=case["layout"])
        return s
    fmt, hkv = case["fmt"], case["hkv"]
    if op == "store":
        n, chunk = case["seqs"], case["chunk"]
        lens = [rng.randint(chunk, case["ctx"]) for _ in range(n)]
        s["tables"], nb = _tables(lens, dev, rng)
        t = n * chunk
        s["token_to_seq"] = torch.arange(n, device=dev).repeat_interleave(chunk).int()
        first = torch.tensor([x - chunk for x in lens], device=dev).repeat_interleave(chunk)
        s["positions"] = (first + torch.arange(chunk, device=dev).repeat(n)).int()
        s["q"], s["k"], s["v"] = (randn(t, h, d).bfloat16() for h in (case["hq"], hkv, hkv))
        s["q_out"] = torch.empty_like(s["q"])
        s["table"] = _table(case["ctx"], case["rotary"], dev)
        out = DTYPES[case["out"]]
        s["k_out"], s["v_out"] = (torch.empty(t, hkv, d, dtype=out, device=dev) for _ in range(2))
    elif op == "load":
        nb = case["blocks"] * 2
        s["src"] = torch.randperm(nb, generator=gen, device=dev)[:case["blocks"]].int()
        s["dst"] = torch.randperm(case["blocks"], generator=gen, device=dev).int()
        s["k_out"], s["v_out"] = (torch.zeros(case["blocks"], hkv, BLOCK, d, dtype=torch.bfloat16,
                                              device=dev) for _ in range(2))
    else:
        lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
        s["tables"], nb = _tables(lens, dev, rng)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["max_len"] = max(1, max(lens))
        s["q"] = randn(case["seqs"], case["hq"], d).bfloat16()
        s["sink"] = randn(case["hq"]) if case["sinks"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=dev)
    # the 4-bit heads' fp32 scales, frozen from a warm-up: amax / (6 * 448), amax about 4.5
    s["k_scale"], s["v_scale"] = (((4.2 + 0.6 * torch.rand(hkv, generator=gen, device=dev)) / 2688.0)
                                  if fmt == "fp4" else None for _ in range(2))
    if op == "store":
        s["k_pool"], s["v_pool"] = (torch.zeros(nb, hkv, _record(fmt, d), dtype=torch.uint8, device=dev)
                                    for _ in range(2))
    else:
        s["k_pool"] = _pool(fmt, nb, hkv, d, gen, dev)
        s["v_pool"] = _pool(fmt, nb, hkv, d, gen, dev)
    if own:
        lib = _lib()
        s["desc"] = lib.make_desc(num_q_heads=case.get("hq", hkv), num_kv_heads=hkv, head_dim=d,
                                  num_blocks=nb, kv_dtype=lib.KV_INT8 if fmt == "int8" else lib.KV_FP4,
                                  max_blocks_per_seq=s["tables"].shape[1] if "tables" in s else 1)
        if op == "store":
            s["rope"] = lib.make_rope(s["table"], layout=case["layout"])
        if op == "decode":
            n = lib.pkv_quant_decode_workspace_size(s["desc"], case["seqs"], s["max_len"],
                                                    window=case["window"])
            s["workspace"] = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev)
    return s


def _lib():
    import paged_kv_attention_21_gb300 as pkv
    return pkv


# ------------------------------------------------------------- plain forms --

def _quant_int8(x):
    """Rows of fp32 -> (codes + 128 as bytes, fp32 scale of each row)."""
    s = x.abs().amax(-1) / torch.full((), 127.0, device=x.device)  # a true quotient, as below
    c = torch.where(s[..., None] > 0, torch.round(x / s[..., None]), torch.zeros_like(x))
    return (c.clamp(-127, 127) + 128).to(torch.uint8), s


def _quant_fp4(x, head_scale):
    """Rows of fp32 [..., D] and a head scale broadcast against [...] -> (packed
    e2m1 bytes [..., D / 2], e4m3 scale bytes [..., D / 16])."""
    b = x.unflatten(-1, (-1, 16))
    g = head_scale[..., None]
    e = (b.abs().amax(-1) / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = (e.float() * g)[..., None]
    y = torch.where(t > 0, b / t, torch.zeros_like(b))
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte() + 8 * torch.signbit(y).byte())
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), e.view(torch.uint8)


def _rows(fmt, d, codes, scales, head_scale):
    """Row bytes [..., row bytes] and scale bytes -> fp32 rows [..., D]."""
    if fmt == "int8":
        return (codes.float() - 128.0) * scales.contiguous().view(torch.float32)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = lut[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    v = v.unflatten(-1, (-1, 16)) * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    return v.flatten(-2) * head_scale[..., None]


def _turn(x, cs, layout):
    """Rotate fp32 rows [T][H][D] by cs [T][rotary / 2][2]; later dims pass."""
    n = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    lo, hi = a * c - b * s, b * c + a * s
    turned = torch.cat((lo, hi), -1) if layout == "half" else torch.stack((lo, hi), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _plain_store(s):
    fmt, d, hkv = s["fmt"], s["d"], s["hkv"]
    pos, seq = s["positions"].long(), s["token_to_seq"].long()
    cs = s["table"][pos]
    q = _turn(s["q"].float(), cs, s["layout"]).bfloat16()
    blk, row = s["tables"][seq, pos // BLOCK].long(), pos % BLOCK
    rb, sb = _row_bytes(fmt, d), _scale_bytes(fmt, d)
    at = _code_at(fmt, d, pos.device)[row][:, None]
    sat = (BLOCK * rb + row[:, None] * sb + torch.arange(sb, device=pos.device))[:, None]
    i, h = blk[:, None, None], torch.arange(hkv, device=pos.device)[None, :, None]

    def through(pool, x, head_scale):
        if fmt == "int8":
            codes, scales = _quant_int8(x)
            scales = scales[..., None].contiguous().view(torch.uint8)
        else:
            codes, scales = _quant_fp4(x, head_scale)
        pool[i, h, at], pool[i, h, sat] = codes, scales
        return _rows(fmt, d, pool[i, h, at], pool[i, h, sat], head_scale).to(s["k_out"].dtype)

    return (q, through(s["k_pool"], _turn(s["k"].float(), cs, s["layout"]), s["k_scale"]),
            through(s["v_pool"], s["v"].float(), s["v_scale"]))


def _blocks(fmt, d, pool, ids, head_scale):
    """fp32 [ids' shape][Hkv][16][D] of the blocks `ids`."""
    rb = _row_bytes(fmt, d)
    rec = pool[ids]
    codes = rec[..., _code_at(fmt, d, pool.device)]
    scales = rec[..., BLOCK * rb:].unflatten(-1, (BLOCK, -1))
    return _rows(fmt, d, codes, scales, None if head_scale is None else head_scale[:, None])


def _plain_decode(s):
    fmt, d, hkv, n = s["fmt"], s["d"], s["hkv"], s["seqs"]
    ids = s["tables"].long().clamp(min=0)
    rows = lambda pool, g: _blocks(fmt, d, pool, ids, g).transpose(1, 2).flatten(2, 3)  # noqa: E731
    q = s["q"].float().view(n, hkv, -1, d)
    x = q @ rows(s["k_pool"], s["k_scale"]).transpose(-1, -2) / math.sqrt(d)
    t = torch.arange(x.shape[-1], device=x.device)
    lens = s["lens"][:, None].long()
    seen = t < lens
    if s["window"] > 0:
        seen = seen & (t >= lens - s["window"])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    sink = None if s["sink"] is None else s["sink"].view(1, hkv, -1, 1)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - m)
    o = p @ rows(s["v_pool"], s["v_scale"]) / torch.where(total > 0, total, torch.ones_like(total))
    lse = m + torch.log(total)
    return o.view(n, -1, d).bfloat16(), lse.view(n, -1)


def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op == "rope":
        cs = s["table"][s["positions"].long()]
        return tuple(_turn(s[x].float(), cs, s["layout"]).to(s["q"].dtype) for x in "qk")
    if op == "store":
        return _plain_store(s)
    if op == "load":
        k, v = s["k_out"], s["v_out"]
        k[s["dst"].long()] = _blocks(s["fmt"], s["d"], s["k_pool"], s["src"].long(), s["k_scale"]).bfloat16()
        v[s["dst"].long()] = _blocks(s["fmt"], s["d"], s["v_pool"], s["src"].long(), s["v_scale"]).bfloat16()
        return k, v
    return _plain_decode(s)


def _own(s):
    lib, op = _lib(), s["op"]
    if op == "rope":
        lib.pkv_rope_rotate(s["rope"], s["positions"], s["q"], s["q_out"], s["k"], s["k_out"])
        return s["q_out"], s["k_out"]
    if op == "store":
        lib.pkv_quant_append(s["desc"], s["k_pool"], s["v_pool"], s["tables"], s["token_to_seq"],
                             s["positions"], s["k"], s["v"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        lib.pkv_quant_read(s["desc"], s["k_pool"], s["v_pool"], s["tables"], s["token_to_seq"],
                           s["positions"], s["k_out"], s["v_out"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
        return s["q_out"], s["k_out"], s["v_out"]
    if op == "load":
        lib.pkv_quant_load_blocks(s["desc"], s["k_pool"], s["v_pool"], s["src"], s["dst"], s["k_out"],
                                  s["v_out"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k_out"], s["v_out"]
    lib.pkv_quant_decode(s["desc"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"],
                         s["max_len"], 1.0 / math.sqrt(s["d"]), s["out"], s["lse"], s["workspace"],
                         window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], sinks=s["sink"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------- costs --

def work(case):
    op, d = case["op"], case["d"]
    if op == "rope":
        size = DTYPES[case["dtype"]].itemsize
        rows = case["tokens"] * (case["hq"] + case["hkv"])
        return dict(bytes=2 * rows * d * size + case["tokens"] * (4 + 4 * case["rotary"]),
                    flops=3 * rows * case["rotary"])
    fmt, hkv = case["fmt"], case["hkv"]
    row = _row_bytes(fmt, d) + _scale_bytes(fmt, d)
    if op == "store":
        t = case["seqs"] * case["chunk"]
        out = DTYPES[case["out"]].itemsize
        return dict(bytes=t * (case["hq"] * d * 4 + 2 * hkv * (2 * d + 2 * row + out * d) + 8 + 4 * case["rotary"]),
                    flops=t * (3 * case["hq"] * case["rotary"] + hkv * (3 * case["rotary"] + 8 * d)))
    if op == "load":
        rows = case["blocks"] * hkv * BLOCK * 2
        return dict(bytes=rows * (row + 2 * d), flops=2 * rows * d)
    mean = (case["lo"] + case["hi"]) / 2.0
    if case["window"] > 0:
        mean = min(mean, case["window"])
    keys = case["seqs"] * max(mean, 1.0)
    return dict(bytes=keys * hkv * 2 * row + case["seqs"] * case["hq"] * (4 * d + 4),
                flops=4 * keys * case["hq"] * d)


# ------------------------------------------------------ 64-bit definitions --

def _values64(fmt, d, rec, head_scale):
    """Records [..., Hkv, bytes] -> their [..., Hkv, 16, D] values in 64 bits."""
    rb = _row_bytes(fmt, d)
    codes = torch.empty(rec.shape[:-1] + (BLOCK, rb), dtype=torch.uint8, device=rec.device)
    for r in range(BLOCK):
        for c in range(rb // 16):
            at = r * rb + 16 * (c ^ ((r * rb // 128) % (rb // 16)))
            codes[..., r, 16 * c:16 * c + 16] = rec[..., at:at + 16]
    tail = rec[..., BLOCK * rb:].contiguous()
    if fmt == "int8":
        scale = tail.view(torch.float32).double()
        return (codes.double() - 128.0) * scale[..., None]
    scale = tail.view(torch.float8_e4m3fn).double().unflatten(-1, (BLOCK, d // 16))
    out = torch.empty(codes.shape[:-1] + (d,), dtype=torch.float64, device=rec.device)
    for nibble in range(2):
        c = ((codes >> (4 * nibble)) & 15).double()
        sign, mag = 1.0 - 2.0 * (c >= 8), c % 8
        expo, frac = torch.floor(mag / 2), mag % 2
        out[..., nibble::2] = sign * torch.where(expo == 0, frac / 2, (1 + frac / 2) * 2.0 ** (expo - 1))
    out = out * scale.repeat_interleave(16, -1)
    return out * head_scale.double()[:, None, None]


def _f32(x):
    """A 64-bit step rounded to 32 bits, where the definition rounds it."""
    return x.float().double()


def _nearest64(fmt, x, head_scale):
    """The value that each x of rows [..., Hkv, D] is stored as: the scale and
    x / scale are each rounded to 32 bits, then to the format (ties to even)."""
    if fmt == "int8":
        scale = _f32(x.abs().amax(-1, keepdim=True) / torch.full((), 127.0, dtype=torch.float64, device=x.device))
        y = _f32(x / scale)
        return torch.where(scale > 0, torch.round(y).clamp(-127, 127), torch.zeros_like(x)) * scale
    g = head_scale.double()[:, None]
    b = x.unflatten(-1, (-1, 16))
    raw = _f32(b.abs().amax(-1) / _f32(6 * g)).clamp(max=448)
    scale = raw.to(torch.float8_e4m3fn).double()
    step = _f32(scale * g)[..., None]
    y = torch.where(step > 0, _f32(b / step), torch.zeros_like(b))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    mid[1::2] = torch.nextafter(mid[1::2], torch.zeros_like(mid[1::2]))  # these ties go up, to the even code
    value = torch.sign(y) * grid[torch.bucketize(y.abs(), mid)] * scale[..., None] * g[..., None]
    return value.flatten(-2)


def _turn64(x, cs, layout, rounded):
    """Rotated rows; `rounded`: each product and sum rounded to 32 bits, as
    the cache's definition has it ahead of a quantisation."""
    keep = _f32 if rounded else (lambda v: v)
    n = cs.shape[1]
    c, s = (cs[..., i].double()[:, None] for i in (0, 1))
    y = x.double().clone()
    first, second = ((slice(0, n), slice(n, 2 * n)) if layout == "half"
                     else (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first] = keep(keep(a * c) - keep(b * s))
    y[..., second] = keep(keep(b * c) + keep(a * s))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "rope":
        cs = s["table"][s["positions"].long()]
        return tuple(_turn64(s[x], cs, case["layout"], False) for x in "qk")
    fmt, hkv = case["fmt"], case["hkv"]
    if op == "store":
        cs = s["table"][s["positions"].long()]
        return (_turn64(s["q"], cs, case["layout"], False),
                _nearest64(fmt, _turn64(s["k"], cs, case["layout"], True), s["k_scale"]),
                _nearest64(fmt, s["v"].double(), s["v_scale"]))
    if op == "load":
        k, v = (torch.zeros(case["blocks"], hkv, BLOCK, d, dtype=torch.float64, device="cuda")
                for _ in range(2))
        k[s["dst"].long()] = _values64(fmt, d, s["k_pool"][s["src"].long()], s["k_scale"])
        v[s["dst"].long()] = _values64(fmt, d, s["v_pool"][s["src"].long()], s["v_scale"])
        return k, v
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    group = case["hq"] // hkv
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] > 0 else 0
        ids = s["tables"][i, :(n + BLOCK - 1) // BLOCK].long()
        keys, vals = (_values64(fmt, d, s[p][ids], s[g]).transpose(1, 2).flatten(0, 1)[lo:n]
                      for p, g in (("k_pool", "k_scale"), ("v_pool", "v_scale")))
        q = s["q"][i].double().view(hkv, group, d)
        x = torch.einsum("hgd,thd->hgt", q, keys) / math.sqrt(d)
        if s["sink"] is not None:
            x = torch.cat((x, s["sink"].double().view(hkv, group, 1)), -1)
        if x.shape[-1] == 0:
            continue
        lse[i] = torch.logsumexp(x, -1).flatten()
        p = torch.exp(x - lse[i].view(hkv, group, 1))[..., :n - lo]
        out[i] = torch.einsum("hgt,thd->hgd", p, vals).flatten(0, 1)
    return out, lse
