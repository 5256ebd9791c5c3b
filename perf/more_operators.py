"""Timing cases for attention with a score rule and for eviction by attention weight.

Five operators are exercised, each in a plain form (elementary torch, 32-bit
arithmetic) and through the library's entry points (``own`` true):

* ``decode``   one query token per sequence over a paged cache, the logits capped
               by a tanh or given a bias that falls with the distance;
* ``prefill``  ragged prompt chunks over a paged cache under the same rules, with
               a prefix that every one of its positions sees whole;
* ``mass``     the attention weight that each cached key receives, summed over the
               queries and over the heads that share the key;
* ``select``   the keys to keep: the first ones, the last ones, and those of the
               largest weight between them;
* ``compact``  the kept keys' K, V and weight moved together into other blocks.

A query at position p sees key t with the logit
    x = sm_scale q.k,   x -> cap tanh(x / cap),   x -> x - slope[head] |p - t|
if t <= p (or both lie in the prefix) and t > p - window.  Pools are
[blocks][Hkv][16][D], bf16 or e4m3 with a scale per head.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16


# ------------------------------------------------------------------- cases --

def _attn(name, op, **kw):
    case = dict(name=name, op=op, kv="bf16", cap=0.0, slopes=False, sinks=False, window=0, prefix=False)
    case.update(kw)
    return case


def listed():
    return [
        # a decode step of four short sequences: latency
        _attn("decode_small", "decode", seqs=4, lo=17, hi=255, hq=8, hkv=2, d=64, cap=30.0),
        # the decode half of a long ragged batch of a model with capped logits
        _attn("decode_long", "decode", seqs=120, lo=1024, hi=16384, hq=32, hkv=8, d=128, cap=50.0),
        # speculative verify: a few drafted tokens of each of 64 sequences
        _attn("prefill_verify", "prefill", seqs=64, q=8, lo=256, hi=4096, hq=16, hkv=2, d=128, cap=50.0),
        # prompt chunks of 512 tokens behind their cached prefixes, capped logits
        _attn("prefill_prompt", "prefill", seqs=8, q=512, lo=0, hi=8192, hq=32, hkv=8, d=128, cap=50.0),
        # whole prompts of odd lengths: a bidirectional prefix, distance bias, an 8-bit cache
        _attn("prefill_prefix", "prefill", seqs=5, q=777, lo=0, hi=0, hq=64, hkv=8, d=64, kv="e4m3",
              slopes=True, prefix=True),
        # the weights of one decode step, added to the running sums
        _attn("mass_step", "mass", seqs=64, q=1, lo=256, hi=4096, hq=16, hkv=2, d=128, keep=0.98),
        # the prompt's last tokens as observers of the whole cache, before it is thinned
        _attn("mass_window", "mass", seqs=8, q=32, lo=1024, hi=32768, hq=32, hkv=8, d=128, keep=0.0),
        # the weights of whole prompt chunks, capped logits
        _attn("mass_prompt", "mass", seqs=8, q=512, lo=0, hi=8192, hq=32, hkv=8, d=128, cap=50.0, keep=1.0),
        # a batch of caches thinned to 2048 keys a head
        dict(name="select_batch", op="select", seqs=64, lo=1024, hi=16384, hkv=8, budget=2048, first=4,
             recent=64),
        # one very long context, few heads
        dict(name="select_long", op="select", seqs=1, lo=131072, hi=131072, hkv=2, budget=8191, first=16,
             recent=256),
        # two short caches with small 8-bit heads
        dict(name="compact_small", op="compact", seqs=2, lo=150, hi=300, hkv=2, d=64, kv="e4m3", budget=101),
        # the batch's kept rows gathered into fresh blocks
        dict(name="compact_batch", op="compact", seqs=32, lo=4096, hi=16384, hkv=8, d=128, kv="bf16",
             budget=2048),
    ]


def _log(rng, lo, hi):
    lo, hi = max(1, lo), max(1, hi)
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "prefill", "prefill", "mass", "mass", "select", "compact"))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 3, 4, 8))
    kv = rng.choice(("bf16", "e4m3"))
    if op == "select":
        seqs = _log(rng, 1, 128)
        hi = _log(rng, 1, min(131072, 8000000 // (seqs * hkv)))
        budget = _log(rng, 1, max(1, hi))
        first = rng.randint(0, min(budget, 16))
        return dict(op=op, seqs=seqs, lo=max(0, hi // rng.choice((1, 4, 16)) - 1), hi=hi, hkv=hkv,
                    budget=budget, first=first, recent=rng.randint(0, min(budget - first, 256)))
    if op == "compact":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, min(32768, 2000000 // (seqs * hkv)))
        return dict(op=op, seqs=seqs, lo=max(0, hi // rng.choice((1, 4, 16)) - 1), hi=hi, hkv=hkv, d=d, kv=kv,
                    budget=_log(rng, 1, max(1, hi)))
    hq = hkv * rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
    rule = dict(op=op, hq=hq, hkv=hkv, d=d, kv=kv, cap=rng.choice((0.0, 20.0, 50.0)), slopes=rng.random() < 0.4,
                sinks=op != "mass" and rng.random() < 0.3, window=rng.choice((0, 0, 0, _log(rng, 1, 512))),
                prefix=False)
    if op == "decode":
        seqs = _log(rng, 1, 128)
        hi = _log(rng, 1, min(16384, 6000000 // (seqs * hkv)))
        return dict(rule, seqs=seqs, lo=max(1, hi // rng.choice((1, 4, 16))), hi=hi)
    seqs = _log(rng, 1, 32)
    q = 1 if op == "mass" and rng.random() < 0.3 else _log(rng, 1, min(1024, 100000 // (seqs * hq)))
    hi = _log(rng, 1, min(16384, 500000000 // (seqs * hq * q) + 1))
    rule.update(seqs=seqs, q=q, lo=hi // rng.choice((1, 4, 16)), hi=hi, prefix=rng.random() < 0.4)
    return dict(rule, keep=rng.choice((0.0, 0.9, 1.0))) if op == "mass" else rule


# ------------------------------------------------------------------ inputs --

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


def _pool(s, nb, gen, dev):
    """A pool of N(0, 1) rows, and the scale of each head (e4m3)."""
    x = torch.randn(nb, s["hkv"], BLOCK, s["d"], generator=gen, device=dev, dtype=torch.bfloat16)
    if s["kv"] == "bf16":
        return x, None
    scale = (4.2 + 0.6 * torch.rand(s["hkv"], generator=gen, device=dev)) / 448.0
    return (x / scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _sizes(case):
    """The sequences' numbers of queries: those of every seed, so that outputs keep their shapes."""
    q, r = case["q"], random.Random(case["seqs"] * 4096 + case["q"])
    return [q if q % 16 == 0 else r.randint(max(1, q // 4), q) for _ in range(case["seqs"])]


def _stride(case):
    return (max(1, case["hi"] + case.get("q", 0)) + 3) // 4 * 4


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case)
    op, n, hkv = case["op"], case["seqs"], case["hkv"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(n)]
    if op in ("prefill", "mass"):  # lo .. hi tokens are cached, then come the queries' own
        ragged = _sizes(case)
        lens = [a + b for a, b in zip(lens, ragged)]
        cu = [sum(ragged[:i]) for i in range(n + 1)]
        s["qo"], s["max_q"] = ints(cu), max(ragged)
        s["qo_host"], s["lens_host"] = (np.array(v, dtype=np.int32) for v in (cu, lens))
    s["lens"], s["max_len"] = ints(lens), max(1, max(lens))
    if op in ("select", "compact"):
        # weights as sums of softmax rows leave them: few large, many small
        s["mass"] = torch.exp(2.0 * torch.randn(n, hkv, _stride(case), generator=gen, device=dev) - 4.0)
    if op == "select":
        s["kept"] = torch.full((n, hkv, case["budget"]), -1, dtype=torch.int32, device=dev)
        s["kept_lens"] = torch.zeros(n, dtype=torch.int32, device=dev)
        return s
    s["tables"], nb = _tables(lens, dev, rng)
    s["k_pool"], s["k_scale"] = _pool(s, nb, gen, dev)
    if op != "mass":
        s["v_pool"], s["v_scale"] = _pool(s, nb, gen, dev)
    if own:
        s["desc"] = _lib().make_desc(num_q_heads=case.get("hq", hkv), num_kv_heads=hkv, head_dim=case["d"],
                                     num_blocks=nb, kv_dtype=_kind(case["kv"]),
                                     max_blocks_per_seq=s["tables"].shape[1])
    if op == "compact":
        keep = [min(x, case["budget"]) for x in lens]
        # which ones are kept: any subset, ascending
        u = torch.rand(n, hkv, s["mass"].shape[2], generator=gen, device=dev)
        t = torch.arange(u.shape[2], device=dev)
        u = u.masked_fill(t >= s["lens"][:, None, None], 2.0)
        order = torch.sort(u, -1).indices[..., :case["budget"]]
        last = torch.arange(order.shape[2], device=dev) >= ints(keep)[:, None, None]
        order = torch.sort(order.masked_fill(last, 1 << 30), -1).values
        s["kept"] = order.masked_fill(last, -1).int().contiguous()
        s["kept_lens"] = ints(keep)
        s["dst_tables"], _ = _tables(keep, dev, rng)
        dst_nb = n * ((case["budget"] + BLOCK - 1) // BLOCK)
        s["k_dst"], s["v_dst"] = (torch.zeros(dst_nb, hkv, BLOCK, case["d"], dtype=s["k_pool"].dtype, device=dev)
                                  for _ in range(2))
        s["mass_out"] = torch.zeros(n, hkv, case["budget"], device=dev)
        if own:
            s["dst_desc"] = _lib().make_desc(num_q_heads=hkv, num_kv_heads=hkv, head_dim=case["d"],
                                             num_blocks=dst_nb, kv_dtype=_kind(case["kv"]),
                                             max_blocks_per_seq=s["dst_tables"].shape[1])
        return s
    rows = n if op == "decode" else int(s["qo_host"][-1])
    s["q_rows"] = (2.0 * torch.randn(rows, case["hq"], case["d"], generator=gen, device=dev)).bfloat16()
    s["out"] = torch.empty_like(s["q_rows"])
    s["lse"] = torch.empty(rows, case["hq"], device=dev)
    s["slope"] = s["sink"] = s["prefix_lens"] = None
    if case["slopes"]:  # a geometric ladder over the heads
        s["slope"] = 2.0 ** (-8.0 * (1 + torch.arange(case["hq"], device=dev)) / case["hq"])
    if case["sinks"]:
        s["sink"] = torch.randn(case["hq"], generator=gen, device=dev)
    if case["prefix"]:
        s["prefix_lens"] = ints([rng.randint(0, x) for x in lens])
    if op == "mass":
        s["mass"] = torch.rand(n, hkv, _stride(case), generator=gen, device=dev)
        x, _ = _scores(s)
        s["lse"] = _ragged(s, torch.logsumexp(x, -1)).contiguous()
        del x
    if own:
        lib = _lib()
        s["score"] = lib.make_score(1.0 / math.sqrt(case["d"]), cap=case["cap"], slopes=s["slope"],
                                    sinks=s["sink"], window=case["window"], prefix_lens=s["prefix_lens"])
        if op == "decode":
            ws = lib.pkv_decode_workspace_size(s["desc"], n, s["max_len"], window=case["window"])
            s["workspace"] = torch.zeros(max(ws, 256), dtype=torch.uint8, device=dev)
    return s


def _lib():
    import paged_kv_attention_21_gb300 as pkv
    return pkv


def _kind(kv):
    return _lib().KV_BF16 if kv == "bf16" else _lib().KV_FP8_E4M3


# ------------------------------------------------------------- plain forms --

def _rows(pool, scale, tables):
    """fp32 [S][Hkv][keys][D] of the rows that the tables name."""
    x = pool[tables.long().clamp(min=0)].float()
    if scale is not None:
        x = x * scale[:, None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _queries(s):
    """fp32 [S][Q][Hq][D], the queries' positions [S][Q] and which are real."""
    n = s["seqs"]
    if s["op"] == "decode":
        return s["q_rows"].float()[:, None], s["lens"].long()[:, None] - 1, None
    i = torch.arange(s["max_q"], device=s["qo"].device)
    size = (s["qo"][1:] - s["qo"][:-1]).long()[:, None]
    real = i < size
    at = (s["qo"][:n].long()[:, None] + i).clamp(max=s["q_rows"].shape[0] - 1)
    return s["q_rows"][at].float(), s["lens"].long()[:, None] - size + i, real


def _ragged(s, x):
    """[S][Hkv][G][Q] (...) of padded queries -> [rows][Hq] (...)."""
    x = x.flatten(1, 2).transpose(1, 2)
    real = _queries(s)[2]
    return x[:, 0] if real is None else x[real]


def _scores(s):
    """Logits [S][Hkv][G][Q][keys], -inf where a key is not seen, and the seen ones."""
    q, pos, real = _queries(s)
    n, hkv, d = s["seqs"], s["hkv"], s["d"]
    k = _rows(s["k_pool"], s["k_scale"], s["tables"])
    q = q.transpose(1, 2).unflatten(1, (hkv, -1))
    x = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (-1, q.shape[3])) * (1.0 / math.sqrt(d))
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    t = torch.arange(k.shape[2], device=k.device)
    p = pos[..., None]
    if s["slope"] is not None:
        x = x - s["slope"].view(1, hkv, -1, 1, 1) * (p - t).abs()[:, None, None].float()
    hi = pos
    if s["prefix_lens"] is not None:
        hi = torch.maximum(pos, s["prefix_lens"].long()[:, None] - 1)
    seen = (t <= hi[..., None]) & (t < s["lens"].long()[:, None, None])
    if s["window"] > 0:
        seen = seen & (t > p - s["window"])
    if real is not None:
        seen = seen & real[..., None]
    return x.masked_fill(~seen[:, None, None], -math.inf), seen


def _plain_attention(s):
    x, _ = _scores(s)
    m = x.amax(-1, keepdim=True)
    sink = None if s["sink"] is None else s["sink"].view(1, s["hkv"], -1, 1, 1)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - m)
    v = _rows(s["v_pool"], s["v_scale"], s["tables"])
    o = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4])
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return _ragged(s, o).bfloat16(), _ragged(s, (m + torch.log(total))[..., 0])


def _plain_mass(s):
    x, _ = _scores(s)
    n, hkv = s["seqs"], s["hkv"]
    _, pos, real = _queries(s)
    lse = torch.zeros(n, s["max_q"], s["hq"], device=x.device)
    lse[real] = s["lse"]
    lse = lse.transpose(1, 2).unflatten(1, (hkv, -1))[..., None]
    w = torch.where(lse == -math.inf, torch.zeros_like(x), torch.exp(x - lse)).sum((2, 3))
    t = torch.arange(s["mass"].shape[2], device=x.device)
    w = torch.nn.functional.pad(w, (0, max(0, t.numel() - w.shape[2])))[..., :t.numel()]
    size = (s["qo"][1:] - s["qo"][:-1])[:, None, None]
    lens = s["lens"][:, None, None]
    old = s["mass"]
    kept = torch.where((t < lens - size) & torch.full((), s["keep"] != 0.0, device=x.device), s["keep"] * old,
                       torch.zeros_like(old))
    s["mass"] = torch.where(t < lens, kept + w, old)
    return s["mass"]


def _plain_select(s):
    lens = s["lens"].long()[:, None, None]
    n_keep = lens.clamp(max=s["budget"])
    t = torch.arange(s["mass"].shape[2], device=lens.device)
    all_kept = lens <= s["budget"]
    ends = (t < s["first"]) | (t >= lens - s["recent"]) | all_kept
    middle = ~ends & (t < lens)
    order = torch.sort(s["mass"].masked_fill(~middle, -math.inf), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order))
    keep = (t < lens) & (ends | (middle & (rank < s["budget"] - s["first"] - s["recent"])))
    slot = torch.cumsum(keep, -1) - 1
    slot = torch.where(keep, slot, torch.full_like(slot, s["budget"]))
    kept = torch.cat((s["kept"], s["kept"][..., :1]), -1)
    kept.scatter_(-1, slot, t.int().expand_as(slot).contiguous())
    return kept[..., :-1].contiguous(), n_keep[:, 0, 0].int()


def _plain_compact(s):
    kept = s["kept"].long()
    j = torch.arange(kept.shape[2], device=kept.device)
    live = (j < s["kept_lens"].long()[:, None, None]).expand_as(kept)
    seq, head, slot = torch.nonzero(live, as_tuple=True)
    r = kept[live]
    src = s["tables"].long()[seq, r // BLOCK]
    dst = s["dst_tables"].long()[seq, slot // BLOCK]
    raw = torch.uint8 if s["kv"] == "e4m3" else torch.bfloat16
    for a, b in (("k_pool", "k_dst"), ("v_pool", "v_dst")):
        s[b].view(raw)[dst, head, slot % BLOCK] = s[a].view(raw)[src, head, r % BLOCK]
    s["mass_out"][seq, head, slot] = s["mass"][seq, head, r]
    return s["k_dst"], s["v_dst"], s["mass_out"]


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "mass":
        return _plain_mass(s)
    if op == "select":
        return _plain_select(s)
    if op == "compact":
        return _plain_compact(s)
    return _plain_attention(s)


def _own(s):
    lib, op = _lib(), s["op"]
    if op == "decode":
        lib.pkv_score_decode(s["desc"], s["score"], s["q_rows"], s["k_pool"], s["v_pool"], s["tables"],
                             s["lens"], s["max_len"], s["out"], s["lse"], s["workspace"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    if op == "prefill":
        lib.pkv_score_prefill(s["desc"], s["score"], s["q_rows"], s["qo"], s["k_pool"], s["v_pool"], s["tables"],
                              s["lens"], s["out"], s["lse"], qo_indptr_host=s["qo_host"],
                              kv_lens_host=s["lens_host"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    if op == "mass":
        lib.pkv_score_mass(s["desc"], s["score"], s["q_rows"], s["qo"], s["k_pool"], s["tables"], s["lens"],
                           s["max_len"], s["lse"], s["mass"], keep=s["keep"], max_q_len=s["max_q"],
                           k_scale=s["k_scale"])
        return s["mass"]
    if op == "select":
        lib.pkv_evict_select(s["mass"], s["lens"], s["max_len"], s["budget"], s["first"], s["recent"], s["kept"],
                             s["kept_lens"])
        return s["kept"], s["kept_lens"]
    lib.pkv_evict_compact(s["desc"], s["k_pool"], s["v_pool"], s["tables"], s["kept"], s["kept_lens"],
                          dst_desc=s["dst_desc"], k_dst=s["k_dst"], v_dst=s["v_dst"], dst_tables=s["dst_tables"],
                          mass=s["mass"], mass_out=s["mass_out"])
    return s["k_dst"], s["v_dst"], s["mass_out"]


# ------------------------------------------------------------------- costs --

def work(case):
    op, n, hkv = case["op"], case["seqs"], case["hkv"]
    mean = (case["lo"] + case["hi"]) / 2.0
    if op == "select":
        kept = min(mean, case["budget"])
        return dict(bytes=4 * n * (hkv * (mean + kept) + 2), flops=n * hkv * mean)
    if op == "compact":
        kept = min(mean, case["budget"])
        row = case["d"] * (2 if case["kv"] == "bf16" else 1)
        return dict(bytes=n * hkv * kept * (4 * row + 4 + 8), flops=0)
    elem, d, hq = (2 if case["kv"] == "bf16" else 1), case["d"], case["hq"]
    size = 1 if op == "decode" else sum(_sizes(case)) / n
    cached = mean - 1 if op == "decode" else mean
    keys = cached + size
    pairs = size * cached + size * (size + 1) / 2.0
    if case["prefix"]:  # half the keys are the prefix, on average, and its positions see all of it
        pairs += size * size / 6.0 if cached == 0 else 0.0
    if case["window"] > 0:
        keys = min(keys, case["window"] + size - 1)
        pairs = min(pairs, size * case["window"])
    if op == "mass":
        return dict(bytes=n * (hkv * keys * (d * elem + (8 if case["keep"] else 4)) + size * hq * (2 * d + 4)),
                    flops=2 * n * pairs * hq * d)
    return dict(bytes=n * (hkv * keys * 2 * d * elem + size * hq * (4 * d + 4)), flops=4 * n * pairs * hq * d)


# ------------------------------------------------------ 64-bit definitions --

def _keys64(s, pool, scale, i):
    """The first lens[i] rows of sequence i, [Hkv][keys][D] in 64 bits."""
    n = int(s["lens"][i])
    ids = s["tables"][i, :(n + BLOCK - 1) // BLOCK].long()
    x = s[pool][ids].float().double()
    if s[scale] is not None:
        x = x * s[scale].double()[None, :, None, None]
    return torch.cat(tuple(x), 1)[:, :n] if len(ids) else x.new_zeros(s["hkv"], 0, s["d"])


def _logits64(s, i, a, b):
    """Logits [Hq][b - a][keys] of query rows a .. b of sequence i."""
    n, group = int(s["lens"][i]), s["hq"] // s["hkv"]
    k = _keys64(s, "k_pool", "k_scale", i).repeat_interleave(group, 0)
    x = torch.einsum("qhd,htd->hqt", s["q_rows"][a:b].double(), k) / math.sqrt(s["d"])
    if s["cap"]:
        x = torch.tanh(x / s["cap"]) * s["cap"]
    p = torch.arange(n - (b - a), n, device=x.device)[:, None]
    t = torch.arange(n, device=x.device)[None]
    if s["slope"] is not None:
        x = x - s["slope"].double()[:, None, None] * torch.abs(p - t).double()
    hidden = t > p
    if s["prefix_lens"] is not None:
        m = int(s["prefix_lens"][i])
        hidden &= ~((t < m) & (p < m))
    if s["window"] > 0:
        hidden |= p - t >= s["window"]
    return torch.where(hidden, torch.full_like(x, -math.inf), x)


def _select64(s):
    kept, lens = s["kept"].cpu(), []
    for i, n in enumerate(s["lens"].tolist()):
        lens.append(min(n, s["budget"]))
        for h in range(s["hkv"]):
            pick = list(range(n))
            if n > s["budget"]:
                head, tail = pick[:s["first"]], pick[n - s["recent"]:]
                row = s["mass"][i, h, s["first"]:n - s["recent"]].double().cpu().numpy()
                best = (-row).argsort(kind="stable")[:s["budget"] - s["first"] - s["recent"]]
                pick = head + sorted((best + s["first"]).tolist()) + tail
            kept[i, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return kept, torch.tensor(lens, dtype=torch.int32)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return _select64(s)
    if op == "compact":
        outs = [torch.zeros(s[b].shape, dtype=torch.float64, device="cuda") for b in ("k_dst", "v_dst")]
        mass = s["mass_out"].double()
        for i, n in enumerate(s["kept_lens"].tolist()):
            at = s["kept"][i, :, :n].long()
            for pool, out in zip(("k_pool", "v_pool"), outs):
                ids = s["tables"][i, :(int(s["lens"][i]) + BLOCK - 1) // BLOCK].long()
                rows = s[pool][ids].float().double().transpose(0, 1).flatten(1, 2)
                rows = torch.gather(rows, 1, at[..., None].expand(-1, -1, case["d"]))
                for j in range(0, n, BLOCK):
                    part = rows[:, j:j + BLOCK]
                    out[int(s["dst_tables"][i, j // BLOCK]), :, :part.shape[1]] = part
            mass[i, :, :n] = torch.gather(s["mass"][i].double(), 1, at)
        return outs[0], outs[1], mass
    group = case["hq"] // case["hkv"]
    if op == "mass":
        mass = s["mass"].double()
        for i in range(case["seqs"]):
            a, b, n = (int(x) for x in (s["qo_host"][i], s["qo_host"][i + 1], s["lens_host"][i]))
            w = torch.exp(_logits64(s, i, a, b) - s["lse"][a:b].double().t()[..., None])
            mass[i, :, :n - (b - a)] *= case["keep"]
            mass[i, :, n - (b - a):n] = 0.0
            mass[i, :, :n] += w.sum(1).view(case["hkv"], group, n).sum(1)
        return mass
    out = torch.zeros(s["q_rows"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q_rows"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i in range(case["seqs"]):
        a, b = (i, i + 1) if op == "decode" else s["qo_host"][i:i + 2].tolist()
        x = _logits64(s, i, a, b)
        if s["sink"] is not None:
            x = torch.cat((x, s["sink"].double()[:, None, None].expand(-1, b - a, 1)), -1)
        z = torch.logsumexp(x, -1)
        w = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[..., None])
        v = _keys64(s, "v_pool", "v_scale", i).repeat_interleave(group, 0)
        out[a:b] = torch.einsum("hqt,htd->qhd", w[..., :v.shape[1]], v)
        lse[a:b] = z.t()
    return out, lse
