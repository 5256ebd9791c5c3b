"""Attention under a score rule, and the weight that each key receives, on the GPU against
64 bits, within bounds added up from the roundings."""
import numpy as np
import pytest
import torch

from _score import Paged, Rule, close
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu


def decode(p, r, q, chunk=0, max_len=None, stream=None, out=None, ws=None):
    n = len(p.lens)
    max_len = max_len or max(1, max(p.lens))
    out = torch.full_like(q, float("nan")) if out is None else out
    lse = torch.full((n, p.hq), float("nan"), device=q.device)
    size = pkv.pkv_decode_workspace_size(p.desc, n, max_len, r.window, chunk)
    ws = torch.zeros(max(256, size), dtype=torch.uint8, device=q.device) if ws is None else ws
    pkv.pkv_score_decode(p.desc, r.score, q, p.k_pool, p.v_pool, p.t, p.lens_t, max_len, out, lse, ws,
                         chunk_blocks=chunk, stream=stream, **p.scales)
    return out, lse


def check_decode(p, r, q64, out, lse):
    assert pkv.pkv_device_errors() == 0
    for s, n in enumerate(p.lens):
        o, z, bo, bz = r.attend(p, s, q64[s:s + 1], [n - 1])
        close(out[s:s + 1], o, bo, "out of sequence %d" % s)
        close(lse[s:s + 1], z, bz, "lse of sequence %d" % s)


LENS = [1, 16, 0, 17, 255, 64, 700, 2]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (4, 4, 128), (16, 1, 128), (15, 3, 64), (12, 1, 128)])
@pytest.mark.parametrize("rule", [dict(cap=50.0), dict(slopes=1.0), dict(cap=5.0, slopes=0.3, sinks=True),
                                  dict(window=37, cap=20.0), dict(slopes=-0.02), dict(sinks=True, window=1)])
def test_decode_against_64_bits(hq, hkv, d, kv, rule):
    p = Paged(LENS, hq, hkv, d, kv, seed=hq + d)
    r = Rule(d, hq, len(LENS), **rule)
    q, q64 = p.queries(len(LENS))
    check_decode(p, r, q64, *decode(p, r, q))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("chunk", [1, 2, 12, 23, 44])
def test_decode_merges_chunks(kv, chunk):
    """One chunk, clusters of two to four, and more through the workspace, left zeroed."""
    p = Paged(LENS, 8, 2, 128, kv, seed=chunk)
    r = Rule(128, 8, len(LENS), cap=8.0, slopes=0.1, sinks=True)
    q, q64 = p.queries(len(LENS), 4.0)
    check_decode(p, r, q64, *decode(p, r, q, chunk=chunk))


@pytest.mark.parametrize("cap,size", [(0.5, 30.0), (1e-3, 1.0), (1e4, 3.0), (30.0, 300.0)])
def test_decode_caps_far_below_and_above_the_logits(cap, size):
    p = Paged([333, 20], 8, 8, 64, seed=3)
    r = Rule(64, 8, 2, cap=cap)
    q, q64 = p.queries(2, size)
    check_decode(p, r, q64, *decode(p, r, q))


def test_decode_over_a_ring():
    for ring, window, lens in ((4, 40, [1, 39, 64, 500, 3000]), (9, 128, [129, 1000, 5])):
        p = Paged(lens, 8, 2, 64, seed=ring, ring=ring, window=window)
        r = Rule(64, 8, len(lens), cap=10.0, slopes=0.5, window=window, sinks=True)
        q, q64 = p.queries(len(lens))
        check_decode(p, r, q64, *decode(p, r, q))


def test_decode_captured_replayed_and_on_another_stream():
    p = Paged(LENS, 16, 2, 128, seed=9)
    r = Rule(128, 16, len(LENS), cap=20.0, slopes=0.2)
    q, q64 = p.queries(len(LENS))
    want, want_lse = decode(p, r, q, chunk=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, got_lse = decode(p, r, q, chunk=3)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    out = torch.empty_like(q)
    ws = torch.zeros(max(256, pkv.pkv_decode_workspace_size(p.desc, len(LENS), 700, 0, 3)), dtype=torch.uint8,
                     device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        decode(p, r, q, chunk=3, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ------------------------------------------------------------------ prefill --

def problem(p, q_lens):
    qo = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q, q64 = p.queries(int(qo[-1]))
    return qo, torch.from_numpy(qo).to(p.device), q, q64


def prefill(p, r, q, qo, qo_t, hosts=True):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=q.device)
    pkv.pkv_score_prefill(p.desc, r.score, q, qo_t, p.k_pool, p.v_pool, p.t, p.lens_t, out, lse,
                          qo_indptr_host=qo if hosts else None, kv_lens_host=p.lens if hosts else None,
                          causal=r.causal, **p.scales)
    return out, lse


def check_prefill(p, r, q64, qo, out, lse):
    assert pkv.pkv_device_errors() == 0
    for s, n in enumerate(p.lens):
        a, b = int(qo[s]), int(qo[s + 1])
        o, z, bo, bz = r.attend(p, s, q64[a:b], np.arange(n - (b - a), n))
        close(out[a:b], o, bo, "out of sequence %d" % s)
        close(lse[a:b], z, bz, "lse of sequence %d" % s)


RULES = [dict(cap=50.0), dict(slopes=1.0, prefix=[0, 40, 9, 1000, 33, 1]), dict(cap=5.0, slopes=0.3, sinks=True),
         dict(window=37, cap=20.0, prefix=[-5, 130, 300, 17, 90, 0]), dict(causal=False, slopes=0.05),
         dict(causal=False, window=20, sinks=True), dict(cap=3.0, prefix=[400, 400, 400, 400, 400, 400])]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (3, 3, 128), (16, 1, 128), (6, 2, 128)])
@pytest.mark.parametrize("rule", RULES)
def test_prefill_against_64_bits(hq, hkv, d, kv, rule):
    q_lens = [1, 70, 200, 0, 33, 129]
    p = Paged([1, 130, 300, 17, 33, 513], hq, hkv, d, kv, seed=hq + d)
    r = Rule(d, hq, 6, **rule)
    qo, qo_t, q, q64 = problem(p, q_lens)
    check_prefill(p, r, q64, qo, *prefill(p, r, q, qo, qo_t))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (16, 1, 128), (5, 5, 128)])
@pytest.mark.parametrize("rule", RULES)
def test_few_queries_against_64_bits(hq, hkv, d, kv, rule):
    """At most 64 query rows per sequence: one and several chunks of keys."""
    for lens, q_lens in (([1, 130, 300, 17, 33, 513], [1, 4, 3, 0, 2, 4]), ([3, 40, 30, 17, 20, 1], [3, 1, 2, 2, 0, 1])):
        p = Paged(lens, hq, hkv, d, kv, seed=hq + d)
        r = Rule(d, hq, 6, **rule)
        qo, qo_t, q, q64 = problem(p, q_lens)
        check_prefill(p, r, q64, qo, *prefill(p, r, q, qo, qo_t))


def test_prefill_without_host_arrays_is_the_same():
    p = Paged([50, 300], 8, 2, 128, seed=5)
    r = Rule(128, 8, 2, cap=9.0, slopes=0.1, prefix=[20, 100])
    qo, qo_t, q, q64 = problem(p, [50, 90])
    want, got = prefill(p, r, q, qo, qo_t), prefill(p, r, q, qo, qo_t, hosts=False)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_prefill_reads_no_block_below_the_windows():
    """Their table entries name no block, as an engine leaves them that has freed these."""
    p = Paged([700, 650], 8, 2, 128, seed=6)
    r = Rule(128, 8, 2, cap=20.0, window=50)
    for q_lens in ([100, 40], [3, 2]):
        qo, qo_t, q, q64 = problem(p, q_lens)
        p.t = torch.from_numpy(p.tables).to("cuda")
        for s, (n, m) in enumerate(zip(p.lens, q_lens)):
            p.t[s, :max(0, n - m - 49) // 16] = -1
        check_prefill(p, r, q64, qo, *prefill(p, r, q, qo, qo_t))


# ------------------------------------------------------------------- weights --

def mass_of(p, r, q, qo_t, lse, start, keep, max_q, max_len=None):
    got = start.clone()
    pkv.pkv_score_mass(p.desc, r.score, q, qo_t, p.k_pool, p.t, p.lens_t, max_len or max(1, max(p.lens)), lse, got,
                       keep=keep, max_q_len=max_q, causal=r.causal, k_scale=p.scales["k_scale"])
    return got


def check_mass(p, r, q64, qo, lse, start, keep, got):
    assert pkv.pkv_device_errors() == 0
    z = lse.cpu().numpy()
    got, start = got.cpu().numpy().astype(np.float64), start.cpu().numpy().astype(np.float64)
    for s, n in enumerate(p.lens):
        a, b = int(qo[s]), int(qo[s + 1])
        want, bound = r.mass(p, s, q64[a:b], np.arange(n - (b - a), n), z[a:b])
        if keep:
            own = n - (b - a)
            want[:, :own] += keep * start[s, :, :own]
            bound[:, :own] += 3 * 2.0 ** -24 * np.abs(want[:, :own])
        # the sum's own rounding: one half step a query row
        close(got[s, :, :n], want, bound + 2.0 ** -24 * (b - a + 8) * want + 1e-38, "weights of sequence %d" % s)
        assert np.array_equal(got[s, :, n:], start[s, :, n:], equal_nan=True), "behind sequence %d" % s


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (3, 3, 128), (16, 1, 128), (10, 2, 64)])
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("q_lens", [[1, 70, 200, 0, 33, 129], [1, 2, 3, 0, 4, 2], [1, 17, 32, 17, 20, 1]])
def test_mass_against_64_bits(hq, hkv, d, kv, rule, q_lens):
    p = Paged([1, 130, 300, 17, 33, 513], hq, hkv, d, kv, seed=hq + d)
    r = Rule(d, hq, 6, **dict(rule, sinks=False))
    qo, qo_t, q, q64 = problem(p, q_lens)
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    out = torch.empty_like(q)
    pkv.pkv_score_prefill(p.desc, r.score, q, qo_t, p.k_pool, p.v_pool, p.t, p.lens_t, out, lse, causal=r.causal,
                          **p.scales)
    for keep in (0.0, 0.75, 1.0):
        start = torch.rand(6, hkv, 520, device="cuda")
        if not keep:
            start[:] = float("nan")  # not read
        for s in range(6):  # what the call's own keys held counts as 0
            start[s, :, p.lens[s] - q_lens[s]:p.lens[s]] = float("nan")
        got = mass_of(p, r, q, qo_t, lse, start, keep, max(q_lens))
        check_mass(p, r, q64, qo, lse, start, keep, got)
        assert torch.equal(mass_of(p, r, q, qo_t, lse, start, keep, max(q_lens)).view(torch.int32), got.view(torch.int32))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (16, 1, 128), (7, 7, 128), (12, 1, 64)])
def test_mass_of_a_decode_step(hq, hkv, d, kv):
    p = Paged(LENS, hq, hkv, d, kv, seed=hq)
    r = Rule(d, hq, len(LENS), cap=20.0, slopes=0.1, sinks=True)
    q, q64 = p.queries(len(LENS))
    _, lse = decode(p, r, q)
    lse[4] = float("-inf")  # a row that saw nothing adds nothing
    lens = list(p.lens)
    start = torch.rand(len(LENS), hkv, 703, device="cuda")
    got = mass_of(p, r, q, None, lse, start, 0.5, 1)
    z = lse.cpu().numpy()
    got, start = got.cpu().numpy().astype(np.float64), start.cpu().numpy().astype(np.float64)
    for s, n in enumerate(lens):
        assert np.array_equal(got[s, :, max(n, 0):], start[s, :, max(n, 0):])
        if n <= 0:
            continue
        want, bound = r.mass(p, s, q64[s:s + 1], [n - 1], z[s:s + 1])
        want[:, :n - 1] += 0.5 * start[s, :, :n - 1]
        close(got[s, :, :n], want, bound + 8 * 2.0 ** -24 * want + 1e-38)
    assert pkv.pkv_device_errors() == 0


def test_mass_flags_what_it_cannot_read():
    p = Paged([100, 60], 4, 2, 64, seed=2)
    r = Rule(64, 4, 2)
    q, _ = p.queries(2)
    lse = torch.zeros(2, 4, device="cuda")
    start = torch.rand(2, 2, 128, device="cuda")
    good = mass_of(p, r, q, None, lse, start, 1.0, 1)
    assert pkv.pkv_device_errors() == 0
    p.t[0, 2] = 10 ** 6  # a bad block: its keys' weights stay, the others' do not change
    got = mass_of(p, r, q, None, lse, start, 1.0, 1)
    assert pkv.pkv_device_errors() == pkv.DEVERR_BLOCK_ID
    assert torch.equal(got[0, :, 32:48], start[0, :, 32:48])
    good[0, :, 32:48] = got[0, :, 32:48]
    assert torch.equal(got, good)
    mass_of(p, r, q, None, lse, start, 1.0, 1, max_len=90)
    assert pkv.pkv_device_errors() == pkv.DEVERR_LENGTH | pkv.DEVERR_BLOCK_ID
    bad = torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda")
    got = mass_of(p, r, q, bad, lse, start, 1.0, 3)
    assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION
    assert torch.equal(got, start)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,q_max", [(8, 2, 64, 32), (8, 2, 128, 30), (12, 4, 128, 80), (2, 2, 64, 200)])
def test_mass_of_many_ragged_sequences(kv, hq, hkv, d, q_max):
    """Every CTA goes from tile to tile, head to head and sequence to sequence: many short
    sequences (one to four key tiles at a time), a few long ones, some without queries."""
    rng = np.random.default_rng(hq + q_max)
    q_lens = [int(x) for x in rng.integers(0, q_max + 1, 70)]
    q_lens[3] = q_max
    lens = [m + int(x) for m, x in zip(q_lens, np.where(rng.random(70) < 0.1, rng.integers(0, 3000, 70), rng.integers(0, 700, 70)))]
    p = Paged(lens, hq, hkv, d, kv, seed=hq)
    r = Rule(d, hq, 70, cap=30.0)
    qo, qo_t, q, q64 = problem(p, q_lens)
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    pkv.pkv_score_prefill(p.desc, r.score, q, qo_t, p.k_pool, p.v_pool, p.t, p.lens_t, torch.empty_like(q), lse, **p.scales)
    start = torch.rand(70, hkv, max(lens), device="cuda")
    got = mass_of(p, r, q, qo_t, lse, start, 1.0, q_max)
    check_mass(p, r, q64, qo, lse, start, 1.0, got)


def test_mass_counts_at_most_max_q_len():
    """More queries than the bound: the first ones count, the flag says so."""
    p = Paged([90, 200], 4, 2, 64, seed=12)
    r = Rule(64, 4, 2)
    for q_lens, top in (([3, 6], 4), ([60, 90], 70)):
        qo, qo_t, q, q64 = problem(p, q_lens)
        lse = torch.rand(q.shape[:2], device="cuda") + 4
        start = torch.rand(2, 2, 200, device="cuda")
        got = mass_of(p, r, q, qo_t, lse, start, 1.0, top).cpu().numpy().astype(np.float64)
        assert pkv.pkv_device_errors() == pkv.DEVERR_LENGTH
        for s, n in enumerate(p.lens):
            a, m = int(qo[s]), min(q_lens[s], top)
            pos = np.arange(n - q_lens[s], n)[:m]
            want, bound = r.mass(p, s, q64[a:a + m], pos, lse[a:a + m].cpu().numpy())
            own = n - q_lens[s]
            want[:, :own] += start[s, :, :own].cpu().numpy()
            close(got[s, :, :n], want, bound + 2.0 ** -24 * (m + 8) * want + 1e-38)


def test_mass_refuses_on_the_device_more_queries_than_keys():
    p = Paged([3, 40], 4, 2, 64, seed=13)
    r = Rule(64, 4, 2)
    qo_t = torch.tensor([0, 5, 7], dtype=torch.int32, device="cuda")
    q, _ = p.queries(7)
    start = torch.rand(2, 2, 40, device="cuda")
    for top in (5, 40):
        got = mass_of(p, r, q, qo_t, torch.zeros(7, 4, device="cuda"), start, 1.0, top)
        assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION
        assert torch.equal(got[0], start[0]) and not torch.equal(got[1], start[1])


def test_infinite_keys_that_no_query_sees_change_nothing():
    """Values no query may look at: K and V rows behind the window, and behind a query's
    position where the keys of the same tile are K alone."""
    p = Paged([400], 8, 2, 64, seed=14)
    r = Rule(64, 8, 1, cap=12.0, window=100)
    q, q64 = p.queries(1)
    lse0 = decode(p, r, q)
    mass0 = mass_of(p, r, q, None, lse0[1], torch.zeros(1, 2, 400, device="cuda"), 0.0, 1)
    for bad in (float("inf"), float("-inf"), float("nan"), 3e38, -3e38):
        for t in (0, 150, 299):
            for pool in (p.k_pool, p.v_pool):
                pool[p.tables[0, t // 16], :, t % 16] = bad
        out, lse = decode(p, r, q)
        assert torch.equal(out, lse0[0]) and torch.equal(lse, lse0[1])
        got = mass_of(p, r, q, None, lse, torch.zeros(1, 2, 400, device="cuda"), 0.0, 1)
        assert torch.equal(got, mass0)
    # the observers of a prompt's end: keys past a query's position are masked, not multiplied
    p = Paged([256], 2, 1, 64, seed=15)
    r = Rule(64, 2, 1)
    for m in (8, 100):
        q, q64 = p.queries(m)
        qo_t = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        lse = torch.full((m, 2), 5.0, device="cuda")
        lse[-1] = float("-inf")  # the only query that sees the last key counts for nothing
        start = torch.zeros(1, 1, 256, device="cuda")
        want = mass_of(p, r, q, qo_t, lse, start, 0.0, m)
        kept = p.k_pool.clone()
        p.k_pool[p.tables[0, 15], :, 15] = 1e30
        got = mass_of(p, r, q, qo_t, lse, start, 0.0, m)
        assert torch.equal(got[..., :255], want[..., :255])
        p.k_pool.copy_(kept)


def test_pools_past_32_bits():
    """Blocks whose bytes lie past 2^32 in pools of 4.6 GB."""
    p = Paged([100, 300], 32, 8, 128, seed=16)
    far = 140000
    k, v = (torch.zeros(far + p.nb, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[far:], v[far:] = p.k_pool, p.v_pool
    p.k_pool, p.v_pool, p.nb = k, v, far + p.nb
    p.tables = np.where(p.tables >= 0, p.tables + far, -1).astype(np.int32)
    p.t, p.desc = torch.from_numpy(p.tables).to("cuda"), p.make_desc()
    r = Rule(128, 32, 2, cap=20.0)
    q, q64 = p.queries(2)
    out, lse = decode(p, r, q)
    check_decode(p, r, q64, out, lse)
    for q_lens in ([3, 5], [60, 90]):
        qo, qo_t, q, q64 = problem(p, q_lens)
        out, lse = prefill(p, r, q, qo, qo_t)
        check_prefill(p, r, q64, qo, out, lse)
        start = torch.rand(2, 8, 300, device="cuda")
        check_mass(p, r, q64, qo, lse, start, 1.0, mass_of(p, r, q, qo_t, lse, start, 1.0, max(q_lens)))
