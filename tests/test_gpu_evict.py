"""Eviction on the GPU: which keys are kept, their rows moved, and a cache served through all of it."""
import numpy as np
import pytest
import torch

from _score import Paged, Rule, close, select
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run_select(mass, lens, budget, first, recent, max_len=None, width=None):
    n, h, stride = mass.shape
    width = width or budget
    kept = torch.full((n, h, width), -7, dtype=torch.int32, device=DEV)
    kept_lens = torch.full((n,), -7, dtype=torch.int32, device=DEV)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pkv.pkv_evict_select(torch.from_numpy(mass).to(DEV), lens_t, max_len or stride, budget, first, recent, kept,
                         kept_lens)
    return kept.cpu().numpy(), kept_lens.cpu().numpy()


def check_select(mass, lens, budget, first, recent, **kw):
    kept, kept_lens = run_select(mass, lens, budget, first, recent, **kw)
    assert pkv.pkv_device_errors() == 0
    for s, n in enumerate(lens):
        c = min(max(n, 0), budget)
        assert kept_lens[s] == c
        for h in range(mass.shape[1]):
            want = select(mass[s, h], n, budget, first, recent)
            assert np.array_equal(kept[s, h, :c], want), (s, h, n)
            assert (kept[s, h, c:] == -7).all()


@pytest.mark.parametrize("budget,first,recent", [(1, 0, 0), (1, 1, 0), (5, 2, 3), (64, 4, 16), (100, 0, 100),
                                                 (999, 16, 64), (4096, 0, 1)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_select_is_the_definition(budget, first, recent, kind):
    rng = np.random.default_rng(budget)
    lens = [0, 1, 7, 65, 1000, 1024, 5000, 33, -3, 2047]
    mass = np.exp(3 * rng.standard_normal((len(lens), 3, 5003))).astype(np.float32)
    if kind == "ties":
        mass = np.round(mass).astype(np.float32)  # few values, many zeros
    if kind == "odd":
        odd = np.array([0.0, -0.0, np.nan, np.inf, -np.inf, -1.0, 1e-45, -1e-45, 3e38, -3e38, -np.nan], np.float32)
        mass = np.where(rng.random(mass.shape) < 0.5, odd[rng.integers(0, len(odd), mass.shape)], mass)
    check_select(mass, lens, budget, first, recent)


def test_select_of_equal_weights_keeps_the_first_ones():
    mass = np.full((2, 1, 300000), 0.25, np.float32)
    check_select(mass, [300000, 299999], 1000, 10, 20)
    check_select(np.full((1, 2, 40), np.nan, np.float32), [40], 11, 1, 2)


@pytest.mark.parametrize("n,heads,budget", [(131072, 2, 8191), (262147, 1, 100000), (70001, 5, 70000), (49153, 3, 1)])
def test_select_of_long_rows(n, heads, budget):
    rng = np.random.default_rng(n)
    mass = np.exp(2 * rng.standard_normal((1, heads, n + 1))).astype(np.float32)
    check_select(mass, [n], budget, min(3, budget // 2), min(100, budget // 2))


def test_select_at_more_sequences_and_cut_lengths():
    rng = np.random.default_rng(8)
    lens = list(rng.integers(0, 200, 700))
    mass = rng.random((700, 2, 200)).astype(np.float32)
    check_select(mass, lens, 50, 3, 7, max_len=200)
    kept, kept_lens = run_select(mass[:1], [200], 500, 0, 0, max_len=150, width=150)  # a length beyond the bound
    assert pkv.pkv_device_errors() == pkv.DEVERR_LENGTH
    assert kept_lens[0] == 150 and np.array_equal(kept[0, 0], np.arange(150))


# -------------------------------------------------------------- compaction --

def ascending(rng, lens, heads, width):
    """Random kept positions: [s][h][width], their numbers at most `width`."""
    kept = np.full((len(lens), heads, width), -1, np.int32)
    counts = np.array([rng.integers(0, min(n, width) + 1) for n in lens], np.int32)
    for s, n in enumerate(lens):
        for h in range(heads):
            kept[s, h, :counts[s]] = np.sort(rng.permutation(n)[:counts[s]])
    return kept, counts


def rows_of(pool, tables, s, h, at):
    """The bytes of rows `at` of (s, h) in a pool."""
    raw = pool.view(torch.uint8 if pool.element_size() == 1 else torch.int16).cpu().numpy()
    return np.stack([raw[tables[s, t // 16], h, t % 16] for t in at]) if len(at) else np.zeros((0,) + raw.shape[3:], raw.dtype)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
@pytest.mark.parametrize("heads,lens,budget", [
    (35, [16384, 16383, 2049], 2048), (35, [6145, 10241, 14336], 5000), (70, [4097, 8193], 4000),  # a CTA a row
    (1, [8195, 16384], 8000), (3, [140001], 70000), (1, [400003], 3), (1, [420000], 419990)])
def test_select_at_every_width(heads, lens, budget, kind):
    """One to eight fours a thread, several rounds of them, parts that shared memory does not hold;
    with weights of which few or none differ."""
    rng = np.random.default_rng(heads + budget)
    mass = np.exp(2 * rng.standard_normal((len(lens), heads, max(lens) + 3))).astype(np.float32)
    if kind == "ties":
        mass = np.minimum(np.round(mass), 3).astype(np.float32)
    elif kind == "equal":
        mass[:] = 0.25
    check_select(mass, lens, budget, 2, min(70, budget - 2))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_compaction_moves_the_rows(kv, d, in_place, weights):
    rng = np.random.default_rng(d)
    lens = [0, 1, 16, 100, 333, 1500, 40]
    p = Paged(lens, 6, 3, d, kv, seed=4)
    kept, counts = ascending(rng, lens, 3, 700)
    mass = torch.rand(len(lens), 3, 1501, device=DEV)
    args = dict(mass=mass.clone(), mass_out=None)
    if weights and not in_place:
        args["mass_out"] = torch.full((len(lens), 3, 701), -7.0, device=DEV)
    if weights and in_place:
        args["mass_out"] = args["mass"]
    if not weights:
        args = {}
    src = [x.clone() for x in (p.k_pool, p.v_pool)]
    tables = p.tables
    if in_place:
        dst = (p.k_pool, p.v_pool)
        pkv.pkv_evict_compact(p.desc, p.k_pool, p.v_pool, p.t, torch.from_numpy(kept).to(DEV),
                              torch.from_numpy(counts).to(DEV), **args)
    else:
        nb = int(sum((c + 15) // 16 for c in counts)) + 2
        ids = list(rng.permutation(nb))
        tables = np.full((len(lens), 45), -1, np.int32)
        for s, c in enumerate(counts):
            for b in range((c + 15) // 16):
                tables[s, b] = ids.pop()
        dst = [torch.zeros(nb, 3, 16, d, dtype=x.dtype, device=DEV) for x in src]
        pkv.pkv_evict_compact(p.desc, p.k_pool, p.v_pool, p.t, torch.from_numpy(kept).to(DEV),
                              torch.from_numpy(counts).to(DEV), dst_desc=p.make_desc(num_blocks=nb, max_blocks_per_seq=45),
                              k_dst=dst[0], v_dst=dst[1], dst_tables=torch.from_numpy(tables).to(DEV), **args)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(src, (p.k_pool, p.v_pool)))
    assert pkv.pkv_device_errors() == 0
    for s, c in enumerate(counts):
        for h in range(3):
            for a, b in zip(src, dst):
                assert np.array_equal(rows_of(b, tables, s, h, range(c)), rows_of(a, p.tables, s, h, kept[s, h, :c]))
                if in_place:  # rows behind the kept ones stay
                    tail = range(c, lens[s])
                    assert np.array_equal(rows_of(b, tables, s, h, tail), rows_of(a, p.tables, s, h, tail))
            if weights:
                got, want = args["mass_out"][s, h].cpu().numpy(), mass[s, h].cpu().numpy()
                assert np.array_equal(got[:c], want[kept[s, h, :c]])
                assert np.array_equal(got[c:], want[c:] if in_place else np.full(got.size - c, -7.0, np.float32))


def test_compaction_flags_bad_positions_and_blocks():
    p = Paged([64, 64], 2, 2, 64, seed=5)
    kept = torch.tensor([[[0, 3, 99999, 5]] * 2, [[-1, 1, 2, 63]] * 2], dtype=torch.int32, device=DEV)
    counts = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    dst = [torch.full((2, 2, 16, 64), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    dt = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)

    def call(**kw):
        a = dict(dst_desc=p.make_desc(num_blocks=2, max_blocks_per_seq=1), k_dst=dst[0], v_dst=dst[1], dst_tables=dt)
        a.update(kw)
        pkv.pkv_evict_compact(p.desc, p.k_pool, p.v_pool, p.t, kept, counts, **a)
    call()
    assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION
    assert (dst[0][0, :, 2] == 9).all() and (dst[1][1, :, 0] == 9).all() and (dst[0][:, :, 4:] == 9).all()
    for j, r in ((1, 3), (3, 5)):
        assert torch.equal(dst[0][0, 0, j], p.k_pool[p.tables[0, 0], 0, r])
    call(dst_tables=torch.tensor([[0], [2]], dtype=torch.int32, device=DEV))
    assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION | pkv.DEVERR_BLOCK_ID
    kept[:] = torch.arange(4, device=DEV)
    call(max_kept=2)
    assert pkv.pkv_device_errors() == pkv.DEVERR_LENGTH


# ----------------------------------------------------------- all of it --

@pytest.mark.parametrize("kv,d,hq,hkv,in_place", [("bf16", 128, 8, 2, False), ("e4m3", 64, 12, 3, True),
                                                  ("bf16", 64, 16, 2, True)])
def test_a_cache_is_thinned_and_served_on(kv, d, hq, hkv, in_place):
    """Prompt attention, its weights, the choice, the move, then decode steps whose new keys go
    behind the kept ones and whose weights are added, and a second thinning."""
    lens, q_lens, budget = [300, 45, 170], [40, 45, 33], 60
    p = Paged([n + 96 for n in lens], hq, hkv, d, kv, seed=11)  # room for the steps' keys
    for s, n in enumerate(lens):
        p.k[s], p.v[s] = p.k[s][:n], p.v[s][:n]
    p.lens = lens
    p.lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    r = Rule(d, hq, 3, cap=15.0)
    qo = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    qo_t = torch.from_numpy(qo).to(DEV)
    q, q64 = p.queries(int(qo[-1]))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    pkv.pkv_score_prefill(p.desc, r.score, q, qo_t, p.k_pool, p.v_pool, p.t, p.lens_t, out, lse, qo_indptr_host=qo,
                          kv_lens_host=lens, **p.scales)
    mass = torch.empty(3, hkv, 400, device=DEV)
    pkv.pkv_score_mass(p.desc, r.score, q, qo_t, p.k_pool, p.t, p.lens_t, 300, lse, mass, keep=0.0, max_q_len=45,
                       k_scale=p.scales["k_scale"])
    kept = torch.empty(3, hkv, budget, dtype=torch.int32, device=DEV)
    for turn in range(2):
        kept_lens = torch.empty(3, dtype=torch.int32, device=DEV)
        top = max(p.lens)
        pkv.pkv_evict_select(mass, p.lens_t, top, budget, 4, 8, kept, kept_lens)
        m = mass.cpu().numpy()
        chosen = [[select(m[s, h], p.lens[s], budget, 4, 8) for h in range(hkv)] for s in range(3)]
        for s in range(3):
            for h in range(hkv):
                assert np.array_equal(kept[s, h, :len(chosen[s][h])].cpu().numpy(), chosen[s][h])
        if in_place:
            pkv.pkv_evict_compact(p.desc, p.k_pool, p.v_pool, p.t, kept, kept_lens, mass=mass, mass_out=mass)
        else:
            k2, v2 = torch.zeros_like(p.k_pool), torch.zeros_like(p.v_pool)
            m2 = torch.zeros_like(mass)
            t2 = p.t.flip(0).contiguous()  # other blocks of the other pools
            pkv.pkv_evict_compact(p.desc, p.k_pool, p.v_pool, p.t, kept, kept_lens, dst_desc=p.desc, k_dst=k2,
                                  v_dst=v2, dst_tables=t2, mass=mass, mass_out=m2)
            # sequence 1 and 2 have fewer blocks than the row they take over in t2
            p.k_pool, p.v_pool, p.t, mass = k2, v2, t2, m2
        for rows in (p.k, p.v):
            for s in range(3):
                rows[s] = np.stack([rows[s][chosen[s][h], h] for h in range(hkv)], 1)
        p.lens = [len(chosen[s][0]) for s in range(3)]
        assert p.lens == kept_lens.cpu().tolist()
        for step in range(20):
            kv_new = [torch.from_numpy(p.rng.standard_normal((3, hkv, d)).astype(np.float32)).bfloat16() for _ in range(2)]
            slots = torch.tensor(p.lens, dtype=torch.int32, device=DEV)
            pkv.pkv_append_rope(p.desc, p.k_pool, p.v_pool, p.t, torch.arange(3, dtype=torch.int32, device=DEV), slots,
                                kv_new[0].to(DEV), kv_new[1].to(DEV), **p.scales)
            for s in range(3):
                for rows, x, sc in ((p.k, kv_new[0], p.scales["k_scale"]), (p.v, kv_new[1], p.scales["v_scale"])):
                    y = x[s].float()
                    if sc is not None:
                        y = (y / sc.cpu()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double() * sc.cpu().double()[:, None]
                    rows[s] = np.concatenate([rows[s], y.double().numpy()[None]])
            p.lens = [n + 1 for n in p.lens]
            p.lens_t = torch.tensor(p.lens, dtype=torch.int32, device=DEV)
            top = max(p.lens)
            q1, q164 = p.queries(3)
            out, lse = torch.empty_like(q1), torch.empty(3, hq, device=DEV)
            ws = torch.zeros(max(256, pkv.pkv_decode_workspace_size(p.desc, 3, top)), dtype=torch.uint8, device=DEV)
            pkv.pkv_score_decode(p.desc, r.score, q1, p.k_pool, p.v_pool, p.t, p.lens_t, top, out, lse, ws, **p.scales)
            before = mass.cpu().numpy().astype(np.float64)
            pkv.pkv_score_mass(p.desc, r.score, q1, None, p.k_pool, p.t, p.lens_t, top, lse, mass, keep=0.9,
                               k_scale=p.scales["k_scale"])
            if step in (0, 19):
                for s, n in enumerate(p.lens):
                    o, z, bo, bz = r.attend(p, s, q164[s:s + 1], [n - 1])
                    close(out[s:s + 1], o, bo)
                    close(lse[s:s + 1], z, bz)
                    want, bound = r.mass(p, s, q164[s:s + 1], [n - 1], lse[s:s + 1].cpu().numpy())
                    want[:, :n - 1] += float(np.float32(0.9)) * before[s, :, :n - 1]
                    close(mass[s, :, :n], want, bound + 8 * 2.0 ** -24 * want)
    assert pkv.pkv_device_errors() == 0


def test_a_step_and_a_thinning_captured_and_replayed():
    """Decode, weights, choice and move in one graph, replayed on new queries; the same bits as
    eager calls on another stream."""
    p = Paged([200, 333, 90], 8, 2, 128, seed=21)
    r = Rule(128, 8, 3, cap=15.0, slopes=0.05)
    qs = [p.queries(3)[0] for _ in range(3)]
    q = qs[0].clone()
    ws = torch.zeros(max(256, pkv.pkv_decode_workspace_size(p.desc, 3, 333)), dtype=torch.uint8, device=DEV)
    dst_tables = torch.arange(12, dtype=torch.int32, device=DEV).reshape(3, 4)
    dst_desc = p.make_desc(num_blocks=12, max_blocks_per_seq=4)

    def buffers():
        return dict(out=torch.zeros_like(q), lse=torch.zeros(3, 8, device=DEV), mass=torch.zeros(3, 2, 336, device=DEV),
                    kept=torch.zeros(3, 2, 50, dtype=torch.int32, device=DEV),
                    kept_lens=torch.zeros(3, dtype=torch.int32, device=DEV),
                    k=torch.zeros(12, 2, 16, 128, dtype=torch.bfloat16, device=DEV),
                    v=torch.zeros(12, 2, 16, 128, dtype=torch.bfloat16, device=DEV), m=torch.zeros(3, 2, 50, device=DEV))

    def step(b):
        pkv.pkv_score_decode(p.desc, r.score, q, p.k_pool, p.v_pool, p.t, p.lens_t, 333, b["out"], b["lse"], ws)
        pkv.pkv_score_mass(p.desc, r.score, q, None, p.k_pool, p.t, p.lens_t, 333, b["lse"], b["mass"], keep=0.5)
        pkv.pkv_evict_select(b["mass"], p.lens_t, 333, 50, 2, 5, b["kept"], b["kept_lens"])
        pkv.pkv_evict_compact(p.desc, p.k_pool, p.v_pool, p.t, b["kept"], b["kept_lens"], dst_desc=dst_desc, k_dst=b["k"],
                              v_dst=b["v"], dst_tables=dst_tables, mass=b["mass"], mass_out=b["m"])
    eager, graphed = buffers(), buffers()
    step(buffers())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(graphed)
    for x in graphed.values():
        x.zero_()
    side = torch.cuda.Stream()
    for new in qs:
        q.copy_(new)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step(eager)
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(eager[name], graphed[name]), name
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 64)])
def test_in_place_over_many_steps(kv, d):
    """Thousands of rows of one sequence: every step of the move reads behind what it writes, also
    where hardly anything moves, and where all of it moves far."""
    n = 9000
    p = Paged([n], 2, 2, d, kv, seed=22)
    rng = np.random.default_rng(23)
    for kind in range(3):
        kept = np.zeros((1, 2, 5000), np.int32)
        for h in range(2):
            kept[0, h] = (np.sort(rng.permutation(n)[:5000]) if kind == 0 else
                          np.concatenate([np.arange(4999), [n - 1]]) if kind == 1 else np.arange(n - 5000, n))
        src = [x.clone() for x in (p.k_pool, p.v_pool)]
        pkv.pkv_evict_compact(p.desc, p.k_pool, p.v_pool, p.t, torch.from_numpy(kept).to(DEV),
                              torch.tensor([5000], dtype=torch.int32, device=DEV))
        for h in range(2):
            for a, b in zip(src, (p.k_pool, p.v_pool)):
                assert np.array_equal(rows_of(b, p.tables, 0, h, range(5000)), rows_of(a, p.tables, 0, h, kept[0, h])), kind
    assert pkv.pkv_device_errors() == 0


def test_blocks_past_32_bits_are_moved():
    k, v = (torch.zeros(140004, 8, 16, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[140000:] = torch.randn(4, 8, 16, 128, device=DEV).bfloat16()
    v[140000:] = torch.randn(4, 8, 16, 128, device=DEV).bfloat16()
    desc = pkv.make_desc(num_q_heads=8, num_kv_heads=8, head_dim=128, num_blocks=140004, max_blocks_per_seq=4)
    src = torch.arange(140000, 140004, dtype=torch.int32, device=DEV)[None]
    dst = torch.tensor([[139999, 139998, 0, 1]], dtype=torch.int32, device=DEV)
    kept = torch.stack([torch.sort(torch.randperm(64)[:40]).values for _ in range(8)])[None].int().to(DEV)
    pkv.pkv_evict_compact(desc, k, v, src, kept, torch.tensor([40], dtype=torch.int32, device=DEV), dst_desc=desc, k_dst=k,
                          v_dst=v, dst_tables=dst)
    assert pkv.pkv_device_errors() == 0
    for pool in (k, v):
        rows = pool[140000:].transpose(0, 1).reshape(8, 64, 128)
        got = torch.cat([pool[139999], pool[139998], pool[0]], 1)[:, :40]
        assert torch.equal(got, torch.gather(rows, 1, kept[0].long()[..., None].expand(-1, -1, 128)))
