"""pkv_rope_rotate against the 64-bit rotation: layouts, partial heads, types,
strides, padding, the inverse as the gradient, streams and graphs."""
import numpy as np
import pytest
import torch

import _quant as Q
import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def table(theta, r, n, **kw):
    t = pkv.pkv_rope_scaled_table(theta, r, n, **kw)
    return t, torch.from_numpy(t).to(DEV)


def check(got, x, cs, pos, layout, inverse=False):
    """Half a step of the type on the result, and three fp32 roundings of
    2^-24 on |a c| + |b s|; f16's subnormal step as a floor."""
    x64, g = x.double().cpu().numpy(), got.double().cpu().numpy()
    for i, p in enumerate(pos):
        if p < 0 or p >= cs.shape[0]:
            continue
        ref = Q.rotate(x64[i], cs[p], layout, inverse=inverse)
        mag = Q.rotate(np.abs(x64[i]), np.stack((np.abs(cs[p][:, 0]), -np.abs(cs[p][:, 1])), -1), layout)
        mag = np.maximum(np.abs(mag), np.abs(x64[i])) + np.abs(ref)
        tol = STEP[x.dtype] * np.abs(ref) + 3 * 2.0 ** -24 * 2 * mag + 2.0 ** -25
        assert np.all(np.abs(g[i] - ref) <= tol), (i, np.abs(g[i] - ref).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hkv,d,r", [
    (1, 1, 0, 64, 64), (5, 8, 2, 64, 32), (33, 32, 8, 128, 128), (7, 3, 1, 128, 64), (9, 5, 2, 80, 80),
    (4, 2, 2, 96, 18), (3, 2, 1, 6, 2), (2, 4, 1, 512, 512), (17, 7, 7, 128, 16), (301, 16, 4, 128, 96),
    (5, 2, 1, 512, 18), (11, 3, 2, 256, 250), (29, 5, 1, 8, 6), (1, 1, 0, 64, 62), (3, 5, 2, 64, 50)])
def test_rotation(dtype, layout, tokens, hq, hkv, d, r):
    gen = torch.Generator().manual_seed(tokens * d + r)
    cs, t = table(1e4, r, 777, kind="linear", factor=2.0)
    pos = torch.randint(0, 777, (tokens,), generator=gen).int()
    pos[0] = 776
    q = torch.randn(tokens, hq, d, generator=gen).to(dtype)
    k = torch.randn(tokens, hkv, d, generator=gen).to(dtype) if hkv else None
    qd, kd = q.to(DEV), None if k is None else k.to(DEV)
    qo = torch.full_like(qd, float("nan"))
    ko = None if kd is None else torch.full_like(kd, float("nan"))
    pkv.pkv_rope_rotate(pkv.make_rope(t, layout=layout), pos.to(DEV), qd, qo, kd, ko)
    check(qo, q, cs, pos.tolist(), layout)
    assert torch.equal(qd.cpu(), q)
    if k is not None:
        check(ko, k, cs, pos.tolist(), layout)
    assert pkv.pkv_device_errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("where", ["packed", "head_major", "odd_offset", "broadcast"])
@pytest.mark.parametrize("r", [48, 18, 62])
def test_strides_in_place_and_out(dtype, layout, where, r):
    tokens, hq, hkv, d = 37, 6, 2, 64
    gen = torch.Generator().manual_seed(5)
    cs, t = table(1e4, r, 100)
    pos = torch.randint(0, 100, (tokens,), generator=gen).int()
    rope = pkv.make_rope(t, layout=layout)
    if where == "packed":
        buf = torch.randn(tokens, hq + 2 * hkv, d, generator=gen).to(dtype).to(DEV)
        q, k = buf[:, :hq], buf[:, hq:hq + hkv]
    elif where == "head_major":
        q = torch.randn(hq, tokens, d, generator=gen).to(dtype).to(DEV).transpose(0, 1)
        k = torch.randn(hkv, tokens, d, generator=gen).to(dtype).to(DEV).transpose(0, 1)
    elif where == "odd_offset":  # rows that start on no 16-byte boundary
        flat = torch.randn(tokens * (hq + hkv) * (d + 3) + 1, generator=gen).to(dtype).to(DEV)
        q = flat[1:1 + tokens * hq * (d + 3)].view(tokens, hq, d + 3)[..., :d]
        k = flat[1 + tokens * hq * (d + 3):].view(tokens, hkv, d + 3)[..., :d]
    else:
        q = torch.randn(1, hq, d, generator=gen).to(dtype).to(DEV).expand(tokens, hq, d)
        k = torch.randn(tokens, 1, d, generator=gen).to(dtype).to(DEV).expand(tokens, hkv, d)
    q0, k0 = q.cpu().clone(), k.cpu().clone()
    qo, ko = torch.empty(tokens, hq, d, dtype=dtype, device=DEV), torch.empty(tokens, hkv, d, dtype=dtype, device=DEV)
    pkv.pkv_rope_rotate(rope, pos.to(DEV), q, qo, k, ko)
    check(qo, q0, cs, pos.tolist(), layout)
    check(ko, k0, cs, pos.tolist(), layout)
    if where == "broadcast":
        with pytest.raises(pkv.PkvError, match="overlap"):
            pkv.pkv_rope_rotate(rope, pos.to(DEV), q, None, k, ko)
        return
    rest = buf[:, hq + hkv:].clone() if where == "packed" else None
    pkv.pkv_rope_rotate(rope, pos.to(DEV), q, None, k, None)  # in place: the same bits
    assert torch.equal(q, qo) and torch.equal(k, ko)
    if rest is not None:
        assert torch.equal(buf[:, hq + hkv:], rest)


def test_padding_and_positions_outside_the_table():
    cs, t = table(1e4, 64, 10)
    rope = pkv.make_rope(t)
    x = torch.randn(4, 2, 64, device=DEV, dtype=torch.bfloat16)
    out = torch.full_like(x, 7.0)
    pos = torch.tensor([3, -1, 9, -2 ** 31], dtype=torch.int32, device=DEV)
    pkv.pkv_rope_rotate(rope, pos, x, out)
    check(out, x.cpu(), cs, [3, -1, 9, -1], "half")
    assert torch.all(out[1] == 7) and torch.all(out[3] == 7) and pkv.pkv_device_errors() == 0
    out.fill_(7.0)
    pkv.pkv_rope_rotate(rope, torch.tensor([10, 0, 2 ** 31 - 1, 1], dtype=torch.int32, device=DEV), x, out)
    assert torch.all(out[0] == 7) and torch.all(out[2] == 7)
    assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION
    check(out, x.cpu(), cs, [-1, 0, -1, 1], "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("attention", [1.0, 1.3])
def test_inverse_is_the_gradient(layout, attention):
    """L = sum(w * rotate(x)): dL/dx is the transposed rotation of w -- against
    the formula's gradient (64-bit autograd) and against differences."""
    tokens, h, d, r = 6, 3, 32, 24
    gen = torch.Generator().manual_seed(11)
    cs, t = table(1e3, r, 50, attention=attention)
    pos = torch.randint(0, 50, (tokens,), generator=gen).int()
    x = torch.randn(tokens, h, d, generator=gen, dtype=torch.float64, requires_grad=True)
    w = torch.randn(tokens, h, d, generator=gen)
    c, s = (torch.from_numpy(cs)[pos.long()][..., i].double()[:, None] for i in (0, 1))
    i0, i1 = ((slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2)))
    a, b = x[..., i0], x[..., i1]
    ((w[..., i0] * (a * c - b * s)).sum() + (w[..., i1] * (b * c + a * s)).sum()
     + (w[..., r:] * x[..., r:]).sum()).backward()
    got = torch.empty(tokens, h, d, device=DEV)
    pkv.pkv_rope_rotate(pkv.make_rope(t, layout=layout, inverse=True), pos.to(DEV), w.to(DEV), got)
    # three roundings of 2^-24 on |c w| + |s w'| <= 2 * 1.3 * max|w|
    tol = 3 * 2.0 ** -24 * 2.6 * float(w.abs().max())
    assert (got.cpu().double() - x.grad).abs().max() <= tol
    # differences of the forward kernel: the map is linear, so any step is exact but for roundings
    fwd = pkv.make_rope(t, layout=layout)
    x0 = x.detach().float()
    for (i, j, e) in ((0, 0, 0), (3, 2, 1), (5, 1, r - 1), (2, 0, d - 1)):
        hi, lo = x0.clone(), x0.clone()
        hi[i, j, e] += 1.0
        lo[i, j, e] -= 1.0
        ys = []
        for v in (hi, lo):
            y = torch.empty(tokens, h, d, device=DEV)
            pkv.pkv_rope_rotate(fwd, pos.to(DEV), v.to(DEV), y)
            ys.append((y.cpu().double() * w.double())[i, j].sum())
        assert abs(float(ys[0] - ys[1]) / 2 - float(x.grad[i, j, e])) <= 64 * tol


def test_streams_and_graph_replay():
    cs, t = table(1e4, 128, 4096)
    rope = pkv.make_rope(t, layout="interleaved")
    x = torch.randn(130, 8, 128, device=DEV, dtype=torch.bfloat16)
    pos = torch.arange(130, dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.pkv_rope_rotate(rope, pos, x, out)
    other = torch.empty_like(x)
    pkv.pkv_rope_rotate(rope, pos, x, other, stream=side)
    side.synchronize()
    check(out, x.cpu(), cs, pos.tolist(), "interleaved")
    assert torch.equal(out, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_rope_rotate(rope, pos, x, out)
    x.copy_(torch.randn_like(x, dtype=torch.float32).bfloat16())
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    check(out, x.cpu(), cs, pos.tolist(), "interleaved")


def test_offsets_past_32_bits():
    """Rows further than 2^31 elements from the first."""
    cs, t = table(1e4, 64, 64)
    far = (1 << 31) // 2 + 64
    buf = torch.empty(3 * far, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, 1, 64), (far, 64, 1))
    x.copy_(torch.randn(3, 1, 64))
    out = torch.empty(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.tensor([1, 30, 63], dtype=torch.int32, device=DEV)
    pkv.pkv_rope_rotate(pkv.make_rope(t), pos, x, out)
    check(out, x.cpu(), cs, pos.tolist(), "half")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hkv,d,r", [(32, 8, 128, 128), (5, 3, 128, 64), (9, 0, 96, 32), (6, 2, 64, 18)])
def test_many_rows_are_turned_as_few_are(dtype, layout, hq, hkv, d, r):
    """So many rows that a thread takes four heads (heads that are no multiple of four,
    passing dims, padding and bad positions included), against calls of few tokens."""
    n = 4 * 152 * 512 * 16 // ((hq + hkv) * r * dtype.itemsize // (2 if layout == "half" else 1)) + 13
    cs, t = table(1e4, r, 500)
    rope = pkv.make_rope(t, layout=layout)
    gen = torch.Generator().manual_seed(n)
    pos = torch.randint(0, 500, (n,), generator=gen).int()
    pos[[0, 5, n - 1]] = torch.tensor([-1, 500, -7], dtype=torch.int32)
    pd = pos.to(DEV)
    x = torch.randn(n, hq + hkv, d, generator=gen).to(dtype).to(DEV)

    def run(step, in_place):
        src = x.clone() if in_place else x
        out = src if in_place else torch.full_like(x, 7.0)
        for i in range(0, n, step):
            at = slice(i, i + step)
            pkv.pkv_rope_rotate(rope, pd[at], src[at, :hq], None if in_place else out[at, :hq],
                                src[at, hq:] if hkv else None, None if in_place or not hkv else out[at, hq:])
        assert pkv.pkv_device_errors() == pkv.DEVERR_POSITION
        return out
    few = run(997, False)
    check(few[::31], x[::31].cpu(), cs, pos[::31].tolist(), layout)
    assert torch.equal(run(n, False), few)
    padded = torch.tensor([0, 5, n - 1], device=DEV)
    assert torch.all(few[padded] == 7)
    few[padded] = x[padded]
    assert torch.equal(run(n, True), few)


def test_more_threads_than_one_launch_reaches():
    """In place, so many rows that they take several launches: each row turns once, those
    beside the launches' borders included."""
    tokens, heads = 1_500_000_000, 3
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("40 GB of device memory")
    cs = torch.tensor([[[1.0, 0.0]], [[0.6, 0.8]]], device=DEV)
    x = torch.zeros(tokens, heads, 2, dtype=torch.bfloat16, device=DEV)
    x[..., 0] = 1.0
    pos = torch.ones(tokens, dtype=torch.int32, device=DEV)
    pkv.pkv_rope_rotate(pkv.make_rope(cs), pos, x)
    want = torch.tensor([0.6, 0.8]).bfloat16().view(torch.int32).item()  # a pair's bits
    pairs = x.view(torch.int32).view(-1)
    for i in range(0, pairs.numel(), 1 << 29):
        assert torch.all(pairs[i:i + (1 << 29)] == want), i
    del x, pos, pairs
    torch.cuda.empty_cache()
