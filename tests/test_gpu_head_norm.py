"""head_norm on the GPU against its 64-bit form.

Tolerance: u = 2^-24. The sum of squares has at most 22 additions in a row (16 of a lane, 6 over the wave), so half of
23 u on its root; the quotient by d, eps, root, reciprocal, and the products with x's factor and gain take at most 6 more:
18 u of |v|. Sine and cosine are within 3e-7 (5 u), a turned value has 3 roundings more: 26 u (|p| + |q|). One rounding
of the output is half a step.
"""
import pytest
import torch

import kronecker_hessian_rounding_amd as bk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def form64(x, gain, pos, freq, eps, norm, pairs):
    """(value, error bound before the output's rounding) of heads x (T x H x d), in 64 bits."""
    v = x.double()
    if norm:
        v = v / (v.square().mean(2, keepdim=True) + eps).sqrt()
        v = v if gain is None else v * gain.double()
    tol = 18 * U * v.abs() if norm else torch.zeros_like(v)
    if freq is None or freq.numel() == 0:
        return v, tol
    r = freq.numel()
    a = pos.double()[:, None, None] * freq.double()
    i = (slice(0, r), slice(r, 2 * r)) if pairs == "half" else (slice(0, 2 * r, 2), slice(1, 2 * r, 2))
    p, q = v[..., i[0]], v[..., i[1]]
    out, tol = v.clone(), tol.clone()
    out[..., i[0]], out[..., i[1]] = p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()
    tol[..., i[0]] = tol[..., i[1]] = 26 * U * (p.abs() + q.abs())
    return out, tol


def check(y, x, gain, pos, freq, eps, norm, pairs):
    ref, tol = form64(x, gain, pos, freq, eps, norm, pairs)
    fi = torch.finfo(y.dtype)
    tol = tol + (ref.abs() + tol) * fi.eps / 2 + fi.tiny * fi.eps
    err = (y.cpu().double() - ref).abs()
    assert y.shape == x.shape and bool((err <= tol).all()), float((err / tol).max())


def case(T, hq, hk, d, rot, dtype, pairs="half", norm=True, gains="x", eps=1e-6, far=1 << 20, pos32=False, seed=0):
    g = gen(seed)
    q, k = torch.randn(T, hq, d, generator=g).to(dtype), torch.randn(T, hk, d, generator=g).to(dtype)
    gt = {"x": dtype, "f32": F32, None: None}[gains]
    gq, gk = ((1 + 0.3 * torch.randn(d, generator=g)).to(gt) for _ in range(2)) if gt and norm else (None, None)
    pos = torch.randint(-far, far, (T,), generator=g, dtype=torch.int32 if pos32 else torch.int64) if rot else None
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=F32) / max(1, rot // 2)) if rot else None
    return q, k, gq, gk, pos, freq


def dev(t):
    return None if t is None else t.cuda()


def run(q, k, gq, gk, pos, freq, **kw):
    return bk.head_norm(q, k, q_gain=dev(gq), k_gain=dev(gk), positions=dev(pos), freq=dev(freq), **kw)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hk,d,rot", [(1, 1, 1, 1, 0), (2, 3, 1, 2, 2), (5, 4, 2, 7, 6), (3, 5, 3, 16, 16), (4, 32, 8, 128, 128),
                                           (2, 6, 2, 80, 32), (3, 2, 2, 96, 96), (2, 3, 1, 100, 50), (1, 70, 9, 64, 64),
                                           (3, 2, 1, 256, 254), (2, 2, 2, 511, 510), (2, 1, 1, 512, 512), (2, 40, 30, 512, 2),
                                           (2, 3, 3, 144, 0), (2, 5, 5, 33, 16)])
def test_against_64_bits(T, hq, hk, d, rot, pairs, dtype):
    for norm, gains in ((True, "x"), (True, "f32"), (True, None), (False, None)):
        q, k, gq, gk, pos, freq = case(T, hq, hk, d, rot, dtype, norm=norm, gains=gains, seed=d + T)
        yq, yk = run(q.cuda(), k.cuda(), gq, gk, pos, freq, pairs=pairs, norm=norm)
        check(yq, q, gq, pos, freq, 1e-6, norm, pairs)
        check(yk, k, gk, pos, freq, 1e-6, norm, pairs)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_views_of_a_fused_projection(dtype):
    """Queries and keys as column ranges of one buffer at an odd offset, in place and into another; nothing else is written."""
    T, hq, hk, d = 7, 6, 2, 64
    q, k, gq, gk, pos, freq = case(T, hq, hk, d, d, dtype, pos32=True)
    buf = torch.full((T, 1 + (hq + 2 * hk) * d + 5), 9.0, dtype=dtype, device="cuda")
    vq = buf[:, 1:1 + hq * d].unflatten(1, (hq, d))
    vk = buf[:, 1 + hq * d:1 + (hq + hk) * d].unflatten(1, (hk, d))
    vq.copy_(q)
    vk.copy_(k)
    ref = run(q.cuda(), k.cuda(), gq, gk, pos, freq)
    check(ref[0], q, gq, pos, freq, 1e-6, True, "half")
    got = run(vq, vk, gq, gk, pos, freq)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    # heads of one buffer's tokens into heads-major rows, as a cache keeps them
    oq = torch.empty(hq, T, d, dtype=dtype, device="cuda")
    got = run(vq, vk, gq, gk, pos, freq, out_q=oq.transpose(0, 1))
    assert torch.equal(oq.transpose(0, 1), ref[0]) and torch.equal(got[1], ref[1])
    back = run(oq.transpose(0, 1), None, None, None, pos, freq, norm=False)[0]
    assert torch.equal(back, run(ref[0], None, None, None, pos, freq, norm=False)[0])
    run(vq, vk, gq, gk, pos, freq, out_q=vq, out_k=vk)
    assert torch.equal(vq, ref[0]) and torch.equal(vk, ref[1])
    vq.fill_(9.0)
    vk.fill_(9.0)
    assert bool((buf == 9.0).all())


def test_far_positions():
    """Angles of positions up to 2^40: the product is rounded to 53 bits, which the bound's trigonometric part covers."""
    T, d = 64, 128
    q, _, _, _, _, freq = case(T, 1, 1, d, d, F32)
    pos = torch.randint(0, 1 << 40, (T,), generator=gen(3))
    y, _ = bk.head_norm(q.cuda(), positions=pos.cuda(), freq=freq.cuda(), norm=False)
    # 2^40 of angle: 2^-13 turns of rounding at most (2^40 / 6.28 turns times 3 roundings of 2^-53), 4e-4 * 2 pi
    ref, _ = form64(q, None, pos, freq, 0.0, False, "half")
    assert float((y.cpu().double() - ref).abs().max()) <= 2 ** 40 * 3 * 2.0 ** -53 * float(q.abs().max()) * 2 + 1e-5


def test_zeros_and_non_finite():
    q = torch.randn(3, 4, 64, generator=gen(1))
    q[0, 1] = 0.0
    q[1, 2, 5] = float("inf")
    q[2, 3, 7] = float("nan")
    y = bk.head_norm(q.cuda())[0].cpu()
    assert bool((y[0, 1] == 0).all())
    assert bool(torch.isnan(y[1, 2, 5])) and bool((y[1, 2, :5] == 0).all())
    assert bool(torch.isnan(y[2, 3]).all())
    ok = torch.ones(3, 4, dtype=torch.bool)
    ok[1, 2] = ok[2, 3] = False
    ref, tol = form64(q, None, None, None, 1e-6, True, "half")
    assert bool(((y.double() - ref).abs()[ok] <= (tol + ref.abs() * U)[ok]).all())


def test_empty():
    y, z = bk.head_norm(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 2, 64, device="cuda"))
    assert y.shape == (0, 4, 64) and z.shape == (0, 2, 64)


def test_more_tokens_than_a_grid():
    """2^22 + 3 tokens of one small head: workgroups take a second token, with its own angles."""
    T = (1 << 22) + 3
    q = torch.randn(T, 1, 2, generator=gen(5))
    pos = torch.arange(T)
    freq = torch.tensor([0.37])
    y = bk.head_norm(q.cuda(), positions=pos.cuda(), freq=freq.cuda())[0]
    check(y, q, None, pos, freq, 1e-6, True, "half")


def test_offsets_past_2_31():
    ld = (1 << 31) + 64
    small = torch.randn(2, 2, 64, generator=gen(6)).to(BF16).cuda()
    x = torch.empty(ld + 128, dtype=BF16, device="cuda").as_strided((2, 2, 64), (ld, 64, 1))
    x.copy_(small)
    assert torch.equal(bk.head_norm(x)[0], bk.head_norm(small)[0])
    y = torch.empty(ld + 128, dtype=BF16, device="cuda").as_strided((2, 2, 64), (64, ld, 1))
    bk.head_norm(small, out_q=y)
    assert torch.equal(y.contiguous(), bk.head_norm(small)[0])


def test_refusals():
    q, k = torch.zeros(3, 4, 64, device="cuda"), torch.zeros(3, 2, 64, device="cuda")
    pos, freq = torch.arange(3, device="cuda"), torch.ones(32, device="cuda")
    one = torch.ones(64, device="cuda")
    bad = [lambda: bk.head_norm(q[0]), lambda: bk.head_norm(q.double()), lambda: bk.head_norm(q, k.half()),
           lambda: bk.head_norm(q, k[:2]), lambda: bk.head_norm(q, k[..., :32]), lambda: bk.head_norm(q.cpu()),
           lambda: bk.head_norm(q, positions=pos), lambda: bk.head_norm(q, freq=freq),
           lambda: bk.head_norm(q, positions=pos[:2], freq=freq), lambda: bk.head_norm(q, positions=pos.float(), freq=freq),
           lambda: bk.head_norm(q, positions=pos.cpu(), freq=freq), lambda: bk.head_norm(q, positions=pos, freq=freq.double()),
           lambda: bk.head_norm(q, positions=pos, freq=torch.ones(33, device="cuda")),
           lambda: bk.head_norm(q, q_gain=one[:63]), lambda: bk.head_norm(q, q_gain=one, norm=False),
           lambda: bk.head_norm(q, k, q_gain=one, k_gain=one.half()), lambda: bk.head_norm(q.half(), k.half(), one, one.half()),
           lambda: bk.head_norm(q, k_gain=one), lambda: bk.head_norm(q, out_k=k), lambda: bk.head_norm(q, pairs="both"),
           lambda: bk.head_norm(q, out_q=k), lambda: bk.head_norm(q[..., ::2]), lambda: bk.head_norm(q[:, :0])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % i)
    for f in (lambda: bk.head_norm(q, eps=-1.0), lambda: bk.head_norm(torch.zeros(1, 1, 513, device="cuda")),
              lambda: bk.head_norm(q[:2], out_q=q[1:]), lambda: bk.head_norm(q, k, out_q=q, out_k=q[:, :2]),
              lambda: bk.head_norm(q[:1].expand(3, 4, 64)), lambda: bk.head_norm(q[:, :1].expand(3, 4, 64))):
        with pytest.raises(bk.BakronError):
            f()


def test_stream_and_graph():
    q, k, gq, gk, pos, freq = case(4, 8, 2, 128, 128, BF16)
    q, k, gq, gk, pos, freq = (t.cuda() for t in (q, k, gq, gk, pos, freq))

    def step():
        return bk.head_norm(q, k, gq, gk, pos, freq)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other[0], step()[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for i in range(4):
        q.copy_(torch.randn(4, 8, 128, generator=gen(i)))
        pos.add_(1000 * i + 1)
        graph.replay()
        torch.cuda.synchronize()
        e = step()
        assert torch.equal(y[0], e[0]) and torch.equal(y[1], e[1])


@pytest.mark.parametrize("T,H,Hk,d", [(5, 4, 4, 64), (1, 3, 3, 80), (7, 1, 1, 33), (3, 6, 2, 128)])
@pytest.mark.parametrize("heads_outside", [False, True])
def test_in_place_side_by_side(T, H, Hk, d, heads_outside):
    """A projection that leaves query, key and value of one head side by side, [token][head][3][d] (or heads outside): in place,
    and the values stay. Fewer keys than queries use the first heads' places."""
    buf = torch.randn((H, T, 3, d) if heads_outside else (T, H, 3, d), generator=gen(d)).to(BF16).cuda()
    rows = buf.transpose(0, 1) if heads_outside else buf
    q, k, v = rows[:, :, 0], rows[:, :Hk, 1], rows[:, :, 2].clone()
    gq, gk = torch.randn(d, generator=gen(1)).cuda(), torch.randn(d, generator=gen(2)).cuda()
    pos, freq = torch.arange(T).cuda(), torch.rand(d // 2, generator=gen(3)).cuda()
    kw = dict(q_gain=gq, k_gain=gk, positions=pos, freq=freq)
    wq, wk = bk.head_norm(q.contiguous(), k.contiguous(), **kw)
    rest = rows[:, Hk:, 1].clone()
    yq, yk = bk.head_norm(q, k, out_q=q, out_k=k, **kw)
    assert yq.data_ptr() == q.data_ptr() and torch.equal(q, wq) and torch.equal(k, wk)
    assert torch.equal(rows[:, :, 2], v) and torch.equal(rows[:, Hk:, 1], rest)
    # into the values' places and back
    u = rows[:, :, 2]
    bk.head_norm(q, out_q=u, q_gain=gq)
    assert torch.equal(u, bk.head_norm(wq, q_gain=gq)[0]) and torch.equal(q, wq)
