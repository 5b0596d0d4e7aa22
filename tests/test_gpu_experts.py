"""experts on the GPU against its 64-bit form.

Tolerance: u = 2^-24. Both products are those of matvec: exact products, a chunk's sum of at most 256 terms of at most 3
pieces (two fp32 roundings of at most 2 u each), the chunks' sums one addition and product each, unit and scale:
P(n) = 2 u (3 min(n, 256) + n / 128 + 20) of the sum of magnitudes. Between them act has a slope of at most 1.13 and an
error of at most 16 u |g| (an exponential, its argument, a quotient), the products with u and w 2 u more. What lies
between them is held to 2^-17 (2^-24 for an fp32 output). Behind them at most k additions; then half a step of the output's
type.
"""
import pytest
import torch

import kronecker_hessian_rounding_amd as bk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def layers(E, m, n, bits, group, seed):
    g = gen(seed)
    ng = -(-n // group) if group else 1
    return (torch.randint(0, 2 ** bits, (E, m, n), generator=g, dtype=torch.uint8),
            (torch.rand(E, m, ng, generator=g) + 0.25) * n ** -0.5)


def dense(pair, e, bits, group):
    v = pair[0][e].double() - (2 ** bits - 1) / 2
    s = pair[1][e].double()
    return v * (s.repeat_interleave(group, 1)[:, :v.shape[1]] if group else s)


def tokens(T, n, dtype, seed):
    g = gen(seed)
    if dtype == I8:
        return torch.randint(-127, 128, (T, n), generator=g, dtype=I8)
    return torch.randn(T, n, generator=g).to(dtype)


def chosen(T, E, k, seed, none=0.0):
    """Distinct experts of each token, some slots with none."""
    g = gen(seed)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32)
    ids[torch.rand(T, k, generator=g) < none] = -1
    return ids, torch.rand(T, k, generator=g)


def prod_bound(n):
    return 2 * U * (3 * min(n, 256) + n / 128 + 20)


def form64(x, xs, w, ids, weights, act, held=2.0 ** -24):
    """(result, error bound before the output's rounding) in 64 bits."""
    gate, up, down, bits, group, dbits, dgroup = w
    E, n, I = gate[0].shape[0], gate[0].shape[2], gate[0].shape[1]
    T, k = ids.shape
    x = x.double() if xs is None else x.double() * xs.double()[:, None]
    y, tol = torch.zeros(T, n, dtype=torch.float64), torch.zeros(T, n, dtype=torch.float64)
    for e in range(E):
        rows = (ids == e).any(1).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        wt = (weights.double() * (ids == e))[rows].sum(1, keepdim=True)
        G, V, D = dense(gate, e, bits, group), dense(up, e, bits, group), dense(down, e, dbits, dgroup)
        v = x[rows]
        g, u = v @ G.t(), v @ V.t()
        dg, du = v.abs() @ G.abs().t() * prod_bound(n), v.abs() @ V.abs().t() * prod_bound(n)
        a = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        da = 1.13 * dg + 16 * U * (g.abs() + dg)
        h = wt * a * u
        dh = wt.abs() * (da * (u.abs() + du) + (a.abs() + da) * du) + (4 * U + held) * h.abs()
        y[rows] += h @ D.t()
        tol[rows] += (h.abs() * prod_bound(I) + dh) @ D.abs().t()
    return y, tol


def check(T, E, k, n, I, bits, group, dbits, dgroup, dtype, out_dtype, act="silu", none=0.0, seed=0, ids=None, view=None):
    gate, up, down = layers(E, I, n, bits, group, seed), layers(E, I, n, bits, group, seed + 1), layers(E, n, I, dbits, dgroup, seed + 2)
    x, xs = tokens(T, n, dtype, seed + 3), torch.rand(T, generator=gen(seed + 4)) + 0.5
    if dtype == I8:
        xs = xs / 64
    i, wt = chosen(T, E, k, seed + 5, none)
    if ids is not None:
        i = ids
    packed = [bk.pack_experts(c.cuda(), s.cuda(), b, g) for (c, s), b, g in ((gate, bits, group), (up, bits, group), (down, dbits, dgroup))]
    y = bk.experts(x.cuda() if view is None else view(x.cuda()), *packed, i.cuda(), wt.cuda(), x_scale=xs.cuda(), act=act, out_dtype=out_dtype)
    assert y.shape == (T, n) and y.dtype == out_dtype
    ref, tol = form64(x, xs, (gate, up, down, bits, group, dbits, dgroup), i, wt, act, 2.0 ** -24 if out_dtype == F32 else 2.0 ** -17)
    fi = torch.finfo(out_dtype)
    # the sum over a token's experts: k additions of values of at most the parts' magnitudes
    tol = tol + k * U * (ref.abs() + tol) * 2 + (ref.abs() + tol) * fi.eps / 2 + fi.tiny * fi.eps
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), int((err > tol).sum()))
    return y


@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("T,E,k,n,I,bits,group,dbits,dgroup", [
    (1, 1, 1, 1, 1, 4, 0, 4, 0), (1, 4, 2, 64, 48, 4, 32, 4, 32), (3, 5, 3, 100, 77, 3, 32, 2, 0), (1, 16, 4, 1024, 256, 4, 128, 4, 128),
    (16, 8, 2, 256, 300, 4, 64, 3, 128), (7, 3, 3, 513, 130, 2, 0, 4, 64), (20, 4, 4, 96, 512, 4, 128, 1, 256), (33, 6, 1, 200, 40, 1, 64, 2, 32),
    (70, 2, 2, 130, 70, 4, 128, 4, 128), (5, 64, 8, 384, 128, 4, 128, 4, 0), (130, 3, 2, 64, 200, 2, 128, 2, 512), (2, 9, 2, 7, 3, 4, 0, 4, 0)])
def test_against_64_bits(T, E, k, n, I, bits, group, dbits, dgroup, dtype):
    check(T, E, k, n, I, bits, group, dbits, dgroup, dtype, F32, seed=T + n)
    check(T, E, k, n, I, bits, group, dbits, dgroup, dtype, BF16 if dtype != F16 else F16, act="gelu", none=0.3, seed=T + I)


@pytest.mark.parametrize("dtype", [F32, BF16, I8])
@pytest.mark.parametrize("T,E,k", [(1, 1000, 64), (2, 70, 60), (16, 1024, 32), (9, 1024, 64), (8, 90, 64), (16, 4, 3), (40, 2, 2), (300, 4, 2), (17, 128, 8), (64, 16, 1), (9000, 2, 2)])
def test_launch_shapes(T, E, k, dtype):
    """Many experts and slots, all tokens at few experts, and more pairs than one round of launches takes."""
    check(T, E, k, 40, 33, 4, 32, 4, 32, dtype, F32, none=0.1, seed=T)


@pytest.mark.parametrize("dtype", [F32, F16, I8])
@pytest.mark.parametrize("T,E,k,n,I,dbits,dgroup", [(6, 8, 4, 4099, 2050, 4, 128), (16, 4, 3, 8200, 2048, 2, 64), (9, 4, 4, 4112, 4000, 4, 32)])
def test_second_product_in_splits(T, E, k, n, I, dbits, dgroup, dtype):
    check(T, E, k, n, I, 4, 128, dbits, dgroup, dtype, F32, none=0.2, seed=T)


@pytest.mark.parametrize("T,k", [(4, 3), (40, 4)])
def test_padding_repeats_and_empty_rows(T, k):
    """No expert at all, ids on either side of the range, one expert twice in a row."""
    E = 5
    ids = torch.randint(0, E, (T, k), generator=gen(1), dtype=torch.int32)
    ids[0] = -1
    ids[1, 0], ids[1, 1] = E, -2 ** 31
    ids[2] = 3
    ids[3, 0], ids[3, 2] = 2, 2
    y = check(T, E, k, 130, 90, 4, 128, 4, 32, BF16, F32, ids=ids)
    assert bool((y[0] == 0).all())
    y = check(T, E, k, 130, 90, 4, 128, 4, 32, F32, BF16, ids=torch.full((T, k), -1, dtype=torch.int32))
    assert bool((y == 0).all())
    check(T, E, k, 130, 90, 4, 128, 4, 32, F32, F32, ids=torch.full((T, k), E - 1, dtype=torch.int32))


@pytest.mark.parametrize("T", [5, 50])
def test_other_rows_do_not_matter(T):
    """A token's result stays bit for bit when the other rows change, to NaN and infinity too."""
    E, k, n, I = 6, 2, 300, 200
    packed = [bk.pack_experts(c.cuda(), s.cuda(), 4, 128) for c, s in (layers(E, I, n, 4, 128, 1), layers(E, I, n, 4, 128, 2), layers(E, n, I, 4, 128, 3))]
    x = tokens(T, n, BF16, 4).cuda()
    ids, wt = (t.cuda() for t in chosen(T, E, k, 5))
    y = bk.experts(x, *packed, ids, wt)
    x2 = x.clone()
    x2[1:, 7] = float("nan")
    x2[2, 9] = float("inf")
    ids2 = ids.clone()
    ids2[1:] = ids[0]
    z = bk.experts(x2, *packed, ids2, wt)
    assert torch.equal(z[0], y[0]) and bool(torch.isnan(z[1]).all())


@pytest.mark.parametrize("T", [1, 3, 7, 16, 60])
def test_other_experts_do_not_matter(T):
    """Scales that are not finite stay with the tokens that name their expert."""
    E, k, n, I = 6, 2, 200, 150
    raw = [layers(E, I, n, 4, 128, 1), layers(E, I, n, 4, 128, 2), layers(E, n, I, 4, 128, 3)]
    x, (ids, wt) = tokens(T, n, BF16, 4).cuda(), chosen(T, E, k, 5)
    mk = lambda: [bk.pack_experts(c.cuda(), s.cuda(), 4, 128) for c, s in raw]
    y = bk.experts(x, *mk(), ids.cuda(), wt.cuda())
    for i, v in enumerate((float("inf"), float("nan"), float("inf"))):
        raw[i][1][4, 3] = v
    z = bk.experts(x, *mk(), ids.cuda(), wt.cuda())
    clean = ~(ids == 4).any(1)
    assert torch.equal(z[clean.cuda()], y[clean.cuda()]) and bool((~torch.isfinite(z[(~clean).cuda()])).any(1).all())


@pytest.mark.parametrize("dtype", [F32, BF16, I8])
@pytest.mark.parametrize("T", [6, 90])
def test_strided_rows(T, dtype):
    """Column ranges of wider buffers at odd offsets; nothing else is written."""
    E, k, n, I = 4, 2, 131, 100
    packed = [bk.pack_experts(c.cuda(), s.cuda(), 4, 64) for c, s in (layers(E, I, n, 4, 64, 1), layers(E, I, n, 4, 64, 2), layers(E, n, I, 4, 64, 3))]
    x = tokens(T, n, dtype, 4).cuda()
    ids, wt = (t.cuda() for t in chosen(T, E, k, 5))
    ref = bk.experts(x, *packed, ids, wt, out_dtype=F32)
    xb = torch.zeros(T, n + 9, dtype=dtype, device="cuda")
    xb[:, 3:3 + n] = x
    yb = torch.full((T + 1, n + 5), 8.0, device="cuda")
    bk.experts(xb[:, 3:3 + n], *packed, ids, wt, out=yb[:T, 1:1 + n])
    assert torch.equal(yb[:T, 1:1 + n], ref)
    yb[:T, 1:1 + n] = 8.0
    assert bool((yb == 8.0).all())


def test_empty():
    packed = [bk.pack_experts(c.cuda(), s.cuda(), 4, 0) for c, s in (layers(2, 32, 64, 4, 0, 1), layers(2, 32, 64, 4, 0, 2), layers(2, 64, 32, 4, 0, 3))]
    y = bk.experts(torch.empty(0, 64, device="cuda"), *packed, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    assert y.shape == (0, 64)


def test_refusals():
    E, k, n, I, T = 3, 2, 64, 32, 4
    mk = lambda m, c, g=32, b=4: bk.pack_experts(*(t.cuda() for t in layers(E, m, c, b, g, 1)), b, g)
    gate, up, down = mk(I, n), mk(I, n), mk(n, I)
    x = tokens(T, n, BF16, 2).cuda()
    ids, wt = (t.cuda() for t in chosen(T, E, k, 3))
    c, s = (t.cuda() for t in layers(E, I, n, 4, 32, 1))
    bad = [lambda: bk.experts(x[:, :63], gate, up, down, ids, wt), lambda: bk.experts(x, gate, up, gate, ids, wt),
           lambda: bk.experts(x, gate, mk(I, n, 64), down, ids, wt), lambda: bk.experts(x, gate, mk(I, n, 32, 2), down, ids, wt),
           lambda: bk.experts(x, gate, mk(I + 1, n), down, ids, wt), lambda: bk.experts(x, gate, up, down, ids.long(), wt),
           lambda: bk.experts(x, gate, up, down, ids[:3], wt[:3]), lambda: bk.experts(x, gate, up, down, ids, wt[:, :1]),
           lambda: bk.experts(x, gate, up, down, ids, wt.double()), lambda: bk.experts(x, gate, up, down, ids.cpu(), wt),
           lambda: bk.experts(x, gate, up, down, ids.t().contiguous().t(), wt), lambda: bk.experts(x.double(), gate, up, down, ids, wt),
           lambda: bk.experts(x, gate, up, down, ids, wt, act="relu"), lambda: bk.experts(x, gate, up, down, ids, wt, out_dtype=I8),
           lambda: bk.experts(x, gate, up, down, ids, wt, x_scale=wt[:, 0]), lambda: bk.experts(x, gate, up, down, ids, wt, out=x[:, :63]),
           lambda: bk.pack_experts(c[0], s[0], 4, 32), lambda: bk.pack_experts(c, s[:2], 4, 32), lambda: bk.pack_experts(c, s, 5, 32),
           lambda: bk.pack_experts(c, s, 4, 48), lambda: bk.pack_experts(c.cpu(), s, 4, 32), lambda: bk.pack_experts(c, s[:, :, :1], 4, 32),
           lambda: bk.PackedExperts(gate.data[:-1], E, I, n, 4, 32), lambda: bk.PackedExperts(gate.data, E + 1, I, n, 4, 32)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % i)
    many = torch.zeros(T, 65, dtype=torch.int32, device="cuda")
    for f in (lambda: bk.experts(x, gate, up, down, ids, wt, out=x), lambda: bk.experts(x, gate, up, down, many, torch.zeros(T, 65, device="cuda")),
              lambda: bk.experts(x, gate, up, down, ids[:, :0].contiguous(), wt[:, :0].contiguous())):
        with pytest.raises(bk.BakronError):
            f()
    # a layer whose bytes were replaced
    data = down.data
    down.data = data[:-16]
    with pytest.raises(bk.BakronError):
        bk.experts(x, gate, up, down, ids, wt)


@pytest.mark.parametrize("T", [1, 8, 60])
def test_stream_and_graph(T):
    """Two captured graphs and eager calls on another stream in between, each with its own workspace."""
    E, k, n, I = 6, 2, 512, 256
    packed = [bk.pack_experts(c.cuda(), s.cuda(), 4, 128) for c, s in (layers(E, I, n, 4, 128, 1), layers(E, I, n, 4, 128, 2), layers(E, n, I, 4, 128, 3))]
    x = [tokens(T, n, BF16, 4 + i).cuda() for i in range(2)]
    iw = [tuple(t.cuda() for t in chosen(T, E, k, 8 + i)) for i in range(2)]

    def step(i):
        return bk.experts(x[i], *packed, *iw[i])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(0)
    torch.cuda.current_stream().wait_stream(s)
    graphs, out = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.append(step(i))
        graphs.append(g)
    for r in range(4):
        for i in range(2):
            x[i].copy_(tokens(T, n, BF16, 20 + 2 * r + i))
            ni, nw = chosen(T, E, k, 40 + 2 * r + i, none=0.2)
            iw[i][0].copy_(ni)
            iw[i][1].copy_(nw)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i], step(i))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_block_of_rounded_layers(T):
    """A step through a block: norm, the fused projection with adapters, head norms with positions; norm, router, experts.
    Each operator against the 64-bit form of its own inputs."""
    from test_gpu_head_norm import check as check_heads
    from test_gpu_lora import check as check_lora
    from test_gpu_route import form64 as route64
    n, hq, hk, d, r, R, E, k, I = 256, 4, 2, 64, 8, 3, 8, 2, 128
    g = gen(T)
    m = (hq + 2 * hk) * d
    h, res = torch.randn(T, n, generator=g).to(BF16).cuda(), torch.randn(T, n, generator=g).to(BF16).cuda()
    proj, ps = layers(1, m, n, 4, 128, 1)
    w = bk.pack(proj[0].cuda(), ps[0].cuda(), 4, 128)
    a, b = (torch.randn(R, r, n, generator=g) * 0.05).to(BF16), torch.randn(R, m, r, generator=g).to(BF16)
    ids = torch.randint(-1, R, (T,), generator=g, dtype=torch.int32)
    nr = bk.rmsnorm(h, residual=res, out_dtype=I8)
    base = bk.matvec(nr.y, w, x_scale=nr.scale)
    qkv = bk.lora(nr.y, a.cuda(), b.cuda(), ids.cuda(), base=base, x_scale=nr.scale)
    check_lora(qkv, nr.y.cpu(), a, b, ids, base.cpu(), None, nr.scale.cpu())
    q, kk = qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    gain, pos = (1 + 0.1 * torch.randn(d, generator=g)).to(BF16), torch.randint(0, 100000, (T,), generator=g)
    freq = 10000.0 ** (-torch.arange(d // 2).float() / (d // 2))
    yq, yk = bk.head_norm(q, kk, gain.cuda(), gain.cuda(), pos.cuda(), freq.cuda())
    check_heads(yq, q.cpu(), gain, pos, freq, 1e-6, True, "half")
    check_heads(yk, kk.cpu(), gain, pos, freq, 1e-6, True, "half")
    n2 = bk.rmsnorm(yq.reshape(T, n), residual=nr.sum)
    router = torch.randn(E, n, generator=g).cuda()
    logits = n2.y.float() @ router.t()
    ei, ew = bk.route(logits, k)
    ri, rw = route64(logits.cpu(), k, "softmax", None, True, 1.0)
    assert torch.equal(ei.cpu(), ri) and float((ew.cpu().double() - rw).abs().max()) < 66 * U
    gate, up, down = layers(E, I, n, 4, 128, 2), layers(E, I, n, 4, 128, 3), layers(E, n, I, 4, 32, 4)
    packed = [bk.pack_experts(c.cuda(), s.cuda(), 4, gr) for (c, s), gr in ((gate, 128), (up, 128), (down, 32))]
    y = bk.experts(n2.y, *packed, ei, ew, out_dtype=F32)
    ref, tol = form64(n2.y.cpu(), None, (gate, up, down, 4, 128, 4, 32), ei.cpu(), ew.cpu(), "silu")
    assert bool(((y.cpu().double() - ref).abs() <= tol + (k + 1) * U * (ref.abs() + tol) * 2).all())


def test_offsets_past_2_31():
    """Rows of x and y more than 2^31 elements apart, and the last of many experts behind 2^31 bytes of codes in each matrix.
    The last expert's sums may meet in another order than the second's: 64 U of the result's norm."""
    n, I, E = 4096, 1024, 1000
    nb = [bk.LIB.bakron_packed_bytes(*s, 4, 128) for s in ((I, n), (I, n), (n, I))]
    assert all((E - 1) * b > 2 ** 31 for b in nb)
    two = [bk.pack_experts(c.cuda(), s.cuda(), 4, 128) for c, s in (layers(2, I, n, 4, 128, 1), layers(2, I, n, 4, 128, 2), layers(2, n, I, 4, 128, 3))]
    many = []
    for w, b in zip(two, nb):
        data = torch.zeros(E * b, dtype=torch.uint8, device="cuda")  # scales of 0 in between
        data[:b] = w.data[:b]
        data[(E - 1) * b:] = w.data[b:]
        many.append(bk.PackedExperts(data, E, w.m, w.n, 4, 128))
    g = gen(9)
    for T in (1, 2, 9, 40):  # 40: list tiles of 16
        x = torch.randn(T, n, generator=g).to(BF16).cuda()
        ids = torch.randint(0, 2, (T, 1), generator=g, dtype=torch.int32).cuda()
        ids[-1] = 1
        wt = torch.rand(T, 1, generator=g).cuda()
        y = bk.experts(x, *two, ids, wt, out_dtype=F32)
        z = bk.experts(x, *many, ids * (E - 1), wt, out_dtype=F32)
        assert float((y - z).norm()) <= 2.0 ** -18 * float(y.norm())
    # tiles of 64: many tokens of few slots
    T, k = 20, 64
    x = torch.randn(T, n, generator=g).to(BF16).cuda()
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    ids[:, 0], ids[:, 1] = 0, 1
    wt = torch.rand(T, k, generator=g).cuda()
    y, z = bk.experts(x, *two, ids, wt, out_dtype=F32), bk.experts(x, *many, torch.where(ids == 1, E - 1, ids), wt, out_dtype=F32)
    assert float((y - z).norm()) <= 2.0 ** -18 * float(y.norm())
    del many, data
    ld = (1 << 31) + 8
    for T in (2, 1):
        ids, wt = ids[:T, :2].contiguous(), wt[:T, :2].contiguous()
        xb = torch.empty((T - 1) * ld + n, dtype=BF16, device="cuda").as_strided((T, n), (ld, 1))
        xb.copy_(x[:T])
        yb = torch.empty((T - 1) * ld + n, dtype=BF16, device="cuda").as_strided((T, n), (ld, 1))
        assert torch.equal(bk.experts(xb, *two, ids, wt, out=yb).contiguous(), bk.experts(x[:T], *two, ids, wt))
    # more tokens: 18 rows, ld 2^28
    ld, T = (1 << 28) + 8, 18
    ids, wt = torch.randint(0, 2, (T, 1), generator=g, dtype=torch.int32).cuda(), torch.rand(T, 1, generator=g).cuda()
    xb = torch.empty((T - 1) * ld + n, dtype=I8, device="cuda").as_strided((T, n), (ld, 1))
    x8 = torch.randint(-127, 128, (T, n), generator=g, dtype=I8).cuda()
    xb.copy_(x8)
    yb = torch.empty((T - 1) * ld + n, dtype=BF16, device="cuda").as_strided((T, n), (ld, 1))
    assert torch.equal(bk.experts(xb, *two, ids, wt, out=yb).contiguous(), bk.experts(x8, *two, ids, wt))


@pytest.mark.parametrize("n,I", [(900, 1100), (1500, 1030), (4000, 1024), (7000, 1100), (9000, 1060), (7000, 100), (5000, 130)])
@pytest.mark.parametrize("T,bits,group", [(3, 4, 128), (7, 2, 32), (12, 4, 32)])
def test_second_product_grids(T, bits, group, n, I):
    """Every number of splits and of row tiles a workgroup, by the number of rows and columns."""
    check(T, 8, 3, n, I, 4, 128, bits, group, BF16, F32, none=0.1, seed=n + T)


@pytest.mark.parametrize("T,E,k", [(24, 1, 1), (25, 1, 1), (48, 4, 2), (50, 4, 2), (72, 6, 2), (17, 1, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16, I8])
def test_tokens_of_an_expert(T, E, k, dtype):
    """Around the border between list tiles of 16 and of 64 tokens, several tiles an expert."""
    check(T, E, k, 300, 200, 4, 128, 4, 64, dtype, F32, seed=T)


@pytest.mark.parametrize("n", [700, 2000, 6000])
@pytest.mark.parametrize("bits,group", [(4, 128), (4, 32), (2, 0), (1, 64)])
def test_list_tiles_of_16(n, bits, group):
    """The second product's workgroups of 8, 4 and 2 waves, by the number of rows."""
    check(24, 8, 2, n, 300, 4, 128, bits, group, BF16, F32, none=0.1, seed=n)
