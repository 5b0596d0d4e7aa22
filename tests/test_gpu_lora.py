"""lora on the GPU against its 64-bit form.

Tolerance: u = 2^-24. Products of 8- and 16-bit values are exact in fp32, those of fp32 have one rounding. A sum of n terms
over 8 waves, at most n / 8 + 8 fp32 roundings of at most 2 u each in a row (the matrix core's being no better than
truncation), gives u_k; the second product has r more, then the factors 3 and the base's addition 1. A 16-bit
output takes u with 17 bits (2^-17), an fp32 one with 22 (2^-22). All relative to the sum of magnitudes; then half a step of
the output's type.
"""
import pytest
import torch

import kronecker_hessian_rounding_amd as bk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn
COMBOS = [(F32, F32), (F16, F16), (BF16, BF16), (I8, F16), (I8, BF16), (E4M3, F16), (E4M3, BF16)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inputs(T, n, m, r, R, xt, wt, seed=0, none=0.2, run=1):
    g = gen(seed)
    x = torch.randint(-127, 128, (T, n), generator=g, dtype=I8) if xt == I8 else torch.randn(T, n, generator=g).to(xt)
    a, b = (torch.randn(R, r, n, generator=g) * n ** -0.5).to(wt), torch.randn(R, m, r, generator=g).to(wt)
    ids = torch.randint(0, R, (-(-T // run),), generator=g, dtype=torch.int32)
    ids[torch.rand(ids.numel(), generator=g) < none] = -1
    return x, a, b, ids.repeat_interleave(run)[:T].contiguous(), torch.rand(R, generator=g) + 0.5, torch.rand(T, generator=g) + 0.5


def form64(x, a, b, ids, base, scales, xs):
    """(result, sum of magnitudes) in 64 bits."""
    T, m = x.shape[0], b.shape[1]
    y = torch.zeros(T, m, dtype=torch.float64) if base is None else base.double()
    mag = y.abs()
    for t in range(T):
        i = int(ids[t])
        if 0 <= i < a.shape[0]:
            f = (1.0 if scales is None else float(scales[i])) * (1.0 if xs is None else float(xs[t]))
            A, B, v = a[i].double(), b[i].double(), x[t].double()
            y[t] = y[t] + f * (B @ (A @ v))
            mag[t] = mag[t] + f * (B.abs() @ (A.abs() @ v.abs()))
    return y, mag


def check(y, x, a, b, ids, base, scales, xs):
    ref, mag = form64(x, a, b, ids, base, scales, xs)
    fi = torch.finfo(y.dtype)
    n, r = x.shape[1], a.shape[1]
    piece = 2.0 ** -22 if y.dtype == F32 else 2.0 ** -17
    tol = mag * (2 * U * (n / 8 + 8 + r + 4) + piece) + ref.abs() * fi.eps / 2 + fi.tiny * fi.eps
    err = (y.cpu().double() - ref).abs()
    assert y.shape == ref.shape and bool((err <= tol).all()), float((err / tol).max())


def call(x, a, b, ids, base=None, scales=None, xs=None, **kw):
    dev = [None if t is None else t.cuda() for t in (x, a, b, ids, base, scales, xs)]
    return bk.lora(dev[0], dev[1], dev[2], dev[3], base=dev[4], scales=dev[5], x_scale=dev[6], **kw)


@pytest.mark.parametrize("xt,wt", COMBOS)
@pytest.mark.parametrize("T,n,m,r,R", [(1, 1, 1, 1, 1), (1, 4096, 512, 16, 3), (2, 64, 64, 4, 2), (3, 63, 65, 13, 2), (7, 128, 200, 8, 3),
                                       (16, 640, 64, 17, 4), (17, 100, 130, 32, 40), (33, 1027, 77, 33, 5), (40, 300, 700, 64, 2),
                                       (5, 200, 100, 100, 2), (19, 96, 40, 130, 3), (3, 40, 70, 512, 2), (100, 50, 30, 16, 100),
                                       (6, 31, 1100, 20, 2), (4, 16, 33, 64, 1)])
def test_against_64_bits(T, n, m, r, R, xt, wt):
    x, a, b, ids, scales, xs = inputs(T, n, m, r, R, xt, wt, seed=T + r)
    base = torch.randn(T, m, generator=gen(1))
    check(call(x, a, b, ids, base, scales, xs, out_dtype=F32), x, a, b, ids, base, scales, xs)
    for out in (F16, BF16):
        bb = base.to(out)
        check(call(x, a, b, ids, bb, scales, xs), x, a, b, ids, bb, scales, xs)
    check(call(x, a, b, ids, out_dtype=F32), x, a, b, ids, None, None, None)


@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("T,run,m,r", [(16, 16, 300, 12), (64, 1, 2000, 16), (65, 1, 2000, 16), (300, 37, 200, 24), (5000, 500, 96, 12), (4200, 1, 64, 8),
                                       (70, 1, 9000, 64), (128, 1, 500, 32), (129, 1, 2000, 32), (300, 1, 500, 20), (1, 1, 300, 64), (40, 3, 700, 48), (500, 60, 333, 128), (130, 3, 4500, 100), (200, 7, 129, 130), (2100, 33, 64, 5)])
def test_launch_shapes(T, run, m, r, xt, wt):
    """Runs of one adapter and every token with another; few and many tiles of tokens; many rows; every rank's tiles."""
    x, a, b, ids, scales, _ = inputs(T, 72, m, r, 9, xt, wt, seed=T, run=run)
    base = torch.randn(T, m, generator=gen(2)).to(wt)
    check(call(x, a, b, ids, base, scales), x, a, b, ids, base, scales, None)


@pytest.mark.parametrize("xt,wt,bt,yt", [(BF16, BF16, BF16, BF16), (BF16, BF16, F32, BF16), (F16, F16, F16, F32), (F32, F32, BF16, F32),
                                         (F32, F32, F32, F16)])
@pytest.mark.parametrize("m", [127, 128, 129, 191, 256, 383, 1100])
@pytest.mark.parametrize("r", [16, 13, 40, 88])
def test_row_blocks(m, r, xt, wt, bt, yt):
    """More tokens, rows in whole blocks and behind them, base and result of other types than the adapters'."""
    x, a, b, ids, scales, _ = inputs(203, 100, m, r, 5, xt, wt, seed=m + r, run=70)
    base = torch.randn(203, m, generator=gen(2)).to(bt)
    check(call(x, a, b, ids, base, scales, out_dtype=yt), x, a, b, ids, base, scales, None)


@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (F32, F32), (I8, F16)])
@pytest.mark.parametrize("T,n,m,r", [(1, 4096, 130, 64), (41, 13056, 100, 64), (140, 6661, 90, 16), (594, 6661, 70, 40), (822, 7424, 66, 13), (16, 6016, 128, 100)])
def test_columns_in_splits(T, n, m, r, xt, wt):
    """Long rows, whose columns several workgroups share: every split's columns once."""
    x, a, b, ids, scales, xs = inputs(T, n, m, r, 3, xt, wt, seed=n, run=9)
    base = torch.randn(T, m, generator=gen(2))
    check(call(x, a, b, ids, base, scales, xs, out_dtype=F32), x, a, b, ids, base, scales, xs)


@pytest.mark.parametrize("T", [21, 250])
@pytest.mark.parametrize("xt,wt", COMBOS)
def test_exact_on_integers(xt, wt, T):
    """Small integers: every partial sum is an integer below 2^24, so the result is exact, whatever the order."""
    n, m, r, R = 150, 140, 20, 4
    g = gen(4)
    x = torch.randint(-4, 5, (T, n), generator=g).to(torch.int8 if xt == I8 else F32).to(xt)
    a, b = (torch.randint(-2, 3, s, generator=g).float().to(wt) for s in ((R, r, n), (R, m, r)))
    ids = torch.randint(-1, R, (T,), generator=g, dtype=torch.int32)
    base = torch.randint(-50, 51, (T, m), generator=g).float()
    y = call(x, a, b, ids, base, torch.full((R,), 2.0), out_dtype=F32)
    assert torch.equal(y.cpu().double(), form64(x, a, b, ids, base, torch.full((R,), 2.0), None)[0])


@pytest.mark.parametrize("T", [37, 171])
@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (F32, F32), (I8, F16), (E4M3, BF16)])
def test_strided_rows_and_place(xt, wt, T):
    """Column ranges of wider buffers at odd offsets, in place on the base; nothing else is written."""
    n, m, r, R = 131, 270, 16, 3
    x, a, b, ids, scales, xs = inputs(T, n, m, r, R, xt, wt, seed=6, run=4)
    base = torch.randn(T, m, generator=gen(7)).to(wt)
    ref = call(x, a, b, ids, base, scales, xs)
    xb = torch.zeros(T, n + 7, dtype=xt, device="cuda")
    xb[:, 3:3 + n] = x.cuda()
    yb = torch.full((T + 1, m + 9), 7.0, dtype=wt, device="cuda")
    y = yb[:T, 5:5 + m]
    y.copy_(base)
    got = bk.lora(xb[:, 3:3 + n], a.cuda(), b.cuda(), ids.cuda(), base=y, scales=scales.cuda(), x_scale=xs.cuda(), out=y)
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, ref)
    y.fill_(7.0)
    assert bool((yb == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T", [20, 140])
def test_tokens_without_an_adapter(T, dtype):
    """Ids on either side of the range leave the base as it is; a NaN or infinity of one request stays its own."""
    x, a, b, ids, scales, _ = inputs(T, 96, 80, 16, 3, dtype, dtype, none=0.0)
    base = torch.randn(T, 80, generator=gen(8)).to(dtype)
    ids[3], ids[4], ids[5], ids[6] = -1, 3, -2 ** 31, 2 ** 31 - 1
    y = call(x, a, b, ids, base, scales)
    assert torch.equal(y[3:7].cpu(), base[3:7])
    check(y, x, a, b, ids, base, scales, None)
    assert bool((call(x, a, b, torch.full_like(ids, -1), out_dtype=BF16) == 0).all())
    ids[:] = torch.arange(T, dtype=torch.int32) % 3
    ref = call(x, a, b, ids, base, scales)
    x[1, 5] = float("nan")
    a[2, 3, 7] = float("inf")
    b[2, 9, 1] = float("nan")
    y = call(x, a, b, ids, base, scales)
    clean = [t for t in range(T) if t != 1 and t % 3 != 2]
    assert torch.equal(y[clean], ref[clean]) and bool(torch.isnan(y[1]).all())


@pytest.mark.parametrize("T", [50, 190])
def test_other_rows_do_not_matter(T):
    """A token's result stays bit for bit when the other rows, and their adapters, change."""
    x, a, b, ids, scales, _ = inputs(T, 700, 333, 24, 5, BF16, BF16, seed=9)
    base = torch.randn(T, 333, generator=gen(9)).to(BF16)
    y = call(x, a, b, ids, base, scales)
    x2, _, _, ids2, _, _ = inputs(T, 700, 333, 24, 5, BF16, BF16, seed=10)
    for t in (0, 17, 49):
        x3, ids3 = x2.clone(), ids2.clone()
        x3[t], ids3[t] = x[t], ids[t]
        assert torch.equal(call(x3, a, b, ids3, base, scales)[t], y[t])


def test_offsets_past_2_31():
    ld = (1 << 31) + 8
    x, a, b, ids, _, _ = inputs(2, 64, 64, 8, 2, BF16, BF16, none=0.0)
    xb = torch.empty(ld + 64, dtype=BF16, device="cuda").as_strided((2, 64), (ld, 1))
    xb.copy_(x)
    yb = torch.empty(ld + 64, dtype=BF16, device="cuda").as_strided((2, 64), (ld, 1))
    assert torch.equal(bk.lora(xb, a.cuda(), b.cuda(), ids.cuda(), out=yb).contiguous(), call(x, a, b, ids))
    # the last adapter behind 2^31 elements
    R = (1 << 31) // (64 * 64) + 2
    big = torch.zeros(R, 64, 64, dtype=BF16, device="cuda")
    big[R - 1] = torch.randn(64, 64, generator=gen(3)).to(BF16)
    ids = torch.tensor([R - 1, 0], dtype=torch.int32, device="cuda")
    y = bk.lora(x.cuda(), big, big, ids, out_dtype=F32)
    small = bk.lora(x.cuda(), big[R - 1:].clone(), big[R - 1:].clone(), ids - (R - 1), out_dtype=F32)
    assert torch.equal(y[:1], small[:1]) and bool((y[1] == 0).all())


def test_empty():
    x, a, b, ids, _, _ = inputs(1, 64, 32, 8, 2, BF16, BF16)
    y = bk.lora(x[:0].cuda(), a.cuda(), b.cuda(), ids[:0].cuda())
    assert y.shape == (0, 32)


def test_refusals():
    x, a, b, ids, scales, xs = (t.cuda() for t in inputs(4, 64, 48, 8, 2, BF16, BF16))
    base = torch.zeros(4, 48, dtype=BF16, device="cuda")
    bad = [lambda: bk.lora(x.float(), a, b, ids), lambda: bk.lora(x, a.half(), b.half(), ids), lambda: bk.lora(x, a, b.float(), ids),
           lambda: bk.lora(x[:, :63], a, b, ids), lambda: bk.lora(x, a[:1], b, ids), lambda: bk.lora(x, a[:, :7].contiguous(), b, ids),
           lambda: bk.lora(x, a[:, :7], b, ids), lambda: bk.lora(x, a.transpose(1, 2), b, ids), lambda: bk.lora(x, a[0], b[0], ids),
           lambda: bk.lora(x, a, b, ids.long()), lambda: bk.lora(x, a, b, ids[:3]), lambda: bk.lora(x, a, b, ids.cpu()),
           lambda: bk.lora(x, a, b, ids, base=base[:3]), lambda: bk.lora(x, a, b, ids, base=base.double()),
           lambda: bk.lora(x, a, b, ids, scales=scales[:1]), lambda: bk.lora(x, a, b, ids, x_scale=xs[:3]),
           lambda: bk.lora(x, a, b, ids, out=base[:, :47]), lambda: bk.lora(x, a, b, ids, out=base, out_dtype=F32),
           lambda: bk.lora(x, a, b, ids, out_dtype=I8), lambda: bk.lora(x.cpu(), a, b, ids), lambda: bk.lora(x, a.cpu(), b, ids),
           lambda: bk.lora(x.to(E4M3), a.float(), b.float(), ids), lambda: bk.lora(x, a[:0], b[:0], ids),
           lambda: bk.lora(x, torch.zeros(1, 513, 64, dtype=BF16, device="cuda"), torch.zeros(1, 4, 513, dtype=BF16, device="cuda"), ids)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % i)
    for f in (lambda: bk.lora(x, a, b, ids, out=x[:, :48]), lambda: bk.lora(x[:3], a, b, ids[:3].clone(), base=base[:3], out=base[1:])):
        with pytest.raises(bk.BakronError):
            f()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [5, 180])
def test_values_over_the_types_range(T, dtype):
    """u far above and below what 16 bits hold in fp16, and zeros: the second product keeps them."""
    n, m, r, R = 64, 96, 16, 4
    x, a, b, _, _, _ = inputs(T, n, m, r, R, dtype, dtype, none=0.0)
    ids = torch.arange(T, dtype=torch.int32) % R
    a = a.float() * torch.tensor([1.0, 2.0 ** 12, 2.0 ** -12, 0.0])[:, None, None]
    xs = torch.where(torch.arange(T) % 3 == 0, 2.0 ** 20, 2.0 ** -20)
    a = a.to(dtype)
    check(call(x, a, b, ids, None, None, xs, out_dtype=F32), x, a, b, ids, None, None, xs)


@pytest.mark.parametrize("T", [1, 40, 200])
def test_stream_and_graph(T):
    x, a, b, ids, scales, _ = (t.cuda() for t in inputs(T, 512, 384, 16, 5, BF16, BF16))
    base = torch.randn(T, 384, device="cuda").to(BF16)

    def step():
        return bk.lora(x, a, b, ids, base=base, scales=scales)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for i in range(4):
        nx = inputs(T, 512, 384, 16, 5, BF16, BF16, seed=50 + i)
        x.copy_(nx[0])
        ids.copy_(nx[3])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step())


@pytest.mark.parametrize("rest", [100, 3000])
@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (I8, F16)])
def test_tokens_past_a_round_of_launches(rest, xt, wt):
    """More than 65536 tokens go through in rounds; the last one in one launch (100) or two (3000). Rows at the rounds' ends
    against 64 bits, and all against calls of 5000 tokens (whose sums start in other columns: twice the tolerance's part of those)."""
    T, n, m, r, R = 65536 + rest, 40, 24, 8, 3
    x, a, b, ids, scales, xs = inputs(T, n, m, r, R, xt, wt, seed=rest, none=0.1, run=7)
    base = torch.randn(T, m, generator=gen(1))
    xb = torch.zeros(T, n + 5, dtype=xt, device="cuda")
    xb[:, 2:2 + n] = x.cuda()
    yb = torch.full((T, m + 3), 9.0, device="cuda")
    args = dict(scales=scales.cuda(), out_dtype=F32)
    y = yb[:, 1:1 + m]
    bk.lora(xb[:, 2:2 + n], a.cuda(), b.cuda(), ids.cuda(), base=base.cuda(), x_scale=xs.cuda(), out=y, **args)
    for s in (slice(0, 40), slice(65536 - 70, 65536 + 100), slice(T - 90, T)):
        check(y[s], x[s], a, b, ids[s], base[s], scales, xs[s])
    for t0 in range(0, T, 5000):
        s = slice(t0, min(T, t0 + 5000))
        part = bk.lora(x[s].cuda(), a.cuda(), b.cuda(), ids[s].cuda(), base=base[s].cuda(), x_scale=xs[s].cuda(), **args)
        mag = base[s].abs() + 2 * 1.5 * 1.5 * n * r * x[s].float().abs().amax() * a.float().abs().amax() * b.float().abs().amax()
        assert bool(((y[s] - part).abs().cpu() <= 2 * U * (n / 8 + 8 + r + 4) * 2 * mag).all())
    y.fill_(9.0)
    assert bool((yb == 9.0).all())
