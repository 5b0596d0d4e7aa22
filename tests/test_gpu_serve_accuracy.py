"""What the serving operators hold, on the GPU: fp32 sums for every type of tokens, against 64 bits.

The tolerances are bounds of the 2-norm of all results' errors. Roundings of a sum whose partial sums have random
signs add in squares, so these are far below the worst case of every element, and a type that is summed in fewer
bits, or a part of it left out, shows.
"""
import math

import pytest
import torch

import kronecker_hessian_rounding_amd as bk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def layer(m, n, bits, group, seed):
    g = gen(seed)
    codes = torch.randint(0, 2 ** bits, (m, n), generator=g, dtype=torch.uint8)
    return codes, torch.rand(m, -(-n // group) if group else 1, generator=g) + 0.25


def dense(codes, scales, bits, group):
    v = codes.double() - (2 ** bits - 1) / 2
    s = scales.double()
    return v * (s.repeat_interleave(group, 1)[:, :codes.shape[1]] if group else s)


def activations(T, n, dtype, seed):
    """Values with a few large channels; in 8 bits each token's largest magnitude takes the top value."""
    g = gen(seed)
    x = torch.randn(T, n, generator=g) * (0.5 + torch.randn(n, generator=g).square())
    if dtype == I8:
        return (x / (x.abs().amax(1, keepdim=True) / 127)).round().clamp(-127, 127).to(I8)
    return (x / (x.abs().amax(1, keepdim=True) / 448)).to(E4M3) if dtype == E4M3 else x.to(dtype)


def wide_rows(T, n, dtype, seed):
    """Magnitudes spread evenly over the type's octaves (bf16 and fp32: over 60 of them), both signs."""
    g = gen(seed)
    lo, hi = {E4M3: (-9.0, 8.8), F16: (-24.0, 15.0), BF16: (-40.0, 20.0), F32: (-40.0, 20.0)}[dtype]
    x = torch.exp2(torch.rand(T, n, generator=g) * (hi - lo) + lo)
    return torch.where(torch.rand(T, n, generator=g) < 0.5, x, -x).to(dtype)


def norm_bound(n, dtype, group):
    """The relative 2-norm of the error. The products are exact. A scale's unit (a chunk of 128 columns, or 32 where
    groups are shorter) takes k matrix operations, each off by at most 2 U of its sum, so 2 U / sqrt(3) in the mean
    square: 2 U sqrt(k / 3) (int8: exact integers, 0). The N units' sums meet in N additions, each rounded to nearest
    (U / sqrt(3)) and none of a larger partial sum than the result's norm: U sqrt(N / 3). Adding the waves' sums: 2 U."""
    steps = 1 if group and group < 128 else 4
    k = 0 if dtype == I8 else steps * (3 if dtype == F32 else 1)
    return U * (2 * math.sqrt(k / 3) + math.sqrt(n / (32 * steps) / 3) + 2)


@pytest.mark.parametrize("rows", [activations, wide_rows])
@pytest.mark.parametrize("bits,group", [(4, 32), (4, 128), (4, 0), (3, 64), (2, 64), (2, 0), (1, 0)])
@pytest.mark.parametrize("T", [1, 4, 7, 16, 40, 100])
@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
def test_matvec_holds_fp32_sums(dtype, T, bits, group, rows):
    if rows is wide_rows and dtype == I8:
        rows = activations
    m, n = 300, 4096
    codes, scales = layer(m, n, bits, group, T)
    x = rows(T, n, dtype, T + 1)
    y = bk.matvec(x.cuda(), bk.pack(codes.cuda(), scales.cuda(), bits, group), out_dtype=F32).cpu().double()
    ref = x.double() @ dense(codes, scales, bits, group).t()
    assert float((y - ref).norm() / ref.norm()) <= norm_bound(n, dtype, group)


@pytest.mark.parametrize("bits,group", [(4, 0), (4, 32), (2, 0), (2, 64)])
@pytest.mark.parametrize("T", [1, 5, 20, 100])
def test_matvec_e4m3_smallest_beside_largest(T, bits, group):
    """448 and 127 of the smallest value, 2^-9, in a chunk: their sum takes 25 bits below which nothing is left, and
    every partial sum of it is a multiple of 2^-10 below 2^14, so the result is exact."""
    x = torch.full((T, 128), 2.0 ** -9)
    x[torch.arange(T), (torch.arange(T) * 37) % 128] = 448.0
    codes = torch.full((16, 128), 2 ** bits - 1, dtype=torch.uint8)
    scales = torch.ones(16, 128 // group if group else 1)
    y = bk.matvec(x.to(E4M3).cuda(), bk.pack(codes.cuda(), scales.cuda(), bits, group), out_dtype=F32).cpu().double()
    assert torch.equal(y, torch.full((T, 16), (448 + 127 * 2.0 ** -9) * (2 ** bits - 1) / 2, dtype=torch.float64))


@pytest.mark.parametrize("bits,group", [(4, 0), (4, 32), (2, 0), (2, 32)])
@pytest.mark.parametrize("T", [1, 5, 16, 20, 50, 100, 300])
def test_matvec_every_bit_of_an_fp32_token(T, bits, group):
    """One value of 24 bits a row, in every column in turn, against weights of -1/2 and 1/2: the results are halves of
    the values, exact, whatever the launch; a piece of x that is lost or misplaced shows."""
    m, n = 40, 141
    g = gen(T)
    codes = torch.randint(2 ** (bits - 1) - 1, 2 ** (bits - 1) + 1, (m, n), generator=g, dtype=torch.uint8)
    ones = torch.ones(m, -(-n // group) if group else 1)
    w, v = bk.pack(codes.cuda(), ones.cuda(), bits, group), dense(codes, ones, bits, group)
    for first in range(0, n, T):
        value = (torch.randint(2 ** 23, 2 ** 24, (T,), generator=g) | 1).float() * 2.0 ** -20
        col = (first + torch.arange(T)) % n
        x = torch.zeros(T, n)
        x[torch.arange(T), col] = value
        y = bk.matvec(x.cuda(), w).cpu().double()
        assert torch.equal(y, value.double()[:, None] * v[:, col].t())


@pytest.mark.parametrize("T", [1, 12, 40])
def test_matvec_fp32_tokens_near_the_smallest(T):
    """An fp32 value is taken to a multiple of 2^-133 towards zero: itself from 2^-110 on, and never more than 2^-133
    off. Weights of 1/2 and scales of 2^20 keep the results normal, so they are exact."""
    w = bk.pack(torch.full((16, 32), 8, dtype=torch.uint8).cuda(), torch.full((16,), 2.0 ** 20).cuda(), 4)
    g = gen(T)
    for e in (-149, -140, -133, -126, -120, -111, -110, -100):
        x = torch.zeros(T, 32, dtype=torch.float64)
        x[:, 5] = (1 + torch.rand(T, generator=g, dtype=torch.float64)) * 2.0 ** e
        x = x.float()
        y = bk.matvec(x.cuda(), w).cpu().double() / 2.0 ** 19
        held = (x.double() * 2.0 ** 133).trunc() / 2.0 ** 133
        assert torch.equal(y, held[:, 5:6].expand(T, 16)), e
        assert e < -110 or torch.equal(held, x.double())


def hadamard(b):
    h = torch.ones(1, 1, dtype=torch.float64)
    while len(h) < b:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h


def signs(seed, n):
    out = []
    for i in range(1, n + 1):
        z = (seed + i * 0x9E3779B97F4A7C15) % 2 ** 64
        z = (z ^ z >> 30) * 0xBF58476D1CE4E5B9 % 2 ** 64
        z = (z ^ z >> 27) * 0x94D049BB133111EB % 2 ** 64
        out.append(-1.0 if (z ^ z >> 31) >> 63 else 1.0)
    return torch.tensor(out, dtype=torch.float64)


def rotation(seed, n):
    """U = (I (x) H_b / sqrt(b)) diag(signs), b the largest power of two that divides n."""
    b = n & -n
    return torch.block_diag(*[hadamard(b)] * (n // b)) / math.sqrt(b) * signs(seed, n)


@pytest.mark.parametrize("bits,q", [(4, I8), (4, E4M3), (4, BF16), (3, F32), (2, I8), (2, E4M3), (1, F16)])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_rotated_layer_chain(T, bits, q):
    """A layer rotated, rounded by the solve, packed and used: norm with rotation, product, rotation back, in 64 bits.

    First from the norm's own output, with fp32 tolerances: the product's (norm_bound, and U for the token's scale),
    and a rounding a stage and for the scale of the rotation back, which is orthogonal. Then from the layer's inputs:
    the rotation keeps 2-norms, so what the rounding of the activations does is at most ||W'|| times its 2-norm."""
    m, n = 192, 320
    g = gen(bits)
    W = torch.randn(m, n, generator=g).cuda()
    HI = bk.hessian_accum(torch.randn(900, n, generator=g).cuda())
    HO = bk.hessian_accum(torch.randn(700, m, generator=g).cuda())
    bk.rotate_layer(W, HI, HO, seed_O=11, seed_I=22)
    (LO, DO), (LI, DI) = bk.ldl_pair(HO, HI)
    res = bk.solve(W, LO, LI, bits, D_O=DO, D_I=DI)
    w = bk.pack(res.codes, res.scales, bits)
    x, r = torch.randn(T, n, generator=g).to(BF16), torch.randn(T, n, generator=g).to(BF16)
    gain = 1 + 0.1 * torch.randn(n, generator=g)
    nr = bk.rmsnorm(x.cuda(), gain.cuda(), residual=r.cuda(), rotate_seed=22, out_dtype=q)
    y = bk.rht(bk.matvec(nr.y, w, x_scale=nr.scale, out_dtype=F32), 1, 11, transpose=True).cpu().double()

    wq = dense(res.codes.cpu(), res.scales.cpu().reshape(-1, 1), bits, 0)
    back = rotation(11, m)
    held = nr.y.cpu().double() * (1.0 if nr.scale is None else nr.scale.cpu().double()[:, None])
    own = held @ wq.t() @ back  # rows times U_O: U_O^T y
    fp32 = norm_bound(n, q, 0) + U + U * (math.log2(m & -m) + 1)
    assert float((y - own).norm()) <= fp32 * float(own.norm())

    h = x.double() + r.double()
    v = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * gain.double() @ rotation(22, n).t()
    full = v @ wq.t() @ back
    lost = (v - held).norm(dim=1)
    half = {I8: 0.5 / 127, E4M3: 2.0 ** -4, BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}[q]
    # the norm's own fp32 error: n / 64 + 16 roundings of the sum, halved by the root, 8 more, one a stage
    norm = U * (n / 128 + 16 + math.log2(n & -n) + 3)
    top = v.abs().amax(1, keepdim=True) if q == I8 else torch.maximum(v.abs(), v.abs().amax(1, keepdim=True) / 448 / 8)
    assert bool((lost <= half * top.expand_as(v).norm(dim=1) * (1 + 2.0 ** -10) + norm * v.norm(dim=1)).all())
    limit = torch.linalg.matrix_norm(wq, 2) * lost + fp32 * own.norm(dim=1)
    assert bool(((y - full).norm(dim=1) <= limit).all())
    assert bool((limit <= 0.25 * full.norm(dim=1)).all())  # and that is small beside the result
