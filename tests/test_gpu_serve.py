"""The serving operators on the GPU (pack, matvec, rmsnorm) against plain 64-bit forms on the CPU.

Tolerances are bounds of the arithmetic, derived at each check: u = 2^-24 is half a step of
fp32, and an output type's half step is finfo.eps / 2.
"""
import numpy as np
import pytest
import torch

import kronecker_hessian_rounding_amd as bk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def layer(m, n, bits, group, seed, integer=False):
    g = gen(seed)
    codes = torch.randint(0, 2 ** bits, (m, n), generator=g, dtype=torch.uint8)
    ng = -(-n // group) if group else 1
    scales = torch.rand(m, ng, generator=g) + 0.25
    if integer:
        scales = torch.full((m, ng), 2.0)
    return codes, scales


def dense(codes, scales, bits, group):
    """The weights that the codes stand for, in 64 bits."""
    v = codes.double() - (2 ** bits - 1) / 2
    n = codes.shape[1]
    s = scales.double()
    return v * (s.repeat_interleave(group, 1)[:, :n] if group else s)


def tokens(T, n, dtype, seed, integer=False):
    g = gen(seed)
    if dtype == I8:
        return torch.randint(-127, 128, (T, n), generator=g, dtype=torch.int8)
    x = torch.randint(-8, 9, (T, n), generator=g).float() if integer else torch.randn(T, n, generator=g)
    return x.to(dtype)


def matvec_bound(x, xs, w, out_dtype):
    """|error| of a result: the products are exact; a sum of a chunk has at most 256 terms of at
    most 3 pieces (two fp32 roundings of at most 2 u each, the matrix core's being no better than
    truncation), the chunks' sums one addition and one product each per wave, at most n / 128 + 16,
    then the unit and the token's scale; the output is rounded once."""
    n = x.shape[1]
    a = x.double().abs() @ w.abs().t()
    y = x.double() @ w.t()
    if xs is not None:
        a, y = a * xs.double()[:, None], y * xs.double()[:, None]
    fi = torch.finfo(out_dtype)
    return y, a * 2 * U * (3 * min(n, 256) + n / 128 + 20) + y.abs() * fi.eps / 2 + fi.tiny


def check_matvec(T, m, n, bits, group, dtype, out_dtype, seed=0, scaled=True, view=None):
    codes, scales = layer(m, n, bits, group, seed)
    x = tokens(T, n, dtype, seed + 1)
    xs = torch.rand(T, generator=gen(seed + 2)) + 0.5 if scaled else None
    w = bk.pack(codes.cuda(), scales.cuda(), bits, group)
    xd = x.cuda() if view is None else view(x.cuda())
    y = bk.matvec(xd, w, x_scale=None if xs is None else xs.cuda(), out_dtype=out_dtype)
    assert y.shape == (T, m) and y.dtype == out_dtype
    ref, tol = matvec_bound(x, xs, dense(codes, scales, bits, group), out_dtype)
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), int((err > tol).sum()))


# ------------------------------------------------------------------ matvec
@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("bits", [1, 2, 3, 4])
@pytest.mark.parametrize("T,m,n,group", [(1, 1, 1, 0), (3, 20, 31, 0), (16, 33, 128, 32), (17, 64, 300, 64),
                                         (5, 48, 1025, 128), (2, 31, 2100, 256), (1, 130, 1111, 512)])
def test_matvec_exact_on_integers(T, m, n, group, bits, dtype):
    """Small integers and scales of 2: every partial sum is an integer below 2^24, so the result is exact."""
    codes, scales = layer(m, n, bits, group, 3, integer=True)
    x = tokens(T, n, dtype, 4, integer=True)
    w = bk.pack(codes.cuda(), scales.cuda(), bits, group)
    y = bk.matvec(x.cuda(), w, out_dtype=F32).cpu().double()
    ref = x.double() @ dense(codes, scales, bits, group).t()
    assert float(x.double().abs().max()) * 16 * n < 2 ** 24
    assert torch.equal(y, ref)


@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("T,m,n,bits,group", [
    (1, 256, 4096, 4, 128), (1, 100, 8192, 2, 0), (4, 80, 4096, 4, 32), (7, 67, 4013, 3, 64), (16, 64, 2048, 2, 64),
    (15, 64, 2048, 2, 32), (33, 96, 1024, 4, 128), (64, 128, 1152, 4, 256), (65, 130, 640, 2, 128),
    (130, 272, 513, 4, 0), (300, 140, 256, 4, 128), (257, 260, 1000, 4, 64), (129, 200, 777, 3, 32)])
def test_matvec_against_64_bits(T, m, n, bits, group, dtype):
    check_matvec(T, m, n, bits, group, dtype, F32)


# every launch shape: tokens 1, <= 4, 8, 16, 32, 48, 64, more; layers of few and of many row tiles; a row length
# that ends inside a chunk and inside 16 bytes, and rows shorter than 16 bytes
SHAPES = [(T, m) for T in (1, 3, 7, 13) for m in (40, 8200)] + \
         [(T, m) for T in (20, 33, 50, 64) for m in (50, 4200)] + \
         [(100, 130), (100, 8300), (300, 11100), (260, 8192)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("bits,group", [(4, 128), (4, 32), (2, 0), (2, 64)])
@pytest.mark.parametrize("T,m", SHAPES)
def test_matvec_launch_shapes(T, m, bits, group, dtype):
    n = 391
    codes, scales = layer(m, n, bits, group, T)
    x = tokens(T, n, dtype, T + 1)
    w = bk.pack(codes.cuda(), scales.cuda(), bits, group)
    buf = torch.zeros(T, n + 10, dtype=dtype, device="cuda")
    buf[:, 1:n + 1] = x.cuda()
    out = torch.full((T + 1, m + 5), -3.0, device="cuda")
    y = bk.matvec(buf[:, 1:n + 1], w, out=out[:T, 2:m + 2])
    # a sample of the rows, the last ones among them, so that the 64-bit product stays small
    rows = torch.unique(torch.cat([torch.arange(0, m, max(1, m // 150)), torch.arange(max(0, m - 20), m)]))
    ref, tol = matvec_bound(x, None, dense(codes[rows], scales[rows], bits, group), F32)
    assert bool(((y[:, rows.cuda()].cpu().double() - ref).abs() <= tol).all())
    out[:T, 2:m + 2] = -3.0
    assert bool((out == -3.0).all())


# workgroups of 64 rows x 32 tokens in one round and in several, of 64 x 48, 64 x 64 with columns split over 4 waves,
# 128 x 128 at exactly one a compute unit, and fp32 on both sides of two rounds
@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("bits,group", [(4, 128), (4, 32), (2, 0)])
@pytest.mark.parametrize("T,m", [(40, 4200), (32, 16400), (80, 8190), (100, 8190), (512, 8190), (129, 8190), (128, 8190)])
def test_matvec_launch_shapes_by_workgroups(T, m, bits, group, dtype):
    test_matvec_launch_shapes(T, m, bits, group, dtype)


@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("T", [1, 2, 5, 16, 30, 45, 64, 70, 600])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 15, 16, 17, 33, 127, 129])
def test_matvec_short_rows(n, T, dtype):
    """Rows down to one element, at the end of their buffer."""
    codes, scales = layer(35, n, 4, 0, n, integer=True)
    x = tokens(T, n, dtype, T, integer=True)
    y = bk.matvec(x.cuda(), bk.pack(codes.cuda(), scales.cuda(), 4), out_dtype=F32).cpu().double()
    assert torch.equal(y, x.double() @ dense(codes, scales, 4, 0).t())


@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("T", [1, 3, 16])
@pytest.mark.parametrize("n", [1025, 2051, 3077, 6151])
def test_matvec_unit_that_the_rows_end_cuts(n, T, dtype):
    """The last elements of a row weigh most: what another lane leaves in their place would show."""
    codes, scales = layer(18, n, 4, 0, n, integer=True)
    x = torch.ones(T, n)
    x[:, n - n % 4:] = 8.0
    y = bk.matvec(x.to(dtype).cuda(), bk.pack(codes.cuda(), scales.cuda(), 4), out_dtype=F32).cpu().double()
    assert torch.equal(y, x.double() @ dense(codes, scales, 4, 0).t())


@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("bits,group", [(4, 0), (4, 32), (2, 64)])
@pytest.mark.parametrize("T", [1, 4, 8, 16])
@pytest.mark.parametrize("n", [4100, 8197, 10239])
def test_matvec_staging_is_reused(n, T, bits, group, dtype):
    """Rows that pass several times through a wave's staging area and end inside 16 bytes: exact, as above."""
    codes, scales = layer(20, n, bits, group, n, integer=True)
    x = tokens(T, n, dtype, T, integer=dtype != I8)
    if dtype == I8:
        x = (x.int() % 9 - 4).to(I8)
    y = bk.matvec(x.cuda(), bk.pack(codes.cuda(), scales.cuda(), bits, group), out_dtype=F32).cpu().double()
    assert float(x.double().abs().max()) * 16 * n < 2 ** 24
    assert torch.equal(y, x.double() @ dense(codes, scales, bits, group).t())


@pytest.mark.parametrize("out_dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T", [1, 9, 40, 200])
def test_matvec_output_types(T, out_dtype):
    check_matvec(T, 77, 500, 4, 128, BF16, out_dtype, scaled=False)


@pytest.mark.parametrize("dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("T", [1, 6, 50, 140])
def test_matvec_rows_of_a_wider_buffer(T, dtype):
    """Odd leading dimensions and first columns: rows that start at any element."""
    def view(x):
        buf = torch.full((T, x.shape[1] + 7), 99, dtype=F32, device="cuda").to(x.dtype)
        buf[:, 3:3 + x.shape[1]] = x
        return buf[:, 3:3 + x.shape[1]]
    check_matvec(T, 50, 771, 4, 64, dtype, F32, view=view)


@pytest.mark.parametrize("T", [1, 20, 150])
def test_matvec_writes_its_own_columns_only(T):
    codes, scales = layer(45, 200, 4, 0, 1)
    w = bk.pack(codes.cuda(), scales.cuda(), 4)
    x = tokens(T, 200, BF16, 2).cuda()
    buf = torch.full((T + 2, 60), -7.0, device="cuda")
    bk.matvec(x, w, out=buf[1:T + 1, 5:50])
    ref = bk.matvec(x, w, out_dtype=F32)
    assert torch.equal(buf[1:T + 1, 5:50], ref)
    buf[1:T + 1, 5:50] = -7.0
    assert bool((buf == -7.0).all())


@pytest.mark.parametrize("T", [1, 3, 18, 90, 200])
@pytest.mark.parametrize("dtype", [F32, F16, BF16, E4M3])
def test_matvec_not_finite(T, dtype):
    """Infinities and NaN reach the token they are in as the formula says, and no other token. Columns
    past the end of a row (NaN here) are not read as x."""
    codes, scales = layer(40, 130, 4, 32, 5)
    buf = torch.full((T, 140), float("nan"))
    buf[:, :130] = tokens(T, 130, F32, 6)
    if dtype != E4M3:
        buf[0, 5] = float("inf")
        if T > 2:
            buf[2, 100], buf[2, 40] = float("inf"), float("-inf")
    if T > 1:
        buf[1, 129] = float("nan")
    x = buf.to(dtype)[:, :130]
    y = bk.matvec(buf.to(dtype).cuda()[:, :130], bk.pack(codes.cuda(), scales.cuda(), 4, 32), out_dtype=F32).cpu()
    w = dense(codes, scales, 4, 32)
    ref = (x.double()[:, None, :] * w[None]).sum(2)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(torch.isinf(y), torch.isinf(ref))
    inf = torch.isinf(ref)
    assert torch.equal(y[inf].double(), ref[inf])


def test_matvec_fp32_special_values():
    """NaN payloads in the low bits, subnormals and the largest fp32 values keep their meaning."""
    codes = torch.full((16, 64), 8, dtype=torch.uint8)  # v = 1/2
    w = bk.pack(codes.cuda(), torch.ones(16).cuda(), 4)
    x = torch.zeros(4, 64)
    x[0, 3] = torch.tensor([0x7F800001], dtype=torch.int32).view(F32)[0]
    x[1, 3] = 3.0e38
    x[2, 3] = 1.0 + 2.0 ** -23
    x[3, 3] = 2.0 ** -100 * (1 + 2.0 ** -23)
    y = bk.matvec(x.cuda(), w).cpu()
    assert bool(torch.isnan(y[0]).all())
    assert torch.equal(y[1:, 0], x[1:, 3] / 2)


def test_matvec_scales_of_zero_and_infinity():
    codes, _ = layer(16, 256, 4, 128, 7)
    scales = torch.ones(16, 2)
    scales[3] = 0.0
    scales[5, 1] = float("inf")
    x = tokens(2, 256, BF16, 8)
    y = bk.matvec(x.cuda(), bk.pack(codes.cuda(), scales.cuda(), 4, 128), out_dtype=F32).cpu()
    v = codes.double() - 7.5
    part = x.double()[:, 128:] @ v[5, 128:]
    assert bool((y[:, 3] == 0).all())
    assert torch.equal(y[:, 5].double(), torch.where(part > 0, float("inf"), float("-inf")).double())
    ok = [i for i in range(16) if i not in (5,)]
    assert bool(torch.isfinite(y[:, ok]).all())


def test_matvec_empty_and_single():
    codes, scales = layer(20, 96, 4, 0, 1)
    w = bk.pack(codes.cuda(), scales.cuda(), 4)
    assert bk.matvec(torch.empty(0, 96, dtype=BF16, device="cuda"), w).shape == (0, 20)
    x = tokens(1, 96, BF16, 2).cuda()
    y = bk.matvec(x[0], w)
    assert y.shape == (20,) and torch.equal(y, bk.matvec(x, w)[0])
    out = torch.empty(20, dtype=F32, device="cuda")
    assert torch.equal(bk.matvec(x[0], w, out=out), bk.matvec(x, w, out_dtype=F32)[0])


@pytest.mark.parametrize("T", [1, 16, 48, 200])
@pytest.mark.parametrize("dtype", [F32, BF16, I8])
def test_matvec_token_depends_on_its_row_only(T, dtype):
    """The same token gives the same bits whatever the other rows hold, and a call repeats bit for bit."""
    codes, scales = layer(96, 1000, 4, 128, 1)
    w = bk.pack(codes.cuda(), scales.cuda(), 4, 128)
    x = tokens(T, 1000, dtype, 2).cuda()
    y = bk.matvec(x, w, out_dtype=F32)
    assert torch.equal(y, bk.matvec(x, w, out_dtype=F32))
    z = x.flip(0).contiguous()
    assert torch.equal(bk.matvec(z, w, out_dtype=F32).flip(0), y)


@pytest.mark.parametrize("dtype,out_dtype", [(I8, BF16), (BF16, F32)])
def test_matvec_offsets_past_2_31(dtype, out_dtype):
    """Rows whose byte offsets pass 2^31 and 2^32 in x and y."""
    codes, scales = layer(40, 100, 4, 0, 1)
    w = bk.pack(codes.cuda(), scales.cuda(), 4)
    ld = (1 << 31) + 72
    small = tokens(3, 100, dtype, 2).cuda()
    buf = torch.empty(2 * ld + 100, dtype=dtype, device="cuda")
    x = buf.as_strided((3, 100), (ld, 1))
    x.copy_(small)
    ybuf = torch.empty(2 * ld + 40, dtype=out_dtype, device="cuda")
    out = ybuf.as_strided((3, 40), (ld, 1))
    bk.matvec(x, w, out=out)
    assert torch.equal(out.contiguous(), bk.matvec(small, w, out_dtype=out_dtype))


@pytest.mark.parametrize("T", [2, 100])
def test_matvec_packed_layer_past_4_gib(T):
    m, n = 540_000, 16_384
    codes = torch.empty((m, n), dtype=torch.uint8, device="cuda")
    for i in range(0, m, 60_000):
        codes[i:i + 60_000] = torch.randint(0, 16, (60_000, n), dtype=torch.uint8, device="cuda")
    scales = torch.rand(m, 1, device="cuda") + 0.5
    w = bk.pack(codes, scales, 4)
    assert w.data.numel() > 1 << 32
    x = tokens(T, n, BF16, 3)
    y = bk.matvec(x.cuda(), w, out_dtype=F32)
    for r in (slice(0, 40), slice(m - 40, m), slice(262_000, 262_200), slice(524_200, 524_400)):
        c, s = codes[r].cpu(), scales[r].cpu()
        ref, tol = matvec_bound(x, None, dense(c, s, 4, 0), F32)
        assert bool(((y[:, r].cpu().double() - ref).abs() <= tol).all())


def test_matvec_tokens_in_ranges():
    """So many rows that 2060 tokens take two grids: whole numbers, each token against its own value."""
    m, T = 1 << 22, 2060
    codes = (torch.arange(m, device="cuda") % 16).to(torch.uint8).reshape(m, 1)
    w = bk.pack(codes, torch.full((m,), 2.0, device="cuda"), 4)
    x = (torch.arange(T, device="cuda") % 16).to(BF16).reshape(T, 1)
    xs = torch.where(torch.arange(T, device="cuda") % 3 == 0, 2.0, 1.0)
    y = bk.matvec(x, w, x_scale=xs)
    for t in (0, 1, 2045, 2046, 2047, 2048, 2049, 2059):
        ref = x[t, 0].float() * xs[t] * (codes[:, 0].float() * 2 - 15)
        assert torch.equal(y[t].float(), ref.to(BF16).float())


def test_pack_clamps_and_overwrites_all_of_it():
    """Codes past the grid count as the largest; every byte of the packed buffer is written."""
    codes, scales = layer(19, 140, 4, 32, 1)
    big = codes.clone()
    big[codes == 15] = 200
    a = bk.pack(codes.cuda(), scales.cuda(), 4, 32).data
    b = bk.pack(big.cuda(), scales.cuda(), 4, 32).data
    assert torch.equal(a, b)
    c = torch.full_like(a, 0xA5)
    lib = bk.LIB
    cd, sd = codes.cuda(), scales.cuda()
    st = lib.bakron_pack(cd.data_ptr(), 19, 140, 140, 4, sd.data_ptr(), 5, 32, c.data_ptr(), c.numel(),
                         torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(a, c)


@pytest.mark.parametrize("bits", [1, 2, 3, 4])
def test_pack_clamps_to_the_layers_own_grid(bits):
    """A code past 2^bits - 1 counts as that, also where codes are stored in more bits than they have."""
    top = 2 ** bits - 1
    codes, scales = layer(21, 150, bits, 32, 1)
    big = codes.clone()
    at = codes == top
    big[at] = torch.tensor([top + 1, top + 2, 200, 255], dtype=torch.uint8)[torch.arange(int(at.sum())) % 4]
    a = bk.pack(codes.cuda(), scales.cuda(), bits, 32)
    b = bk.pack(big.cuda(), scales.cuda(), bits, 32)
    assert torch.equal(a.data, b.data)
    y = bk.matvec(torch.eye(150, device="cuda"), b).cpu()  # w itself: exact in fp32
    assert torch.equal(y, dense(codes, scales, bits, 32).float().t())


def test_pack_strided_codes():
    codes, scales = layer(30, 100, 2, 64, 1)
    wide = torch.zeros(30, 131, dtype=torch.uint8)
    wide[:, 9:109] = codes
    swide = torch.zeros(30, 5)
    swide[:, 1:3] = scales
    a = bk.pack(codes.cuda(), scales.cuda(), 2, 64).data
    b = bk.pack(wide.cuda()[:, 9:109], swide.cuda()[:, 1:3], 2, 64).data
    assert torch.equal(a, b)


# ------------------------------------------------------------------ rmsnorm
def signs(seed, n):
    with np.errstate(over="ignore"):
        z = np.uint64(seed & (2**64 - 1)) + np.arange(1, n + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    return torch.from_numpy(1.0 - 2.0 * (z >> np.uint64(63)).astype(np.float64))


def rotate64(v, seed):
    T, n = v.shape
    v = v * signs(seed, n)
    h = 1
    while n % (2 * h) == 0:
        v = v.reshape(T, n // (2 * h), 2, h)
        v = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).reshape(T, n) / np.sqrt(2.0)
        h *= 2
    return v


def norm64(x, r, gain, eps, seed):
    """(v, bound of v's error before its output rounding). The sum of squares of n terms: at most
    n / 64 + 16 roundings on any path to the total (lanes, then a tree), halved by the root; h, the
    quotient by n, eps, root, reciprocal and two products add 8; the rotation adds a rounding per
    stage and its scale, each relative to the block's absolute sum over sqrt(b)."""
    h = x.double() + (r.double() if r is not None else 0.0)
    n = h.shape[1]
    v = h / (h.square().mean(1, keepdim=True) + eps).sqrt()
    if gain is not None:
        v = v * gain.double()
    # h itself is a sum rounded to fp32: relative to it, half a step (counted in the 8)
    c = U * (n / 128 + 16)
    if seed is None:
        return v, v.abs() * c
    b = n & -n
    block = v.abs().reshape(len(v), n // b, b).sum(2, keepdim=True).expand(-1, -1, b).reshape(v.shape) / np.sqrt(b)
    return rotate64(v, seed), block * (c + U * (np.log2(b) + 3))


def check_norm(T, n, dtype, out_dtype, residual=True, gain="x", seed=None, eps=1e-5, big=1.0, threads=None):
    g = gen(n + T)
    x = (big * torch.randn(T, n, generator=g)).to(dtype)
    r = (big * torch.randn(T, n, generator=g)).to(dtype) if residual else None
    gv = None if gain is None else (1 + 0.3 * torch.randn(n, generator=g)).to(dtype if gain == "x" else F32)
    res = bk.rmsnorm(x.cuda(), None if gv is None else gv.cuda(), residual=None if r is None else r.cuda(), eps=eps,
                     rotate_seed=seed, out_dtype=out_dtype)
    v, tol = norm64(x, r, gv, eps, seed)
    if residual:
        h = x.double() + r.double()
        # exact fp32 sum or one rounding to fp32, then one to the type
        fi = torch.finfo(dtype)
        assert bool(((res.sum.cpu().double() - h).abs() <= h.abs() * (fi.eps / 2 * (1 + 2 * U) + U) + fi.tiny).all())
    else:
        assert res.sum is None
    y = res.y.cpu().double()
    if out_dtype not in (I8, E4M3):
        fi = torch.finfo(out_dtype)
        err, tol = (y - v).abs(), tol + (v.abs() + tol) * fi.eps / 2 + fi.tiny
        assert bool((err <= tol).all()), float((err / tol).max())
        return
    top = 127.0 if out_dtype == I8 else 448.0
    s = res.scale.cpu().double()
    amax = v.abs().amax(1)
    assert bool(((s - amax / top).abs() <= tol.amax(1) / top + amax / top * 2 * U).all())
    # half a step: s / 2 in int8; in e4m3 2^-4 of the value, at least 2^-10 s; the quotient's rounding moves a
    # value by U of itself before that; the top value may be cut by the rounding of s
    half = 0.5 * s[:, None] if out_dtype == I8 else torch.maximum(v.abs() * 2.0 ** -4, s[:, None] * 2.0 ** -10)
    err = (y * s[:, None] - v).abs()
    bound = half + tol * (1 + 2.0 ** -4) + v.abs() * 4 * U
    assert bool((err <= bound).all()), float((err / bound).max())
    assert float(y.abs().max()) <= top
    assert bool((y.abs().amax(1) == top).all())  # the largest magnitude takes the top code


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,n", [(1, 1), (2, 7), (3, 64), (1, 4096), (5, 4099), (9, 5120), (4, 8192), (3, 14336),
                                 (2, 16384), (2, 20000), (2, 32768), (1, 32776), (2, 70001)])
def test_rmsnorm_same_type(T, n, dtype):
    check_norm(T, n, dtype, dtype)


@pytest.mark.parametrize("out_dtype", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,n", [(2, 96), (3, 4096), (1, 12288), (2, 40001)])
def test_rmsnorm_output_types(T, n, dtype, out_dtype):
    check_norm(T, n, dtype, out_dtype, gain="f32")


@pytest.mark.parametrize("out_dtype", [F32, BF16, I8, E4M3])
@pytest.mark.parametrize("T,n", [(1, 1), (2, 2), (3, 7), (2, 24), (1, 64), (3, 512), (2, 640), (5, 1024), (1, 2048),
                                 (4, 4096), (2, 5120), (3, 8192), (2, 14336), (1, 16384), (2, 28672), (1, 32768),
                                 (2, 32764), (2, 12300), (2, 10001), (3, 9984), (2, 16352), (1500, 8448)])
def test_rmsnorm_rotated(T, n, out_dtype):
    check_norm(T, n, BF16, out_dtype, seed=n * 12345 + 7)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("gain", [None, "x", "f32"])
def test_rmsnorm_optional_arguments(gain, residual):
    check_norm(4, 300, F16, F32, residual=residual, gain=gain, eps=0.0)
    check_norm(4, 256, BF16, I8, residual=residual, gain=gain, seed=2**64 - 1)


@pytest.mark.parametrize("T", [1, 700, 5000])
def test_rmsnorm_many_rows(T):
    check_norm(T, 130, BF16, BF16)
    check_norm(T, 256, F32, E4M3, seed=1)


def test_rmsnorm_rotation_is_the_layers_rotation():
    """The same rotation as rht applies to the rows of a matrix: fp32 sums of one order, so within the bound of both."""
    x = tokens(3, 1536, F32, 1)
    rot = bk.rmsnorm(x.cuda(), rotate_seed=99).y
    ref = bk.rht(bk.rmsnorm(x.cuda()).y.clone(), 1, 99)
    v, tol = norm64(x, None, None, 1e-6, 99)
    assert bool(((rot - ref).cpu().double().abs() <= 2 * tol).all())


@pytest.mark.parametrize("n", [100, 4096, 40000])
@pytest.mark.parametrize("out_dtype", [F32, I8, E4M3])
def test_rmsnorm_special_rows(n, out_dtype):
    """Rows of zeros, an infinity, a NaN, tiny and huge values, each alone in its row."""
    x = torch.randn(6, n, generator=gen(1))
    x[0] = 0.0
    x[1, n // 2] = float("inf")
    x[2, n - 1] = float("nan")
    x[3] *= 1e-18
    x[4] *= 1e15
    rows = bk.rmsnorm(x.cuda(), eps=1e-6, out_dtype=out_dtype)
    y = rows.y.cpu().double()
    if out_dtype == F32:
        assert bool((y[0] == 0).all()) and bool(torch.isnan(y[2]).all())
        assert bool(torch.isnan(y[1, n // 2])) and bool((y[1, :n // 2] == 0).all())
    else:
        s = rows.scale.cpu()
        assert s[0] == 0 and bool(torch.isnan(s[1:3]).all()) and bool((y[:3] == 0).all())
        y = y * s.double()[:, None]
    v, tol = norm64(x, None, None, 1e-6, None)
    if out_dtype == F32:
        assert bool(((y[3:] - v[3:]).abs() <= tol[3:] + v[3:].abs() * U + 2.0 ** -126).all())
    else:
        half = 0.5 / 127 if out_dtype == I8 else 2.0 ** -4
        assert bool(((y[3:] - v[3:]).abs() <= half * v[3:].abs().amax(1, keepdim=True) * (1 + 1e-4)).all())


@pytest.mark.parametrize("n", [100, 4096, 40000])
def test_rmsnorm_sum_of_squares_past_fp32(n):
    """(1e20)^2 passes fp32's largest value: the row's values are zeros; the next row's are its own."""
    x = tokens(2, n, BF16, 3).cuda()
    ref = bk.rmsnorm(x)
    x[0] *= 1e20
    y = bk.rmsnorm(x).y
    assert bool((y[0] == 0).all()) and torch.equal(y[1], ref.y[1])
    q = bk.rmsnorm(x, out_dtype=I8)
    assert bool(torch.equal(q.scale[0] * q.y[0].float(), torch.zeros(n, device="cuda"))) and q.scale[1] > 0


@pytest.mark.parametrize("n", [100, 4096, 20000, 40000])
def test_rmsnorm_without_eps(n):
    """eps = 0: a row of zeros, or of values whose squares are 0 in fp32, has no finite values; others are right."""
    x = tokens(4, n, F32, 3)
    x[1] = 0.0
    x[2] *= 1e-30
    x[3] *= 1e-15
    y = bk.rmsnorm(x.cuda(), eps=0.0).y.cpu().double()
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[2]).any())
    v, tol = norm64(x, None, None, 0.0, None)
    assert bool(((y - v).abs() <= tol + v.abs() * U)[[0, 3]].all())
    for out_dtype in (I8, E4M3):
        q = bk.rmsnorm(x.cuda(), eps=0.0, out_dtype=out_dtype)
        assert bool(torch.isnan(q.scale[1:3]).all()) and bool((q.y[1:3].float() == 0).all())
        assert bool(torch.isfinite(q.scale[[0, 3]]).all())


@pytest.mark.parametrize("n", [200, 33000])
def test_rmsnorm_in_place(n):
    """sum_out = residual, out = x: the values are those of a call with buffers of its own."""
    x, r = tokens(3, n, BF16, 1).cuda(), tokens(3, n, BF16, 2).cuda()
    ref = bk.rmsnorm(x, residual=r)
    x2, r2 = x.clone(), r.clone()
    bk.rmsnorm(x2, residual=r2, sum_out=r2, out=x2)
    assert torch.equal(x2, ref.y) and torch.equal(r2, ref.sum)
    x2, r2 = x.clone(), r.clone()
    bk.rmsnorm(x2, residual=r2, sum_out=x2, out=r2)
    assert torch.equal(r2, ref.y) and torch.equal(x2, ref.sum)
    with pytest.raises(bk.BakronError):
        bk.rmsnorm(x, residual=r, sum_out=r, out=r)


def test_rmsnorm_rows_of_wider_buffers():
    """x, residual, sum and y as column ranges of one buffer, at odd offsets; nothing else is written."""
    T, n = 5, 333
    for dtype in (F32, F16, BF16):
        buf = torch.full((T, 4 * n + 9), 55.0, device="cuda", dtype=dtype)
        parts = [buf[:, 1 + i * (n + 1):1 + i * (n + 1) + n] for i in range(4)]
        x, r = tokens(T, n, dtype, 1).cuda(), tokens(T, n, dtype, 2).cuda()
        parts[0].copy_(x)
        parts[1].copy_(r)
        ref = bk.rmsnorm(x, residual=r, rotate_seed=5)
        bk.rmsnorm(parts[0], residual=parts[1], sum_out=parts[2], out=parts[3], rotate_seed=5)
        assert torch.equal(parts[3], ref.y) and torch.equal(parts[2], ref.sum)
        assert torch.equal(parts[0], x) and torch.equal(parts[1], r)
        for p in parts:
            p.fill_(55.0)
        assert bool((buf == 55.0).all())


def test_rmsnorm_empty():
    r = bk.rmsnorm(torch.empty(0, 64, device="cuda", dtype=BF16), out_dtype=I8)
    assert r.y.shape == (0, 64) and r.scale.shape == (0,)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rmsnorm_more_rows_than_a_grid(dtype):
    """2^21 + 5 rows of one column: workgroups take a second row."""
    x = tokens((1 << 21) + 5, 1, dtype, 1).cuda()
    y = bk.rmsnorm(x, eps=1e-5).y
    ref = x.double() / (x.double().square() + 1e-5).sqrt()
    assert float((y.double() - ref).abs().max()) <= torch.finfo(dtype).eps / 2 + 10 * U


def test_rmsnorm_offsets_past_2_31():
    ld = (1 << 31) + 8
    small = tokens(3, 256, BF16, 1).cuda()
    x = torch.empty(2 * ld + 256, dtype=BF16, device="cuda").as_strided((3, 256), (ld, 1))
    x.copy_(small)
    y = torch.empty(2 * ld + 256, dtype=I8, device="cuda").as_strided((3, 256), (ld, 1))
    a = bk.rmsnorm(x, rotate_seed=3, out=y)
    b = bk.rmsnorm(small, rotate_seed=3, out_dtype=I8)
    assert torch.equal(a.y.contiguous(), b.y) and torch.equal(a.scale, b.scale)


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refusals():
    codes, scales = layer(32, 128, 4, 32, 1)
    c, s = codes.cuda(), scales.cuda()
    w = bk.pack(c, s, 4, 32)
    x = tokens(2, 128, BF16, 2).cuda()
    bad = [lambda: bk.pack(c, s, 5, 32), lambda: bk.pack(c, s, 4, 48), lambda: bk.pack(c, s, 4),
           lambda: bk.pack(c.float(), s, 4, 32), lambda: bk.pack(c, s.double(), 4, 32), lambda: bk.pack(c.t(), s, 4, 32),
           lambda: bk.pack(c, s.cpu(), 4, 32),
           lambda: bk.matvec(x[:, :100], w), lambda: bk.matvec(x.double(), w), lambda: bk.matvec(x, w, out_dtype=I8),
           lambda: bk.matvec(x, w, out=torch.empty(2, 31, device="cuda")),
           lambda: bk.matvec(x, w, out=torch.empty(2, 32, device="cuda"), out_dtype=BF16),
           lambda: bk.matvec(x, w, x_scale=torch.ones(3, device="cuda")),
           lambda: bk.matvec(x, w, x_scale=torch.ones(2)),
           lambda: bk.matvec(x[:1].expand(2, 128), w), lambda: bk.matvec(x.unsqueeze(0), w),
           lambda: bk.matvec(x, w, out=torch.empty(32, 2, device="cuda").t()),
           lambda: bk.rmsnorm(x, residual=x.float()), lambda: bk.rmsnorm(x, torch.ones(127, device="cuda")),
           lambda: bk.rmsnorm(x, torch.ones(128)), lambda: bk.rmsnorm(x, torch.ones(128, device="cuda").half()),
           lambda: bk.rmsnorm(x, out_dtype=torch.int32), lambda: bk.rmsnorm(x, scale_out=torch.ones(2, device="cuda")),
           lambda: bk.rmsnorm(x, out_dtype=I8, scale_out=torch.ones(3, device="cuda")),
           lambda: bk.rmsnorm(tokens(2, 128, I8, 1).cuda()), lambda: bk.rmsnorm(x[0])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % i)
    for f in (lambda: bk.rmsnorm(x, eps=-1.0),
              lambda: bk.rmsnorm(torch.zeros(1, 40000, device="cuda"), rotate_seed=1),
              lambda: bk.matvec(x, w, out=x[:, :32])):
        with pytest.raises(bk.BakronError):
            f()


def test_binding_refuses_a_layer_whose_bytes_were_replaced():
    codes, scales = layer(32, 128, 4, 32, 1)
    w = bk.pack(codes.cuda(), scales.cuda(), 4, 32)
    x = tokens(2, 128, BF16, 2).cuda()
    data = w.data
    w.data = data[:-16]
    with pytest.raises(bk.BakronError):
        bk.matvec(x, w)
    for bad in (data[:1].expand(data.numel()), data.cpu()):
        w.data = bad
        with pytest.raises(ValueError):
            bk.matvec(x, w)
    w.data = data.clone()
    assert bk.matvec(x, w).shape == (2, 32)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("bits,q", [(4, I8), (4, E4M3), (2, I8), (3, BF16)])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_rotated_layer_end_to_end(T, bits, q):
    """A layer is rotated, rounded by the solve, packed, and used: norm + rotation + 8 bits, product, rotation back.

    Every operator is compared with the 64-bit form of its own inputs; the whole is compared with the 64-bit
    product of the unrotated codes' weights, with the 8-bit rounding of the activations as the bound."""
    m, n = 192, 320
    g = gen(bits)
    W = torch.randn(m, n, generator=g)
    X, G = torch.randn(900, n, generator=g), torch.randn(700, m, generator=g)
    Wd = W.cuda()
    HI, HO = bk.hessian_accum(X.cuda()), bk.hessian_accum(G.cuda())
    bk.rotate_layer(Wd, HI, HO, seed_O=11, seed_I=22)
    (LO, DO), (LI, DI) = bk.ldl_pair(HO, HI)
    res = bk.solve(Wd, LO, LI, bits, D_O=DO, D_I=DI)
    w = bk.pack(res.codes, res.scales, bits)
    x, r = tokens(T, n, BF16, 5), tokens(T, n, BF16, 6)
    gain = (1 + 0.1 * torch.randn(n, generator=g)).to(BF16)
    nr = bk.rmsnorm(x.cuda(), gain.cuda(), residual=r.cuda(), rotate_seed=22, out_dtype=q)
    y = bk.matvec(nr.y, w, x_scale=nr.scale, out_dtype=F32)
    wq = dense(res.codes.cpu(), res.scales.cpu().reshape(-1, 1), bits, 0)
    ref, tol = matvec_bound(nr.y.cpu(), None if nr.scale is None else nr.scale.cpu(), wq, F32)
    assert bool(((y.cpu().double() - ref).abs() <= tol).all())
    out = bk.rht(y.clone(), 1, 11, transpose=True).cpu().double()
    # in 64 bits and the original basis: v U_I^T W'^T U_O = (U_O^T W' U_I v)
    v, _ = norm64(x, r, gain, 1e-6, 22)
    full = v @ wq.t()
    b = m & -m
    full = full.reshape(T, m // b, b)
    hmat = torch.tensor([[(-1.0) ** bin(i & j).count("1") for j in range(b)] for i in range(b)], dtype=torch.float64)
    full = (full @ hmat).reshape(T, m) / np.sqrt(b) * signs(11, m)
    step = {I8: 0.5 / 127, E4M3: 2.0 ** -4, BF16: 2.0 ** -8}[q]
    lim = step * v.abs().amax(1) * wq.abs().sum(1).max()  # |U_O^T e| <= sqrt(b) max|e|, e a weighted sum of half steps
    assert bool(((out - full).abs() <= 1.01 * np.sqrt(b) * lim[:, None]).all())


def test_on_another_stream_and_device_guard():
    codes, scales = layer(64, 512, 4, 128, 1)
    w = bk.pack(codes.cuda(), scales.cuda(), 4, 128)
    x = tokens(8, 512, BF16, 2).cuda()
    ref_n = bk.rmsnorm(x, rotate_seed=1, out_dtype=I8)
    ref = bk.matvec(ref_n.y, w, x_scale=ref_n.scale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nr = bk.rmsnorm(x, rotate_seed=1, out_dtype=I8)
        y = bk.matvec(nr.y, w, x_scale=nr.scale)
    s.synchronize()
    assert torch.equal(y, ref)


@pytest.mark.parametrize("T", [1, 24, 160])
def test_graph_replays(T):
    """Norm and product captured once and replayed on new inputs, with eager work between the replays."""
    codes, scales = layer(160, 1024, 4, 128, 1)
    w = bk.pack(codes.cuda(), scales.cuda(), 4, 128)
    x, r = tokens(T, 1024, BF16, 2).cuda(), tokens(T, 1024, BF16, 3).cuda()
    gain = torch.ones(1024, device="cuda", dtype=BF16)

    def step():
        nr = bk.rmsnorm(x, gain, residual=r, rotate_seed=4, out_dtype=I8)
        return bk.matvec(nr.y, w, x_scale=nr.scale, out_dtype=F32), nr.sum

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = step()
    for k in range(4):
        x.copy_(tokens(T, 1024, BF16, 10 + k))
        r.copy_(tokens(T, 1024, BF16, 20 + k))
        graph.replay()
        torch.cuda.synchronize()
        ey, eh = step()
        assert torch.equal(y, ey) and torch.equal(h, eh)
