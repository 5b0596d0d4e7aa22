"""What passes between the two products of lora and experts, and the last roundings, on the GPU.

Inputs whose second product adds no error show every bit of what enters it: a value of 24 bits that reaches an output
by itself has to come out whole in fp32, and rounded once, to nearest even, in 16 bits.
"""
import pytest
import torch

import kronecker_hessian_rounding_amd as bk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn
KEPT = {F32: 24, F16: 11, BF16: 8}  # bits of a value of the type


def gen(seed):
    return torch.Generator().manual_seed(seed)


def whole_numbers(shape, out, seed):
    """24-bit numbers, 2^23 .. 2^24 - 1. For a 16-bit output each lies one beside a tie of its rounding, on either side."""
    g = gen(seed)
    v = torch.randint(2 ** 23, 2 ** 24, shape, generator=g)
    if out != F32:
        low = 24 - KEPT[out]
        v = (v >> low << low) + 2 ** (low - 1) + 2 * torch.randint(0, 2, shape, generator=g) - 1
    return v


# ------------------------------------------------------------------ lora
def lora_case(T, n, m, r, R, xt, wt, out, seed):
    """x has ones in three columns, A the three bytes of a number there; B picks one rank a row, with a sign."""
    g = gen(seed)
    u = whole_numbers((R, r), out, seed + 1)
    at = torch.randperm(n, generator=g)[:3]
    x = torch.zeros(T, n)
    x[:, at] = 1.0
    a = torch.zeros(R, r, n)
    for i, shift in enumerate((16, 8, 0)):
        a[:, :, at[i]] = (u >> shift & 255).float() * 2.0 ** (shift - 8)  # within fp16's range
    sign = 2.0 * torch.randint(0, 2, (R, m), generator=g) - 1
    rank = torch.randint(0, r, (R, m), generator=g)
    b = torch.zeros(R, m, r).scatter_(2, rank[:, :, None], sign[:, :, None])
    ids = torch.randint(0, R, (T,), generator=g, dtype=torch.int32)
    want = (u.double().gather(1, rank) * sign * 2.0 ** -8)[ids.long()]
    return x.to(xt), a.to(wt), b.to(wt), ids, want


@pytest.mark.parametrize("xt,wt", [(F32, F32), (F16, F16), (BF16, BF16), (I8, F16), (I8, BF16), (E4M3, F16), (E4M3, BF16)])
@pytest.mark.parametrize("T,n,m,r", [(1, 300, 200, 16), (5, 1500, 130, 13), (40, 700, 700, 8), (100, 96, 65, 32), (20, 200, 100, 20),  # one launch
                                     (19, 96, 90, 130), (3, 200, 70, 512),                                              # ranks in passes
                                     (1, 4096, 300, 64), (150, 700, 200, 13), (140, 6661, 700, 16), (200, 96, 130, 32),  # two
                                     (130, 300, 383, 40), (70, 128, 64, 64), (300, 500, 260, 100), (300, 500, 260, 128)])
def test_lora_holds_every_bit_between_its_products(T, n, m, r, xt, wt):
    for out in (F32, F16, BF16):
        x, a, b, ids, want = lora_case(T, n, m, r, 3, xt, wt, out, T + r)
        y = bk.lora(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), out_dtype=out).cpu()
        # (the 24-bit numbers are fp32 values, so that the cast rounds once; 2^-16 keeps them in fp16's range)
        if out == F16:
            y = bk.lora(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=torch.full((3,), 2.0 ** -16, device="cuda"), out_dtype=out).cpu()
            want = want * 2.0 ** -16
        assert torch.equal(y, want.float().to(out)), (out, int((y != want.float().to(out)).sum()), y.numel())


# ------------------------------------------------------------------ experts
def experts_case(T, E, k, n, I, dbits, dgroup, xt, act, seed):
    """Token t's columns 2 c and 2 c + 1 hold 64, the others 0, and weights are -1/2 or 1/2: Gate gives 64 in every row, which act
    leaves, Up 64 in the one row c % I and 0 in the others, Down +-1/2 of that. So each result is +-2^11 times the router's
    weight, by way of one column of Down's."""
    g = gen(seed)
    c = (torch.randint(0, n // 2, (1,), generator=g) + torch.arange(T)) % (n // 2)
    x = torch.zeros(T, n)
    x[torch.arange(T), 2 * c] = x[torch.arange(T), 2 * c + 1] = 64.0
    gate = torch.full((E, I, n), 8, dtype=torch.uint8)
    up = torch.full((E, I, n), 8, dtype=torch.uint8)
    up[:, :, 1::2] = 7
    pairs = torch.arange(n // 2)
    up[:, pairs % I, 2 * pairs + 1] = 8
    top = 2 ** (dbits - 1)
    down = torch.randint(top - 1, top + 1, (E, n, I), generator=g, dtype=torch.uint8)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    slot, e = torch.randint(0, k, (T,), generator=g), torch.randint(0, E, (T,), generator=g)
    ids[torch.arange(T), slot] = e.to(torch.int32)
    ones = lambda m, cols, group: torch.ones(E, m, -(-cols // group) if group else 1)
    packed = [bk.pack_experts(w.cuda(), ones(m, cols, gr).cuda(), bits, gr)
              for w, m, cols, bits, gr in ((gate, I, n, 4, 128), (up, I, n, 4, 128), (down, n, I, dbits, dgroup))]
    half = (down.double() - (2 ** dbits - 1) / 2)[e, :, c % I]
    return x.to(xt), packed, ids, (slot, half)


@pytest.mark.parametrize("xt", [F32, F16, BF16, I8, E4M3])
@pytest.mark.parametrize("T,E,k,n,I,dbits,dgroup", [(1, 3, 2, 600, 300, 4, 128), (3, 5, 2, 130, 65, 2, 0), (7, 4, 2, 600, 290, 4, 32), (16, 8, 3, 514, 257, 3, 64),
                                                    (9, 4, 3, 4112, 4000, 4, 128), (16, 4, 3, 8200, 2048, 2, 64),  # in splits
                                                    (20, 40, 2, 200, 100, 4, 128), (33, 12, 1, 600, 300, 2, 32),   # list tiles of 16
                                                    (70, 2, 2, 600, 300, 4, 128), (300, 3, 1, 260, 129, 4, 32)])   # of 64
def test_experts_hold_every_bit_between_their_products(T, E, k, n, I, dbits, dgroup, xt):
    x, packed, ids, (slot, half) = experts_case(T, E, k, n, I, dbits, dgroup, xt, "silu", T + n)
    for out, act in ((F32, "silu"), (F32, "gelu"), (F16, "silu"), (BF16, "gelu")):
        w = whole_numbers((T,), out, T + k)
        # the router's weight, of 24 bits, in one slot; others hold what must not matter. 2^11 times it stays in fp16's range
        wt = torch.full((T, k), 3.0)
        wt[torch.arange(T), slot] = w.float() * 2.0 ** -22
        y = bk.experts(x.cuda(), *packed, ids.cuda(), wt.cuda(), act=act, out_dtype=out).cpu()
        want = (w.double() * 2.0 ** -22 * 64 * 64)[:, None] * half
        assert torch.equal(y, want.float().to(out)), (out, int((y != want.float().to(out)).sum()), y.numel())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [1, 6, 40, 400])
def test_activation_is_formed_in_fp32(T, act):
    """Values from -80 on by themselves through act. The exponential is within an ulp (2 U), its sum with 1, the quotient and the
    product with u one rounding each: 5 U. gelu's argument has six roundings (two constants, four operations), 6 U |z| of the
    result; U more for second-order terms."""
    n = I = 64
    E = 2
    g = gen(T)
    v = torch.rand(T, generator=g) * 90 - 80
    if act == "gelu":
        v = v.clamp_min(-9.5) if T == 1 else torch.rand(T, generator=g) * 15 - 9.5
    x = torch.zeros(T, n)
    x[:, 4] = x[:, 5] = v
    gate = torch.full((E, I, n), 8, dtype=torch.uint8)
    down = torch.full((E, n, I), 8, dtype=torch.uint8)
    up = torch.full((E, I, n), 8, dtype=torch.uint8)
    up[:, :, 1::2] = 7
    up[:, 9, 5] = 8
    one = torch.ones(E, I, 1)
    packed = [bk.pack_experts(c.cuda(), one.cuda(), 4) for c in (gate, up, down)]
    y = bk.experts(x.cuda(), *packed, torch.zeros(T, 1, dtype=torch.int32).cuda(), torch.ones(T, 1).cuda(), act=act).cpu().double()
    d = v.double()
    z = d if act == "silu" else 2 * (2 / torch.pi) ** 0.5 * (d + 0.044715 * d ** 3)
    want = d / (1 + torch.exp(-z)) * d / 2
    tol = want.abs() * U * (6 + (6 * z.abs() if act == "gelu" else 0.0))
    err = (y - want[:, None]).abs()
    assert bool((err <= tol[:, None]).all()), float((err / tol[:, None]).max())


@pytest.mark.parametrize("T,E,k,n,I", [(2, 9, 3, 300, 200), (4, 30, 4, 200, 1400), (7, 12, 4, 513, 300), (8, 64, 6, 130, 700), (16, 6, 2, 300, 1000),
                                       (16, 64, 8, 96, 400), (9, 8, 4, 4112, 4000), (30, 9, 3, 200, 300), (200, 4, 2, 130, 300),
                                       (16, 200, 8, 96, 300), (12, 1000, 40, 64, 140), (3, 400, 30, 70, 260)])
def test_experts_other_rows_do_not_matter(T, E, k, n, I):
    """Every token's result stays bit for bit, in fp32, when the other rows and the experts that they name change."""
    g = gen(T + E)

    def layer(m, c):
        return bk.pack_experts(torch.randint(0, 16, (E, m, c), generator=g, dtype=torch.uint8).cuda(), torch.rand(E, m, -(-c // 128), generator=g).cuda(), 4, 128)

    def choice():
        return torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32)
    packed = [layer(I, n), layer(I, n), layer(n, I)]
    x, ids, wt = torch.randn(T, n, generator=g), choice(), torch.rand(T, k, generator=g)
    y = bk.experts(x.cuda(), *packed, ids.cuda(), wt.cuda()).cpu()
    for r in range(3):
        x2, ids2, w2 = torch.randn(T, n, generator=g), choice(), torch.rand(T, k, generator=g)
        ids2[torch.rand(T, k, generator=g) < (0.0, 0.4, 0.9)[r]] = -1
        for t in sorted({0, 1, T // 3, T // 2, T - 2, T - 1}):
            x3, ids3, w3 = x2.clone(), ids2.clone(), w2.clone()
            x3[t], ids3[t], w3[t] = x[t], ids[t], wt[t]
            z = bk.experts(x3.cuda(), *packed, ids3.cuda(), w3.cuda()).cpu()
            assert torch.equal(z[t], y[t]), (r, t, int((z[t] != y[t]).sum()), n)


# ------------------------------------------------------------------ lora's other edges
@pytest.mark.parametrize("T,r,m", [(5, 16, 200), (40, 13, 130), (6, 200, 70), (180, 16, 200), (150, 64, 96), (140, 5, 300)])
@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_lora_infinity_in_one_rank(T, r, m, out):
    """An infinite u_k leaves the token's other ranks as they are, above fp16's largest value too: the sum is infinite, not NaN."""
    n, R = 64, 2
    g = gen(r)
    x = torch.full((T, n), 100.0)
    a, b = torch.zeros(R, r, n), torch.where(torch.rand(R, m, r, generator=g) < 0.5, 1.0, -1.0)
    a[:, :, 3] = 1000.0          # u = 10^5
    a[1, 2, 7] = float("inf")
    ids = torch.arange(T, dtype=torch.int32) % R
    y = bk.lora(x.to(F16).cuda(), a.to(F16).cuda(), b.to(F16).cuda(), ids.cuda(), out_dtype=out).cpu()
    want = torch.where(ids[:, None] == 1, b[1, :, 2] * float("inf"), 1e5 * b[0].sum(1)).to(out)
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,r,m", [(5, 16, 200), (40, 13, 130), (6, 200, 70), (180, 16, 300), (150, 64, 100), (140, 5, 128)])
def test_lora_without_an_adapter_is_the_base(T, r, m, dtype):
    """To the sign of a zero, in every row; without a base +0."""
    g = gen(m)
    x, a, b = (torch.randn(s, generator=g).to(dtype).cuda() for s in ((T, 64), (2, r, 64), (2, m, r)))
    base = torch.randn(T, m, generator=g)
    base[torch.rand(T, m, generator=g) < 0.4] = -0.0
    base[torch.rand(T, m, generator=g) < 0.2] = 0.0
    base = base.to(dtype).cuda()
    ids = torch.where(torch.arange(T) % 3 == 1, 1, -1).to(torch.int32).cuda()
    bits = torch.int32 if dtype == F32 else torch.int16
    y = bk.lora(x, a, b, ids, base=base)
    assert torch.equal(y[ids < 0].view(bits), base[ids < 0].view(bits))
    assert bool((bk.lora(x, a, b, ids)[ids < 0].view(bits) == 0).all())


@pytest.mark.parametrize("T,n,m,r", [(50, 700, 333, 24), (190, 700, 333, 24), (170, 3000, 128, 64), (90, 300, 70, 200)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_lora_other_rows_do_not_matter(T, n, m, r, dtype):
    """In fp32, with the others' adapters alike (more than half of a tile's tokens name one) and mixed."""
    g = gen(T)
    x, a, b = torch.randn(T, n, generator=g).to(dtype), (torch.randn(5, r, n, generator=g) * 0.05).to(dtype), torch.randn(5, m, r, generator=g).to(dtype)
    ids, base = torch.randint(-1, 5, (T,), generator=g, dtype=torch.int32), torch.randn(T, m, generator=g)
    run = lambda x, ids: bk.lora(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), base=base.cuda(), out_dtype=F32).cpu()
    y = run(x, ids)
    for others in (torch.full((T,), 2, dtype=torch.int32), torch.full((T,), -1, dtype=torch.int32), torch.randint(-1, 5, (T,), generator=g, dtype=torch.int32)):
        for t in (0, 17, 40, T - 1):
            x2, ids2 = torch.randn(T, n, generator=g).to(dtype), others.clone()
            x2[t], ids2[t] = x[t], ids[t]
            assert torch.equal(run(x2, ids2)[t], y[t])


# ------------------------------------------------------------------ route
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,E,k", [(40, 256, 8), (30, 64, 6), (20, 1000, 64)])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_weights_are_rounded_once(T, E, k, renorm, dtype):
    """They are 64-bit values (off by some 2^-50) times the factor, and one rounding: half a step of fp32, at most U relative."""
    l = (2 * torch.randn(T, E, generator=gen(E))).to(dtype)
    ids, w = bk.route(l.cuda(), k, "sigmoid", renormalize=renorm, scale=2.7)
    p = torch.sigmoid(l.double()).gather(1, ids.cpu().long())
    p = (p / p.sum(1, keepdim=True) if renorm else p) * float(torch.tensor(2.7))
    assert bool(((w.cpu().double() - p).abs() <= p * U * (1 + 2.0 ** -20)).all())
