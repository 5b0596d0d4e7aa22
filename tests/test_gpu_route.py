"""route on the GPU against its 64-bit form.

Choices are equal: softmax's order is that of the logits as given, sigmoid's that of 64-bit scores, and inputs whose
scores lie within 1e-12 of each other without being equal are none of these tests'. Weights: u = 2^-24; an exponential and
its argument's rounding take 3 u + u |l - max| (at most 40 here, below which a term is under 2^-57 of the largest), the sum
of at most 1024 terms 16 + 6 additions in a row, the quotient and the scale 2: 66 u.
"""
import pytest
import torch

import kronecker_hessian_rounding_amd as bk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF = float("inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def form64(l, k, scoring, bias, renorm, scale):
    l = l.double()
    T, E = l.shape
    if scoring == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
        key = score if bias is None else score + bias.double()
        off = ~(l > -INF) | ~(key > -INF)
    else:
        key = l
        off = ~(l > -INF)
        mx = torch.where(off, -INF, l).amax(1, keepdim=True)
        term = torch.where(l == mx, 1.0, torch.exp(l - mx))
        score = torch.where(off, 0.0, term)
        score = score / score.sum(1, keepdim=True).clamp_min(1e-300)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        left = [e for e in range(E) if not bool(off[t, e])]
        left.sort(key=lambda e: (-float(key[t, e]), e))
        for j, e in enumerate(left[:k]):
            ids[t, j], w[t, j] = e, score[t, e]
    if renorm:
        s = w.sum(1, keepdim=True)
        w = torch.where(s > 0, w / s.clamp_min(1e-300), 0.0)
    return ids, w * scale


def check(l, k, scoring="softmax", bias=None, renorm=True, scale=1.0, view=None):
    ids, w = bk.route(l.cuda() if view is None else view(l.cuda()), k, scoring, None if bias is None else bias.cuda(),
                      renorm, scale)
    ri, rw = form64(l, k, scoring, bias, renorm, scale)
    assert ids.dtype == torch.int32 and w.dtype == F32 and ids.shape == w.shape == ri.shape
    assert torch.equal(ids.cpu(), ri)
    assert bool(((w.cpu().double() - rw).abs() <= 66 * U * rw.abs() + 1e-44).all())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 8, 2), (4, 60, 4), (9, 64, 8), (2, 64, 64), (7, 65, 6), (6, 128, 8),
                                   (5, 160, 6), (3, 256, 8), (2, 257, 1), (3, 512, 10), (2, 1000, 33), (1, 1024, 64)])
def test_against_64_bits(T, E, k, scoring, dtype):
    l = (torch.randn(T, E, generator=gen(E + k)) * 2).to(dtype)
    bias = 0.2 * torch.randn(E, generator=gen(1)) if scoring == "sigmoid" else None
    check(l, k, scoring, bias)
    check(l, k, scoring, bias, renorm=False, scale=2.5)
    check(l, k, scoring, None, scale=0.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_logits_take_the_lowest_index(scoring):
    g = gen(2)
    check(torch.zeros(3, 200), 9, scoring)
    check(torch.randint(-2, 3, (40, 150), generator=g).float(), 20, scoring)
    l = torch.randint(0, 2, (5, 70), generator=g).float()
    l[l == 0] = -0.0
    check(l, 64, scoring)
    # sigmoids that 32 bits could not tell apart, and saturated ones that 64 bits cannot either
    check(20.0 + torch.randn(6, 90, generator=g), 12, "sigmoid")
    check(50.0 + torch.randn(6, 90, generator=g), 12, "sigmoid")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_and_non_finite_logits(scoring, renorm):
    l = torch.randn(8, 70, generator=gen(3))
    l[0] = -INF                          # nothing to choose
    l[1, :67] = -INF                     # three left, fewer than k
    l[2, ::2] = float("nan")
    l[3, 69] = INF
    l[4, [3, 66]] = INF                  # two share
    l[5] = torch.finfo(F32).min          # the type's lowest value is a logit like any other
    l[5, 64] = 0.0
    l[6] = torch.finfo(F32).max
    check(l, 6, scoring, renorm=renorm)
    if scoring == "sigmoid":
        bias = torch.zeros(70)
        bias[5], bias[6], bias[65] = -INF, float("nan"), 3.0
        check(l, 6, scoring, bias, renorm=renorm)


def test_very_small_sigmoids():
    """Scores below fp32's range keep their ratio: it is formed in 64 bits."""
    check(torch.tensor([[-200.0, -201.0, -202.0], [-300.0, -300.0, -302.0]]), 2, "sigmoid")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_a_wider_buffer(dtype):
    l = torch.randn(11, 100, generator=gen(4)).to(dtype)

    def view(t):
        buf = torch.full((11, 131), 50.0, dtype=dtype, device="cuda")
        buf[:, 3:103] = t
        return buf[:, 3:103]
    check(l, 8, view=view)


def test_many_rows():
    """Every wave of a workgroup, and rows past one grid."""
    l = torch.randn(1030, 16, generator=gen(5))
    check(l, 4)
    T = (1 << 24) + 7  # 2^22 workgroups of four rows take a second one
    big = torch.randn(T, 2, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    ids, w = bk.route(big, 1)
    assert torch.equal(ids[:, 0].long(), (big[:, 1] > big[:, 0]).long()) and bool((w == 1).all())


def test_empty():
    ids, w = bk.route(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2)


def test_refusals():
    l = torch.zeros(3, 8, device="cuda")
    b = torch.zeros(8, device="cuda")
    for i, f in enumerate([lambda: bk.route(l, 0), lambda: bk.route(l, 9), lambda: bk.route(l[0], 1), lambda: bk.route(l.double(), 1),
                           lambda: bk.route(l.cpu(), 1), lambda: bk.route(l, 1, "relu"), lambda: bk.route(l, 1, bias=b),
                           lambda: bk.route(l, 1, "sigmoid", b[:7]), lambda: bk.route(l, 1, "sigmoid", b.double()),
                           lambda: bk.route(torch.zeros(1, 1025, device="cuda"), 1), lambda: bk.route(l[:, ::2], 1),
                           lambda: bk.route(torch.zeros(1, 100, device="cuda"), 65), lambda: bk.route(l[:1].expand(3, 8), 1)]):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % i)
    for scale in (INF, float("nan")):
        with pytest.raises(bk.BakronError):
            bk.route(l, 1, scale=scale)


def test_stream_and_graph():
    l = torch.randn(5, 64, generator=gen(6)).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bk.route(l, 6)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = bk.route(l, 6)
    for i in range(4):
        l.copy_(torch.randn(5, 64, generator=gen(10 + i)))
        graph.replay()
        torch.cuda.synchronize()
        e = bk.route(l, 6)
        assert torch.equal(ids, e[0]) and torch.equal(w, e[1])
