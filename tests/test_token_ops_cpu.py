"""Argument checks of the operators in which tokens name their own weights, and of the heads' norm; no GPU is needed."""
import ctypes

import pytest
import torch

import kronecker_hessian_rounding_amd as bk

F32, F16, BF16, I8, E4M3 = range(5)
INVALID, WORKSPACE, OK = 1, 3, 0


def at(addr):
    return ctypes.c_void_p(addr)  # never dereferenced: validation fails first


A, B, C, D, E, F, G = (at(i << 36) for i in range(1, 8))


def test_head_norm_refuses():
    f = bk.LIB.bakron_head_norm
    ok = dict(Q=A, hq=4, qt=512, qh=64, K=B, hk=2, kt=128, kh=64, type=BF16, T=3, d=64, qg=C, kg=C, gtype=BF16, eps=1e-6,
              norm=1, pos=D, pos32=0, freq=E, rot=64, inter=0, YQ=F, yqt=256, yqh=64, YK=G, ykt=128, ykh=64, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    for kw in (dict(Q=None), dict(YQ=None), dict(K=None), dict(YK=None), dict(pos=None), dict(freq=None), dict(T=-1),
               dict(T=1 << 31), dict(hq=0), dict(hk=-1), dict(hq=65536), dict(d=0), dict(d=513), dict(rot=63), dict(rot=66),
               dict(rot=-2), dict(type=I8), dict(type=5), dict(gtype=F16), dict(norm=0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(qh=63), dict(qt=255), dict(qt=63, qh=190),
               dict(yqt=255), dict(kt=127), dict(ykh=10),
               # outputs over inputs, shifted, or on each other
               dict(YQ=A), dict(YQ=at((1 << 36) + 2)), dict(YK=A), dict(YQ=B), dict(YQ=G), dict(YQ=C), dict(YQ=D),
               dict(YK=E), dict(YQ=at((4 << 36) + 23))):
        assert call(**kw) == INVALID, kw
    assert call(T=0) == OK
    assert call(T=0, Q=None, K=None, YQ=None, YK=None, pos=None, freq=None) == OK
    # in place is allowed: such a call passes every check but the last one looked at here
    assert call(YQ=A, yqt=512, YK=B, rot=65) == INVALID


def test_head_norm_strides_do_not_wrap():
    f = bk.LIB.bakron_head_norm
    big = 1 << 61
    args = [A, 16, big, 64, None, 0, 0, 0, BF16, 3, 64, None, None, BF16, 1e-6, 1, None, 0, None, 0, 0, B, 64, 63, None, 0, 0, None]
    assert f(*args) == INVALID  # the output's heads overlap, whatever the input's strides


def test_route_refuses():
    f = bk.LIB.bakron_route
    ok = dict(l=A, type=F32, T=4, E=64, ldl=64, k=8, scoring=1, bias=B, renorm=1, scale=1.0, ids=C, w=D, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    for kw in (dict(l=None), dict(ids=None), dict(w=None), dict(type=I8), dict(type=-1), dict(T=-1), dict(T=(1 << 40) + 1),
               dict(E=0), dict(E=1025, ldl=1025), dict(ldl=63), dict(k=0), dict(k=65, E=100, ldl=100), dict(k=9, E=8),
               dict(scoring=2), dict(scoring=0), dict(scale=float("inf")), dict(scale=float("nan")), dict(ids=D), dict(ids=A),
               dict(w=A), dict(w=B), dict(ids=B), dict(w=at((3 << 36) + 4 * 4 * 8 - 4))):
        assert call(**kw) == INVALID, kw
    assert call(T=0) == OK
    assert call(T=0, l=None, ids=None, w=None) == OK


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        bk.head_norm(torch.zeros(2, 4, 64))
    with pytest.raises(ValueError):
        bk.route(torch.zeros(2, 8), 2)


def test_lora_refuses():
    f = bk.LIB.bakron_lora
    ok = dict(X=A, xtype=BF16, T=3, n=64, ldx=64, xs=None, A=B, B=C, wtype=BF16, R=4, r=8, m=32, scales=D, ids=E, base=F,
              btype=F32, ldb=32, Y=G, ytype=F16, ldy=32, ws=None, wb=0, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    for kw in (dict(X=None), dict(A=None), dict(B=None), dict(ids=None), dict(Y=None), dict(T=-1), dict(T=(1 << 40) + 1),
               dict(n=0), dict(m=0), dict(n=1 << 28, ldx=1 << 28), dict(m=1 << 28, ldb=1 << 28, ldy=1 << 28), dict(r=0),
               dict(r=513), dict(R=0), dict(R=1 << 31), dict(xtype=9), dict(wtype=F16), dict(wtype=I8),
               dict(xtype=I8, wtype=F32), dict(xtype=F32), dict(ytype=I8), dict(btype=E4M3), dict(ldx=63), dict(ldb=31), dict(ldy=31),
               dict(Y=A), dict(Y=B), dict(Y=C), dict(Y=D), dict(Y=E), dict(Y=F), dict(Y=F, ytype=F32, ldy=33),
               dict(Y=at((6 << 36) + 4), ytype=F32), dict(xs=G)):
        assert call(**kw) == INVALID, kw
    assert call(T=0) == OK
    assert call(T=0, X=None, A=None, B=None, ids=None, base=None, Y=None) == OK
    wb = bk.LIB.bakron_lora_workspace_bytes(200, 8)
    assert bk.LIB.bakron_lora_workspace_bytes(128, 32) == 0 < wb
    W = at(8 << 36)
    for kw in (dict(), dict(ws=W, wb=wb - 1), dict(ws=None, wb=wb)):
        assert call(T=200, **kw) == WORKSPACE, kw
    for kw in (dict(ws=G), dict(ws=A), dict(ws=F), dict(ws=E), dict(ws=at((8 << 36) + 8)), dict(ws=at((7 << 36) - 16))):
        assert call(T=200, **{"ws": W, "wb": wb, **kw}) == INVALID, kw
    for bad in ((-1, 8), ((1 << 40) + 1, 8), (100, 0), (100, 513)):
        assert bk.LIB.bakron_lora_workspace_bytes(*bad) == 0


def test_lora_binding_refuses_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):
        bk.lora(z(2, 8), z(1, 4, 8), z(1, 6, 4), z(2, dtype=torch.int32))


def test_experts_refuses():
    f, nb = bk.LIB.bakron_experts, bk.LIB.bakron_packed_bytes
    ws = bk.LIB.bakron_experts_workspace_bytes
    gb, db, wb = 4 * nb(32, 64, 4, 32), 4 * nb(64, 32, 2, 0), ws(5, 2, 4, 64, 32)
    assert wb > 0
    ok = dict(gate=A, up=B, gb=gb, bits=4, group=32, down=C, db=db, dbits=2, dgroup=0, E=4, n=64, I=32, X=D, xtype=BF16, T=5, ldx=64,
              xs=None, ids=E, w=F, k=2, act=0, Y=G, ytype=F32, ldy=64, ws=at(8 << 36), wb=wb, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    for kw in (dict(gate=None), dict(up=None), dict(down=None), dict(X=None), dict(ids=None), dict(w=None), dict(Y=None), dict(T=-1),
               dict(T=(1 << 40) + 1), dict(n=0), dict(I=0), dict(n=(1 << 18) + 1, ldx=1 << 19, ldy=1 << 19), dict(I=(1 << 18) + 1),
               dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(bits=5), dict(dbits=0), dict(group=16), dict(dgroup=33),
               dict(xtype=5), dict(ytype=I8), dict(act=2), dict(act=-1), dict(ldx=63), dict(ldy=63), dict(gate=at((1 << 36) + 8)),
               dict(down=at((3 << 36) + 4)), dict(ws=at((8 << 36) + 8)), dict(Y=A), dict(Y=B), dict(Y=C), dict(Y=D), dict(Y=E), dict(Y=F),
               dict(ws=A), dict(ws=D), dict(ws=E), dict(ws=G), dict(xs=G), dict(xs=at(8 << 36))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(gb=gb - 1), dict(db=db - 1), dict(wb=wb - 1), dict(ws=None)):
        assert call(**kw) == WORKSPACE, kw
    assert call(T=0) == OK
    assert call(T=0, gate=None, up=None, down=None, X=None, ids=None, w=None, Y=None, ws=None) == OK
    for bad in ((0, 2, 4, 64, 32), (-1, 2, 4, 64, 32), (5, 0, 4, 64, 32), (5, 65, 4, 64, 32), (5, 2, 0, 64, 32), (5, 2, 1025, 64, 32),
                (5, 2, 4, 0, 32), (5, 2, 4, 64, (1 << 18) + 1)):
        assert ws(*bad) == 0, bad


def test_experts_workspace_does_not_grow_past_a_round():
    """Prompts go through in rounds: the workspace of a million tokens is that of a round."""
    ws = bk.LIB.bakron_experts_workspace_bytes
    assert ws(1 << 20, 8, 64, 2048, 1408) == ws(1 << 14, 8, 64, 2048, 1408) < 1 << 30
    assert ws(1, 2, 8, 4096, 14336) < 1 << 20


def test_packed_experts_refuse_other_bytes():
    nb = bk.LIB.bakron_packed_bytes(64, 256, 4, 128)
    data = torch.zeros(3 * nb, dtype=torch.uint8)
    assert bk.PackedExperts(data, 3, 64, 256, 4, 128).nbytes == 3 * nb
    for d, e in ((data[:-1], 3), (data, 2), (data, 0), (data.int(), 3), (data[:1].expand(3 * nb), 3)):
        with pytest.raises(ValueError):
            bk.PackedExperts(d, e, 64, 256, 4, 128)
    with pytest.raises(ValueError):
        bk.pack_experts(torch.zeros(2, 4, 64, dtype=torch.uint8), torch.ones(2, 4), 4)


def test_ends_of_rows_do_not_wrap():
    """Rows so far apart that 64 bits would take the last one's address round to the first's: an output between the first
    two of them lies in their range."""
    far, between = 1 << 61, at((1 << 36) + 4096)  # of 16 bits an element: 5 rows end where they begin
    lib, nb = bk.LIB, bk.LIB.bakron_packed_bytes
    heads = dict(Q=A, hq=4, qt=far, qh=64, K=None, hk=0, kt=0, kh=0, type=BF16, T=5, d=64, qg=None, kg=None, gtype=BF16, eps=1e-6, norm=1,
                 pos=None, pos32=0, freq=None, rot=0, inter=0, YQ=between, yqt=256, yqh=64, YK=None, ykt=0, ykh=0, stream=None)
    assert lib.bakron_head_norm(*heads.values()) == INVALID
    # heads that hold tokens, as far apart
    assert lib.bakron_head_norm(*{**heads, "hq": 5, "T": 4, "qt": 64, "qh": far}.values()) == INVALID
    assert lib.bakron_lora(A, BF16, 5, 64, far, None, B, C, BF16, 4, 8, 32, D, E, None, 0, 0, between, BF16, 32, None, 0, None) == INVALID
    assert lib.bakron_route(A, BF16, 5, 64, far, 2, 0, None, 1, 1.0, between, D, None) == INVALID
    gb, wb = 4 * nb(32, 64, 4, 0), lib.bakron_experts_workspace_bytes(5, 2, 4, 64, 32)
    assert lib.bakron_experts(B, C, gb, 4, 0, D, 4 * nb(64, 32, 4, 0), 4, 0, 4, 64, 32, A, BF16, 5, far, None, E, F, 2, 0, between, BF16, 64,
                              at(8 << 36), wb, None) == INVALID
    assert lib.bakron_matvec(B, nb(32, 64, 4, 0), 32, 64, 4, 0, A, BF16, 5, far, None, between, BF16, 32, None) == INVALID
    assert lib.bakron_rmsnorm(A, BF16, 5, 64, far, None, 0, None, 0, None, BF16, 1e-6, 0, 0, between, BF16, 64, None, None) == INVALID


def test_head_norm_refuses_heads_that_cross():
    """Queries and keys of one head side by side, [token][head][q k v]: outputs that share an element with an input or output
    of another head, token or place."""
    base, e = 1 << 36, 2
    ok = dict(Q=A, hq=4, qt=768, qh=192, K=at(base + 64 * e), hk=4, kt=768, kh=192, type=BF16, T=3, d=64, qg=None, kg=None, gtype=BF16, eps=1e-6,
              norm=1, pos=None, pos32=0, freq=None, rot=0, inter=0, YQ=A, yqt=768, yqh=192, YK=at(base + 64 * e), ykt=768, ykh=192, stream=None)
    for kw in (dict(YK=A), dict(YQ=at(base + 64 * e)), dict(YK=at(base + 63 * e)), dict(YK=at(base + 65 * e)), dict(YK=at(base + (128 + 1) * e)),
               dict(YQ=at(base + 192 * e)), dict(YQ=at(base + 768 * e)), dict(YQ=at(base + (768 + 3 * 192) * e)), dict(YK=at(base - 1 * e)),
               dict(YK=at(base - (3 * 192 - 63) * e)), dict(YK=at(base + 64 * e), ykh=191), dict(YQ=A, yqt=769), dict(YQ=at(base - 2 * 768 * e)),
               # heads that hold tokens
               dict(qt=192, qh=768, kt=192, kh=768, yqt=192, yqh=768, ykt=192, ykh=768, YK=at(base + 32 * e))):
        assert bk.LIB.bakron_head_norm(*{**ok, **kw}.values()) == INVALID, kw
