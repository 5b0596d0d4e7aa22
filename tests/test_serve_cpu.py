"""Argument checks of the serving entry points (pack, matvec, rmsnorm); nothing here needs a GPU."""
import ctypes

import pytest
import torch

import kronecker_hessian_rounding_amd as bk

F32, F16, BF16, I8, E4M3 = range(5)
INVALID, WORKSPACE, OK = 1, 3, 0


def at(addr):
    return ctypes.c_void_p(addr)  # never dereferenced: validation fails first


A, B, C, D = at(1 << 32), at(2 << 32), at(3 << 32), at(4 << 32)


def test_packed_bytes():
    f = bk.LIB.bakron_packed_bytes
    # 4-bit: tiles of 16 rows, chunks of 128 columns, 1 KB each, plus fp32 scales of whole tiles
    assert f(16, 128, 4, 0) == 1024 + 64
    assert f(17, 129, 3, 0) == 4 * 1024 + 2 * 64
    assert f(16, 128, 4, 32) == 1024 + 4 * 64
    assert f(16, 129, 4, 32) == 2 * 1024 + 8 * 64      # groups of the padded columns
    assert f(16, 300, 4, 256) == 3 * 1024 + 2 * 64
    # 2-bit: 512 bytes
    assert f(16, 256, 2, 128) == 1024 + 2 * 64
    assert f(16, 257, 1, 0) == 3 * 512 + 64
    for bad in ((0, 4, 4, 0), (4, 0, 4, 0), (4, 4, 0, 0), (4, 4, 5, 0), (4, 4, 4, 16), (4, 4, 4, 48), (4, 4, 4, -32),
                (1 << 26, 4, 4, 0), (4, 1 << 28, 4, 0), (1 << 20, 1 << 17, 4, 0)):
        assert f(*bad) == 0, bad


def test_pack_refuses():
    f = bk.LIB.bakron_pack
    nb = bk.LIB.bakron_packed_bytes(64, 256, 4, 128)
    ok = dict(codes=A, m=64, n=256, ldc=256, bits=4, scales=B, lds=2, group=128, packed=C, nb=nb, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    for kw in (dict(codes=None), dict(scales=None), dict(packed=None), dict(m=0), dict(n=-1), dict(ldc=255),
               dict(bits=0), dict(bits=5), dict(lds=1), dict(group=33), dict(group=16),
               dict(packed=at((3 << 32) + 8)), dict(packed=A), dict(packed=B)):
        assert call(**kw) == INVALID, kw
    assert call(nb=nb - 1) == WORKSPACE


def test_matvec_refuses():
    f = bk.LIB.bakron_matvec
    nb = bk.LIB.bakron_packed_bytes(64, 256, 4, 0)
    ok = dict(packed=A, nb=nb, m=64, n=256, bits=4, group=0, X=B, xtype=BF16, T=3, ldx=256, xs=None, Y=C, ytype=F32,
              ldy=64, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    for kw in (dict(packed=None), dict(packed=at((1 << 32) + 4)), dict(m=0), dict(n=0), dict(bits=6), dict(group=31),
               dict(X=None), dict(Y=None), dict(xtype=5), dict(xtype=-1), dict(ytype=I8), dict(ytype=E4M3),
               dict(T=-1), dict(ldx=255), dict(ldy=63), dict(Y=B), dict(Y=A), dict(T=(1 << 40) + 1),
               dict(xs=C), dict(Y=at((2 << 32) + 2 * 256 * 3 - 2))):
        assert call(**kw) == INVALID, kw
    assert call(nb=nb - 1) == WORKSPACE
    assert call(T=0) == OK
    assert call(T=0, X=None, Y=None) == OK


def test_rmsnorm_refuses():
    f = bk.LIB.bakron_rmsnorm
    ok = dict(X=A, xtype=BF16, T=4, n=64, ldx=64, R=B, ldr=64, H=C, ldh=64, gain=None, gtype=BF16, eps=1e-6, rot=0,
              seed=0, Y=D, ytype=BF16, ldy=64, ys=None, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    near = at((4 << 32) + 64)
    for kw in (dict(X=None), dict(Y=None), dict(T=-1), dict(n=0), dict(xtype=I8), dict(xtype=7), dict(ytype=9),
               dict(ldx=63), dict(ldr=63), dict(ldh=63), dict(ldy=63), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(ytype=I8), dict(ytype=E4M3), dict(gain=near, gtype=F16),
               dict(rot=1, n=32769, ldx=32769, ldr=32769, ldh=32769, ldy=32769), dict(T=1 << 31),
               # overlap: shifted by an element, of another type, or between the outputs
               dict(H=at((1 << 32) + 2)), dict(Y=at((1 << 32) + 2)), dict(Y=A, ytype=F32), dict(Y=C),
               dict(gain=D), dict(gain=C), dict(Y=A, ytype=I8, ys=at(5 << 32)), dict(ytype=I8, ys=D),
               dict(ytype=I8, ys=A)):
        assert call(**kw) == INVALID, kw
    assert call(T=0) == OK


def test_interleaved_rows_do_not_overlap():
    """Columns of one buffer are separate arrays: such a call passes the overlap check and is refused for eps only."""
    f = bk.LIB.bakron_rmsnorm
    base = 1 << 32
    args = [at(base), BF16, 4, 64, 256, at(base + 128), 256, at(base + 256), 256, None, BF16, -1.0, 0, 0,
            at(base + 384), BF16, 256, None, None]
    assert f(*args) == INVALID
    # the same with T = 0 and a valid eps returns before anything is enqueued
    args[11], args[2] = 1e-6, 0
    assert f(*args) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        bk.rmsnorm(x)
    with pytest.raises(ValueError):
        bk.pack(torch.zeros(4, 64, dtype=torch.uint8), torch.ones(4), 4)
    with pytest.raises(ValueError):
        bk.matvec(x, bk.PackedWeight(torch.zeros(1, dtype=torch.uint8), 4, 64, 4, 0))


def test_packed_weight_refuses_other_bytes():
    """A layer made or changed by hand holds exactly the bytes that the products read."""
    nb = bk.LIB.bakron_packed_bytes(64, 256, 4, 128)
    data = torch.zeros(nb, dtype=torch.uint8)
    w = bk.PackedWeight(data, 64, 256, 4, 128)
    assert w.nbytes == nb
    w.data = data[:-1]
    assert w.nbytes == nb - 1  # what a product is told, and refuses
    one = torch.zeros(1, dtype=torch.uint8)
    for bad in (data[:-1], torch.zeros(nb + 1, dtype=torch.uint8), data.int(), one.expand(nb),
                torch.zeros(2 * nb, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            bk.PackedWeight(bad, 64, 256, 4, 128)
    with pytest.raises(ValueError):
        bk.PackedWeight(data, 64, 256, 5, 128)
