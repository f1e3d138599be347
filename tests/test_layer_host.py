"""Refusals of the C entry points of the 8-bit form, the norm and the routing, before anything is
enqueued (no GPU)."""
import math

import pytest

import error_bounded_lossy_amd as ec

OK, INVALID, CAPACITY, UNSUPPORTED = (ec.EC_OK, ec.EC_ERR_INVALID, ec.EC_ERR_CAPACITY, ec.EC_ERR_UNSUPPORTED)
F = 1 << 20  # a pointer that is never dereferenced: every call below fails its checks or has no work
F32, BF16 = 0, 2


@pytest.fixture(scope="module")
def L():
    return ec.lib()


def test_quantization(L):
    q, d = L.ec_i8_quantize, L.ec_i8_dequantize
    assert q(None, BF16, 0, 8, 8, None, None, None) == OK
    for args in ((F, 3, 1, 8, 8, F, F), (F, -1, 1, 8, 8, F, F), (F, BF16, 1, 0, 8, F, F), (F, BF16, 1, 8, 7, F, F),
                 (None, BF16, 1, 8, 8, F, F), (F + 1, BF16, 1, 8, 8, F, F), (F + 2, F32, 1, 8, 8, F, F),
                 (F, BF16, 1, 8, 8, F + 8, F), (F, BF16, 1, 8, 8, F, F + 2), (F, BF16, 1, 8, 8, F, None), (F, BF16, 1, 8, 8, None, F)):
        assert q(*args, None) == INVALID, args
    assert q(F, BF16, 1, (1 << 24) + 1, 1 << 25, F, F, None) == UNSUPPORTED
    assert q(F, BF16, 1 << 31, 8, 8, F, F, None) == UNSUPPORTED
    assert d(None, None, 0, 8, None, BF16, 8, None) == OK
    for args in ((F, F, 1, 8, None, BF16, 8), (F, F, 1, 8, F + 1, BF16, 8), (F + 1, F, 1, 8, F, BF16, 8), (F, F + 1, 1, 8, F, BF16, 8),
                 (F, F, 1, 8, F, 7, 8), (F, F, 1, 8, F, BF16, 4), (F, F, 1, 0, F, BF16, 4)):
        assert d(*args, None) == INVALID, args


def test_products(L):
    p, e = L.ec_i8_product, L.ec_i8_product_experts
    assert p(None, None, 0, None, None, 8, 128, None, BF16, None) == OK
    for args in ((F, F, 1, F, F, 0, 128, F, BF16), (F, F, 1, F, F, 8, 100, F, BF16), (F, F, 1, F, F, 8, 0, F, BF16),
                 (F, F, 1, F, F, 8, 128, F, 5), (F, F, 1, F, F, 8, 128, None, BF16), (F, F, 1, F, F, 8, 128, F + 1, BF16),
                 (F + 4, F, 1, F, F, 8, 128, F, BF16), (F, F, 1, F + 8, F, 8, 128, F, BF16), (F, F + 2, 1, F, F, 8, 128, F, BF16),
                 (F, F, 1, F, None, 8, 128, F, BF16), (None, F, 1, F, F, 8, 128, F, BF16)):
        assert p(*args, None) == INVALID, args
    assert p(F, F, 1, F, F, 8, 131072, F, BF16, None) == UNSUPPORTED
    assert p(F, F, 1 << 31, F, F, 8, 128, F, BF16, None) == UNSUPPORTED
    assert p(F, F, 1, F, F, 1 << 31, 128, F, BF16, None) == UNSUPPORTED
    for off, n, want in ((None, 2, INVALID), (F + 2, 2, INVALID), (F, 0, INVALID), (F, 1025, UNSUPPORTED)):
        assert e(F, F, 1, F, F, 8, 128, off, n, F, BF16, None) == want
    assert e(None, None, 0, None, None, 8, 128, F, 2, None, BF16, None) == OK
    assert e(F, F, 1, F, F, 8, 64, F, 2, F, BF16, None) == INVALID


def test_products_in_parts(L):
    p, size = L.ec_i8_product_parts, L.ec_i8_product_parts_bytes
    for rows, cols, depth in ((16, 64, 12160), (257, 64, 16384), (0, 64, 16384), (17, 0, 16384), (17, 64, 0), (17, 64, 16400), (17, 64, 131072),
                              (17, 1 << 31, 16384), (17, (1 << 64) - 1, 16384), ((1 << 64) - 1, 64, 16384), (17, 64, 4992), (17, 64, (1 << 64) - 128)):
        assert size(rows, cols, depth) == 0, (rows, cols, depth)
    assert L.ec_i8_linear_workspace_bytes(100, 16384, 0, 0) == 100 * (16384 + 4)
    assert size(1, 128, 12288) == 12 * 128 * 4 and size(16, 8192, 12288) == 4 * 16 * 8192 * 4
    for rows in (17, 64, 65, 256):
        for cols in (1, 64, 1000, 4096):
            for depth in (5632, 16384, 130944):
                need, row = size(rows, cols, depth), rows * ((cols + 63) // 64 * 64) * 4
                if rows <= 64 or cols <= 1000:
                    assert need >= 2 * row, (rows, cols, depth)
                # no part is empty, and no more workgroups than fill the units twice
                parts = need // row
                assert need == parts * row and parts <= depth // 128 // 8
                assert parts * -(-rows // 64) * -(-cols // 64) <= 512
                each = -(-depth // 128 // parts) if parts else 0
                assert parts * each < depth // 128 + each if parts else True
    need = size(100, 64, 16384)
    good = [F, F, 100, F, F, 64, 16384, F, BF16]
    assert p(None, None, 0, None, None, 8, 128, None, BF16, None, 0, None) == OK
    assert p(*good, F, need - 1, None) == CAPACITY
    assert p(*good, F + 8, need, None) == INVALID
    assert p(*good, None, need, None) == INVALID
    assert p(F, F, 100, F, F, 8, 100, F, BF16, F, need, None) == INVALID
    assert p(F, F, 1, F, F, 8, 131072, F, BF16, F, need, None) == UNSUPPORTED


def test_linear(L):
    lin = L.ec_i8_linear
    assert L.ec_i8_linear_workspace_bytes(0, 64, 8, 0) == 0
    need = L.ec_i8_linear_workspace_bytes(100, 64, 8, 0)
    assert need == 100 * 132
    assert lin(F, BF16, 0, 64, 64, F, F, 8, None, 0, F, None, 0, None) == OK
    assert lin(F, BF16, 100, 64, 64, F, F, 8, None, 0, F, None, need, None) == INVALID
    assert lin(F, BF16, 100, 64, 64, F, F, 8, None, 0, F, F, need - 1, None) == CAPACITY
    for args in ((F, BF16, 100, 64, 64, F, F, 8, None, 0, F, F + 8), (F, BF16, 100, 64, 63, F, F, 8, None, 0, F, F),
                 (F, BF16, 100, 64, 64, F, F, 8, F, 0, F, F), (F, BF16, 100, 64, 64, F, F, 8, None, 3, F, F),
                 (F, BF16, 100, 64, 64, F, F, 0, None, 0, F, F), (F, BF16, 100, 0, 64, F, F, 8, None, 0, F, F),
                 (F, 4, 100, 64, 64, F, F, 8, None, 0, F, F), (None, BF16, 100, 64, 64, F, F, 8, None, 0, F, F),
                 (F, BF16, 100, 64, 64, F, None, 8, None, 0, F, F), (F, BF16, 100, 64, 64, F + 4, F, 8, None, 0, F, F),
                 (F, BF16, 100, 64, 64, F, F, 8, F + 1, 2, F, F)):
        assert lin(*args, need, None) == INVALID, args
    assert lin(F, BF16, 100, 64, 64, F, F, 8, F, 1025, F, F, need, None) == UNSUPPORTED
    assert lin(F, BF16, 1, 130945, 130945, F, F, 8, None, 0, F, F, 1 << 30, None) == UNSUPPORTED


def test_norm(L):
    n, q, b = L.ec_rms_norm, L.ec_rms_norm_i8, L.ec_rms_norm_backward
    good = dict(x=F, xs=8, r=F, rs=8, t=BF16, rows=4, cols=8, w=F, wt=BF16, eps=1e-5, h=F)

    def args(**kw):
        return list({**good, **kw}.values())

    assert n(*args(rows=0, x=None, r=None, h=None, w=None), None, None, None) == OK
    assert q(*args(rows=0, x=None, r=None, h=None, w=None), None, None, None) == OK
    for kw in (dict(t=3), dict(wt=-1), dict(cols=0), dict(xs=7), dict(rs=7), dict(r=None), dict(h=None), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(eps=1e-60), dict(x=None), dict(x=F + 1), dict(r=F + 1),
               dict(h=F + 1), dict(w=None), dict(w=F + 1), dict(wt=F32, w=F + 2)):
        assert n(*args(**kw), F, F, None) == INVALID, kw
        assert q(*args(**kw), F, F, None) == INVALID, kw
    for kw in (dict(rows=1 << 31), dict(cols=(1 << 24) + 1, xs=1 << 25, rs=1 << 25)):
        assert n(*args(**kw), F, F, None) == UNSUPPORTED, kw
        assert q(*args(**kw), F, F, None) == UNSUPPORTED, kw
    assert n(*args(), None, F, None) == INVALID and n(*args(), F + 1, F, None) == INVALID and n(*args(), F, F + 2, None) == INVALID
    assert q(*args(), F + 8, F, None) == INVALID and q(*args(), F, F + 1, None) == INVALID and q(*args(), None, F, None) == INVALID

    need = L.ec_rms_norm_backward_workspace_bytes(100, 64)
    assert need > 0 and need % (64 * 4) == 0 and L.ec_rms_norm_backward_workspace_bytes(0, 64) == 0
    assert L.ec_rms_norm_backward_workspace_bytes(100, 0) == 0
    back = dict(dy=F, h=F, dh=F, t=BF16, rows=100, cols=64, rstd=F, w=F, wt=BF16, dx=F, dw=F, ws=F, n=need)

    def args(**kw):
        return list({**back, **kw}.values())

    for kw in (dict(dy=None), dict(h=None), dict(dh=F + 1), dict(t=9), dict(wt=9), dict(cols=0), dict(rstd=None), dict(rstd=F + 2),
               dict(w=None), dict(dx=None), dict(dx=F + 1), dict(dw=None), dict(dw=F + 1), dict(ws=None), dict(ws=F + 8)):
        assert b(*args(**kw), None) == INVALID, kw
    assert b(*args(n=need - 1), None) == CAPACITY
    assert b(*args(rows=1 << 31), None) == UNSUPPORTED


def test_routing(L):
    r, b = L.ec_expert_route, L.ec_expert_route_backward
    good = dict(l=F, t=F32, tokens=4, stride=16, experts=16, bias=None, k=2, score=1, g=4, tg=2, n=1, scale=1.0, ids=F, w=F)

    def args(**kw):
        return list({**good, **kw}.values())

    assert r(*args(tokens=0, l=None, ids=None, w=None), None) == OK
    for kw in (dict(t=3), dict(experts=0), dict(stride=15), dict(k=0), dict(score=2), dict(score=-1), dict(g=0), dict(g=3), dict(tg=0),
               dict(tg=5), dict(k=9), dict(scale=math.nan), dict(scale=math.inf), dict(l=None), dict(l=F + 2), dict(bias=F + 1),
               dict(ids=None), dict(ids=F + 1), dict(w=None), dict(w=F + 2)):
        assert r(*args(**kw), None) == INVALID, kw
    for kw in (dict(experts=1028, stride=1028), dict(experts=256, stride=256, k=65), dict(tokens=1 << 31), dict(tokens=1 << 30, k=4),
               dict(experts=130, stride=130, g=65, tg=65)):
        assert r(*args(**kw), None) == UNSUPPORTED, kw
    back = dict(dw=F, l=F, t=F32, tokens=4, stride=16, experts=16, ids=F, k=2, score=0, n=1, scale=1.0, dl=F)

    def args(**kw):
        return list({**back, **kw}.values())

    assert b(*args(tokens=0, dw=None), None) == OK
    for kw in (dict(dw=None), dict(dw=F + 1), dict(l=F + 1), dict(t=4), dict(stride=3), dict(experts=0), dict(ids=None), dict(k=0),
               dict(score=7), dict(scale=math.nan), dict(dl=None), dict(dl=F + 2)):
        assert b(*args(**kw), None) == INVALID, kw
    for kw in (dict(experts=1025, stride=1025), dict(k=65), dict(tokens=1 << 31)):
        assert b(*args(**kw), None) == UNSUPPORTED, kw


def test_dispatch(L):
    d = L.ec_expert_dispatch_i8
    good = dict(x=F, xs=F, tokens=4, padded=128, place=F, k=2, off=F, e=4, c=F, s=F)

    def args(**kw):
        return list({**good, **kw}.values())

    assert d(*args(tokens=0, x=None), None) == OK
    for kw in (dict(x=None), dict(x=F + 8), dict(xs=F + 2), dict(padded=0), dict(padded=100), dict(place=None), dict(place=F + 1),
               dict(k=0), dict(off=None), dict(e=0), dict(c=F + 4), dict(c=None), dict(s=None), dict(s=F + 1)):
        assert d(*args(**kw), None) == INVALID, kw
    for kw in (dict(k=65), dict(e=1025), dict(padded=(1 << 24) + 128), dict(tokens=1 << 31)):
        assert d(*args(**kw), None) == UNSUPPORTED, kw
