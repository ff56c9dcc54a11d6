"""Refusals of the 4-bit entry points and their layout sizes, without a GPU."""
import ctypes

import pytest
import torch

import post_quantization_kronq_b200 as kq
from oracle import fp4
from post_quantization_kronq_b200 import _lib

L = _lib.lib
P = ctypes.c_void_p(4096)          # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(4097)
BAD, UNSUP = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED
BIG = 1 << 40


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257, 4095, 28672])
def test_row_bytes(n):
    assert kq.kronq_fp4_code_row_bytes(n) == fp4.code_row_bytes(n)
    for fmt in (kq.MXFP4, kq.NVFP4):
        assert kq.kronq_fp4_scale_row_bytes(fmt, n) == fp4.scale_row_bytes(fmt, n)


def test_row_bytes_of_bad_arguments():
    assert kq.kronq_fp4_code_row_bytes(0) == 0 and kq.kronq_fp4_code_row_bytes(-5) == 0
    assert kq.kronq_fp4_scale_row_bytes(2, 64) == 0 and kq.kronq_fp4_scale_row_bytes(kq.MXFP4, -1) == 0
    assert kq.kronq_fp4_quantize_workspace_bytes(0, 64, kq.NVFP4) == 0
    assert kq.kronq_fp4_quantize_workspace_bytes(8, 64, kq.MXFP4) == 0
    assert kq.kronq_fp4_quantize_workspace_bytes(8, 64, kq.NVFP4) > 0
    for f in (kq.kronq_fp4_matmul_workspace_bytes, kq.kronq_fp4_matvec_workspace_bytes):
        assert f(0, 64, 64, 0) == 0 and f(4, -1, 64, 0) == 0 and f(4, 64, 64, 7) == 0


def quantize(x=P, dt=1, rows=8, n=64, ldx=64, fmt=1, codes=P, scales=P, g=P, given=1, deq=None, ldd=0, ws=None, nb=0):
    return L.kronq_fp4_quantize(x, dt, rows, n, ldx, fmt, codes, scales, g, given, deq, ldd, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(fmt=2), dict(dt=2), dict(rows=-1), dict(n=0), dict(n=BIG, ldx=BIG), dict(ldx=63), dict(deq=P, ldd=63),
    dict(x=None), dict(codes=None), dict(scales=None), dict(g=None), dict(fmt=0), dict(codes=ctypes.c_void_p(4104)),
    dict(scales=ctypes.c_void_p(4104)), dict(x=ODD), dict(deq=ODD, ldd=64), dict(g=ODD),
    dict(ldx=(1 << 32) + 1), dict(deq=P, ldd=(1 << 32) + 1), dict(given=0), dict(given=0, ws=P, nb=16), dict(given=0, ws=ctypes.c_void_p(4104), nb=1 << 20)])
def test_quantize_refusals(kw):
    assert quantize(**kw) == BAD
    assert b"fp4_quantize" in L.kronq_last_error()


def test_quantize_of_no_rows_is_a_no_op():
    assert quantize(rows=0) == _lib.OK


def dequantize(codes=P, scales=P, g=P, fmt=1, rows=8, n=64, out=P, dt=1, ldo=64):
    return L.kronq_fp4_dequantize(codes, scales, g, fmt, rows, n, out, dt, ldo, None)


@pytest.mark.parametrize("kw", [
    dict(fmt=-1), dict(dt=5), dict(rows=-1), dict(n=0), dict(ldo=63), dict(ldo=(1 << 32) + 1), dict(codes=None), dict(scales=None), dict(out=None),
    dict(g=None), dict(fmt=0), dict(codes=ODD), dict(scales=ODD), dict(out=ODD)])
def test_dequantize_refusals(kw):
    assert dequantize(**kw) == BAD


def matmul(xc=P, xs=P, xg=P, wc=P, ws=P, wg=P, fmt=1, T=8, m=64, n=64, y=P, ydt=0, ldy=64, w=P, nb=1 << 40):
    return L.kronq_fp4_matmul(xc, xs, xg, wc, ws, wg, fmt, T, m, n, y, ydt, ldy, w, nb, None)


def grouped(xc=P, xs=P, xg=P, off=P, E=4, wc=P, ws=P, wg=P, fmt=1, T=8, m=64, n=64, y=P, ydt=0, ldy=64):
    return L.kronq_fp4_grouped_matmul(xc, xs, xg, off, E, wc, ws, wg, fmt, T, m, n, y, ydt, ldy, None)


PRODUCT = [dict(fmt=2), dict(ydt=2), dict(T=-1), dict(m=0), dict(n=0), dict(n=BIG), dict(m=BIG, ldy=BIG), dict(ldy=63),
           dict(ldy=(1 << 32) + 1),
           dict(wc=None), dict(ws=None), dict(y=None), dict(wg=None), dict(fmt=0), dict(wc=ODD), dict(ws=ODD), dict(y=ODD)]
TOKENS = [dict(xc=None), dict(xs=None), dict(xg=None), dict(xc=ODD), dict(xs=ODD), dict(xg=ODD)]


@pytest.mark.parametrize("kw", PRODUCT + TOKENS)
def test_matmul_refusals(kw):
    assert matmul(**kw) == BAD
    assert b"fp4_matmul" in L.kronq_last_error()


@pytest.mark.parametrize("kw", PRODUCT + TOKENS + [
    dict(E=0), dict(E=-1), dict(E=1025), dict(off=None), dict(off=ODD), dict(E=1024, m=1 << 21, ldy=1 << 21)])
def test_grouped_refusals(kw):
    assert grouped(**kw) == BAD
    assert b"fp4_grouped_matmul" in L.kronq_last_error()


def matvec(x=P, xdt=0, ldx=64, wc=P, ws=P, wg=P, fmt=1, T=4, m=64, n=64, y=P, ydt=0, ldy=64, w=P, nb=1 << 40):
    return L.kronq_fp4_matvec(x, xdt, ldx, wc, ws, wg, fmt, T, m, n, y, ydt, ldy, w, nb, None)


@pytest.mark.parametrize("kw", PRODUCT + [dict(x=None), dict(xdt=3), dict(ldx=63), dict(x=ODD)])
def test_matvec_refusals(kw):
    assert matvec(**kw) == BAD
    assert b"fp4_matvec" in L.kronq_last_error()


def test_limits():
    assert matvec(T=17) == UNSUP
    n = (1 << 24) + 1
    assert matvec(n=n, ldx=n) == UNSUP and matmul(n=n) == UNSUP and grouped(n=n) == UNSUP
    assert matmul(T=1 << 29, m=1 << 29, ldy=1 << 29) == UNSUP


def test_no_tokens_is_a_no_op():
    for f in (matmul, grouped, matvec):
        assert f(T=0) == _lib.OK


def test_workspaces_are_checked():
    T, m, n = 4, 64, 1 << 17
    for f, size in ((matmul, kq.kronq_fp4_matmul_workspace_bytes), (matvec, kq.kronq_fp4_matvec_workspace_bytes)):
        for fmt in (0, 1):
            need = size(T, m, n, fmt)
            g = dict(wg=None, **({"xg": None} if f is matmul else {})) if fmt == 0 else {}
            ld = dict(ldx=n) if f is matvec else {}
            if need:
                assert f(T=T, m=m, n=n, fmt=fmt, nb=need - 1, **g, **ld) == BAD
                assert f(T=T, m=m, n=n, fmt=fmt, w=None, nb=need, **g, **ld) == BAD
                assert f(T=T, m=m, n=n, fmt=fmt, w=ctypes.c_void_p(4104), nb=need, **g, **ld) == BAD


def test_python_refuses_host_tensors_and_wrong_shapes():
    c, s, x = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 64)
    with pytest.raises(ValueError):
        kq.kronq_fp4_quantize(x, kq.MXFP4, c, s)
    with pytest.raises(ValueError):
        kq.kronq_fp4_dequantize(c, s, kq.MXFP4, x)
    with pytest.raises(ValueError):
        kq.kronq_fp4_matmul(c, s, c, s, kq.MXFP4, 64, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        kq.kronq_fp4_matvec(x, c, s, kq.MXFP4, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        kq.kronq_fp4_grouped_matmul(c, s, torch.zeros(2, dtype=torch.int32), c, s, kq.MXFP4, 64, torch.zeros(4, 4))
