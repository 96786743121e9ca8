"""Argument checks of the 8-bit path's entry points, before any GPU work."""
import ctypes

import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library

FAKE = 0x7F0000000000      # never dereferenced: every case below fails validation
BAD, OK = tcr.ERR_INVALID_ARG, tcr.OK


@pytest.fixture(scope="module")
def lib():
    build_library()
    return tcr.c_api()


def norm_args(**kw):
    a = tcr.tcr_norm_args(x=FAKE, ldx=64, residual=FAKE, ldr=64, weight=FAKE, h=FAKE, ldh=64, y=FAKE, ldy=64,
                          scale=FAKE, rstd=FAKE, rows=4, cols=64, eps=1e-6, dtype=tcr.BF16, y_dtype=tcr.I8)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(x=None), dict(x=FAKE + 1), dict(y=None), dict(scale=None), dict(scale=FAKE + 2), dict(rstd=FAKE + 1),
    dict(residual=FAKE + 1), dict(h=FAKE + 3), dict(weight=FAKE + 1), dict(dtype=tcr.I8), dict(dtype=9),
    dict(y_dtype=tcr.F32), dict(y_dtype=tcr.I32), dict(dtype=tcr.F32, x=FAKE + 2), dict(eps=-1e-9),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=63), dict(ldr=1), dict(ldh=0), dict(ldy=63),
    dict(rows=1 << 31), dict(cols=(1 << 27) + 1), dict(rows=1 << 30, cols=1 << 12, ldx=1 << 12),
    dict(ldx=1 << 47), dict(ldy=(1 << 63) + 5),
])
def test_norm_refuses(lib, change):
    assert lib.tcr_rmsnorm(ctypes.byref(norm_args(**change)), None) == BAD


def test_norm_of_no_rows(lib):
    assert lib.tcr_rmsnorm(None, None) == BAD
    assert lib.tcr_rmsnorm(ctypes.byref(norm_args(rows=0, x=None, y=None, scale=None)), None) == OK
    assert lib.tcr_rmsnorm(ctypes.byref(norm_args(rows=0, dtype=7)), None) == BAD


def back_args(**kw):
    a = tcr.tcr_norm_back_args(dy=FAKE, lddy=64, h=FAKE, ldh=64, weight=FAKE, rstd=FAKE, dh=FAKE, lddh=64, dx=FAKE,
                               lddx=64, dweight=FAKE, rows=4, cols=64, dtype=tcr.F16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(dy=None), dict(h=None), dict(dx=None), dict(rstd=None), dict(rstd=FAKE + 2), dict(dweight=FAKE + 1),
    dict(dy=FAKE + 1), dict(dh=FAKE + 1), dict(weight=FAKE + 1), dict(dtype=tcr.I8), dict(dtype=-1), dict(lddy=63),
    dict(ldh=8), dict(lddh=63), dict(lddx=0), dict(rows=1 << 31), dict(cols=1 << 28),
])
def test_backward_refuses(lib, change):
    assert lib.tcr_rmsnorm_backward(ctypes.byref(back_args(**change)), None) == BAD


def test_backward_of_nothing(lib):
    assert lib.tcr_rmsnorm_backward(None, None) == BAD
    assert lib.tcr_rmsnorm_backward(ctypes.byref(back_args(rows=0, dweight=None)), None) == OK
    assert lib.tcr_rmsnorm_backward(ctypes.byref(back_args(cols=0)), None) == OK


@pytest.mark.parametrize("args", [
    # (x, ldx, gate, ldg, q, ldq, scale, rows, cols, dtype)
    (None, 64, None, 0, FAKE, 64, FAKE, 4, 64, tcr.BF16),
    (FAKE + 1, 64, None, 0, FAKE, 64, FAKE, 4, 64, tcr.BF16),
    (FAKE, 64, FAKE + 1, 64, FAKE, 64, FAKE, 4, 64, tcr.BF16),
    (FAKE, 64, FAKE, 63, FAKE, 64, FAKE, 4, 64, tcr.BF16),
    (FAKE, 63, None, 0, FAKE, 64, FAKE, 4, 64, tcr.BF16),
    (FAKE, 64, None, 0, None, 64, FAKE, 4, 64, tcr.BF16),
    (FAKE, 64, None, 0, FAKE, 0, FAKE, 4, 64, tcr.BF16),
    (FAKE, 64, None, 0, FAKE, 64, None, 4, 64, tcr.BF16),
    (FAKE, 64, None, 0, FAKE, 64, FAKE + 1, 4, 64, tcr.BF16),
    (FAKE, 64, None, 0, FAKE, 64, FAKE, 4, 64, tcr.I8),
    (FAKE, 64, None, 0, FAKE, 64, FAKE, 1 << 31, 64, tcr.BF16),
])
def test_quantiser_refuses(lib, args):
    assert lib.tcr_quantize_rows_i8(*args, None) == BAD


@pytest.mark.parametrize("args", [
    # (q, ldq, scale, y, ldy, rows, cols, dtype)
    (None, 64, FAKE, FAKE, 64, 4, 64, tcr.F32),
    (FAKE, 60, FAKE, FAKE, 64, 4, 64, tcr.F32),
    (FAKE, 64, None, FAKE, 64, 4, 64, tcr.F32),
    (FAKE, 64, FAKE, None, 64, 4, 64, tcr.F32),
    (FAKE, 64, FAKE, FAKE + 2, 64, 4, 64, tcr.F32),
    (FAKE, 64, FAKE, FAKE, 0, 4, 64, tcr.F32),
    (FAKE, 64, FAKE, FAKE, 64, 4, 64, tcr.I32),
])
def test_reader_of_codes_refuses(lib, args):
    assert lib.tcr_dequantize_rows_i8(*args, None) == BAD
    assert lib.tcr_dequantize_rows_i8(None, 0, None, None, 0, 0, 64, tcr.F32, None) == OK


@pytest.mark.parametrize("args,status", [
    # (A, lda, W, ldw, scale_a, scale_w, C, ldc, M, N, K, dtype)
    ((None, 64, FAKE, 64, None, None, FAKE, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, None, 64, None, None, FAKE, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, FAKE, 64, None, None, None, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 63, FAKE, 64, None, None, FAKE, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 0, FAKE, 64, None, None, FAKE, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, FAKE, 63, None, None, FAKE, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, FAKE, 64, None, None, FAKE, 7, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, FAKE, 64, FAKE + 2, None, FAKE, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, FAKE, 64, None, FAKE + 1, FAKE, 8, 4, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, FAKE, 64, None, None, FAKE + 1, 8, 4, 8, 64, tcr.BF16), BAD),
    ((FAKE, 64, FAKE, 64, None, None, FAKE, 8, 4, 8, 64, tcr.I8), BAD),
    ((FAKE, 64, FAKE, 64, None, None, FAKE, 8, 1 << 31, 8, 64, tcr.F32), BAD),
    ((FAKE, 64, FAKE, 64, None, None, FAKE, 1 << 20, 1 << 20, 1 << 20, 64, tcr.F32), BAD),
    ((FAKE, 1 << 18, FAKE, 1 << 18, None, None, FAKE, 8, 4, 8, 131072, tcr.F32), tcr.ERR_UNSUPPORTED),
])
def test_product_refuses(lib, args, status):
    assert lib.tcr_gemm_i8(*args, None) == status


def test_product_of_nothing(lib):
    assert lib.tcr_gemm_i8(None, 0, None, 0, None, None, None, 0, 0, 8, 64, tcr.F32, None) == OK
    assert lib.tcr_gemm_i8(None, 0, None, 0, None, None, None, 0, 8, 0, 64, tcr.F32, None) == OK
