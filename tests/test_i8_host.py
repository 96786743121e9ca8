"""Argument checks of the 8-bit path's entry points, before any GPU work."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import BIND_PATH, build_library

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


def test_a_scale_that_nothing_would_write_is_refused():
    torch = pytest.importorskip("torch")
    x, scale = torch.zeros(4, 64), torch.zeros(4)
    for kw in (dict(), dict(out_dtype=torch.float32), dict(out=torch.zeros(4, 64))):
        with pytest.raises(ValueError, match="scale"):
            tcr.tcr_rmsnorm(x, scale=scale, **kw)


SLOW_C = """
#include <time.h>
int slow(void)                /* stands for an entry point that waits */
{
    struct timespec t = {0, 300000000};
    nanosleep(&t, 0);
    return 0;
}
"""

# The binding knows tensors by their attributes only; its module is set up in
# a process of its own with the waiting function for all five entry points.
SLOW_PY = """
import ctypes, importlib.machinery, importlib.util, sys, threading, time
loader = importlib.machinery.ExtensionFileLoader("_tcrbind", sys.argv[1])
m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_tcrbind", sys.argv[1], loader=loader))
loader.exec_module(m)
slow = ctypes.cast(ctypes.CDLL(sys.argv[2]).slow, ctypes.c_void_p).value
m.setup("f16", "bf16", "f32", "i8", "i32", lambda dev: 0, lambda: 0, lambda dev: None, RuntimeError, *[slow] * 5)

class Tensor:
    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape
    def stride(self):
        return (self.shape[1], 1) if len(self.shape) == 2 else (1,)
    def data_ptr(self):
        return 256
    def get_device(self):
        return 0

x, q, c, s, w = Tensor("bf16", 4, 8), Tensor("i8", 4, 8), Tensor("bf16", 4, 4), Tensor("f32", 4), Tensor("bf16", 8)
ticks, stop = [], False

def tick():
    while not stop:
        ticks.append(time.monotonic())
        time.sleep(0.01)

threading.Thread(target=tick, daemon=True).start()
for call in (lambda: m.rmsnorm(x, w, None, 1e-6, None, x, None, s, None),
             lambda: m.rmsnorm_backward(x, x, w, s, None, x, None, None),
             lambda: m.quantize_rows(x, None, q, s, None),
             lambda: m.dequantize_rows(q, s, x, None),
             lambda: m.gemm(q, q, s, s, c, None)):
    a = time.monotonic()
    call()
    b = time.monotonic()
    assert b - a >= 0.29, b - a
    print(sum(a + 0.05 < t < b - 0.05 for t in ticks))
stop = True
"""


def test_calls_leave_the_interpreter_to_other_threads(lib, tmp_path):
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    (tmp_path / "slow.c").write_text(SLOW_C)
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "slow.c"), "-o", str(tmp_path / "slow.so")], check=True)
    r = subprocess.run([sys.executable, "-c", SLOW_PY, BIND_PATH, str(tmp_path / "slow.so")], capture_output=True,
                       text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    counts = [int(n) for n in r.stdout.split()]
    assert len(counts) == 5 and min(counts) >= 1, counts
