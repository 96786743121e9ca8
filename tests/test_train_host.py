"""Argument checks of dropout, the layer norm and the cross entropy, before any
GPU work, and the generator against its published vectors."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import BIND_PATH, build_library
from tests import train_spec as spec
from tests.test_i8_host import SLOW_C, SLOW_PY

FAKE = 0x7F0000000000      # never dereferenced: every case below fails validation
BAD, OK, UNSUPPORTED = tcr.ERR_INVALID_ARG, tcr.OK, tcr.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_library()
    return tcr.c_api()


def test_generator_against_published_vectors():
    for c, k, want in [
        ([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
        ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
        ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
         "d16cfe09 94fdcceb 5001e420 24126ea1"),
    ]:
        got = spec.philox(np.array([c], dtype=np.uint64), k)[0]
        assert " ".join(f"{int(v):08x}" for v in got) == want


def drop(**kw):
    d = tcr.tcr_drop(p=0.5, seed=1, offset=2, state=None)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.pointer(d)


BAD_DROPS = [dict(p=-1e-9), dict(p=1.0000001), dict(p=float("nan")), dict(p=float("inf")), dict(state=FAKE + 4)]


@pytest.mark.parametrize("change", [
    dict(x=None), dict(x=FAKE + 1), dict(y=None), dict(y=FAKE + 1), dict(residual=FAKE + 1), dict(ldx=63), dict(ldr=1),
    dict(ldy=0), dict(rows=1 << 31), dict(cols=(1 << 27) + 1), dict(dtype=tcr.I8), dict(dtype=9),
    dict(dtype=tcr.F32, x=FAKE + 2), dict(ldx=1 << 47), dict(drop=None),
] + [dict(drop=drop(**d)) for d in BAD_DROPS])
def test_dropout_refuses(lib, change):
    a = dict(x=FAKE, ldx=64, residual=FAKE, ldr=64, y=FAKE, ldy=64, rows=4, cols=64, drop=drop(), dtype=tcr.BF16)
    a.update(change)
    assert lib.tcr_dropout(*a.values(), None) == BAD


def test_dropout_of_nothing(lib):
    for rows, cols in ((0, 64), (4, 0)):
        assert lib.tcr_dropout(None, 64, None, 0, None, 64, rows, cols, drop(), tcr.F16, None) == OK


def layer_args(**kw):
    a = tcr.tcr_layernorm_args(x=FAKE, ldx=64, residual=FAKE, ldr=64, weight=FAKE, bias=FAKE, h=FAKE, ldh=64, y=FAKE,
                               ldy=64, scale=FAKE, mean=FAKE, rstd=FAKE, rows=4, cols=64, eps=1e-5, dtype=tcr.BF16,
                               y_dtype=tcr.I8)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(x=None), dict(x=FAKE + 1), dict(y=None), dict(scale=None), dict(scale=FAKE + 2), dict(rstd=FAKE + 1),
    dict(mean=FAKE + 2), dict(residual=FAKE + 1), dict(h=FAKE + 3), dict(weight=FAKE + 1), dict(bias=FAKE + 1),
    dict(dtype=tcr.I8), dict(dtype=9), dict(y_dtype=tcr.F32), dict(y_dtype=tcr.I32), dict(dtype=tcr.F32, bias=FAKE + 2),
    dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=63), dict(ldr=1), dict(ldh=0),
    dict(ldy=63), dict(rows=1 << 31), dict(cols=(1 << 27) + 1), dict(rows=1 << 30, cols=1 << 12, ldx=1 << 12),
] + [dict(drop=drop(**d)) for d in BAD_DROPS])
def test_layernorm_refuses(lib, change):
    assert lib.tcr_layernorm(ctypes.byref(layer_args(**change)), None) == BAD


def layer_back_args(**kw):
    a = tcr.tcr_layernorm_back_args(dy=FAKE, lddy=64, h=FAKE, ldh=64, weight=FAKE, mean=FAKE, rstd=FAKE, dh=FAKE,
                                    lddh=64, dx=FAKE, lddx=64, dresidual=FAKE, lddr=64, dweight=FAKE, dbias=FAKE,
                                    rows=4, cols=64, dtype=tcr.F16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(dy=None), dict(h=None), dict(mean=None), dict(rstd=None), dict(rstd=FAKE + 2), dict(mean=FAKE + 1),
    dict(dweight=FAKE + 1), dict(dbias=FAKE + 2), dict(dx=FAKE + 1), dict(dresidual=FAKE + 1), dict(dy=FAKE + 1),
    dict(dh=FAKE + 1), dict(weight=FAKE + 1), dict(dtype=tcr.I8), dict(dtype=-1), dict(lddy=63), dict(ldh=8),
    dict(lddh=63), dict(lddx=0), dict(lddr=0), dict(rows=1 << 31), dict(cols=1 << 28),
] + [dict(drop=drop(**d)) for d in BAD_DROPS])
def test_layernorm_backward_refuses(lib, change):
    assert lib.tcr_layernorm_backward(ctypes.byref(layer_back_args(**change)), None) == BAD


def test_layernorm_of_nothing(lib):
    assert lib.tcr_layernorm(None, None) == BAD and lib.tcr_layernorm_backward(None, None) == BAD
    assert lib.tcr_layernorm(ctypes.byref(layer_args(rows=0, x=None, y=None, scale=None)), None) == OK
    assert lib.tcr_layernorm_backward(ctypes.byref(layer_back_args(rows=0, dweight=None, dbias=None)), None) == OK
    assert lib.tcr_layernorm_backward(ctypes.byref(layer_back_args(cols=0)), None) == OK
    none = dict(dx=None, dresidual=None, dweight=None, dbias=None)
    assert lib.tcr_layernorm_backward(ctypes.byref(layer_back_args(**none)), None) == OK


def xent_args(**kw):
    a = tcr.tcr_xent_args(x=FAKE, ldx=64, weight=FAKE, ldw=64, target=FAKE, loss=FAKE, lse=FAKE, tokens=4, vocab=9,
                          hidden=64, ignore_index=-100, dtype=tcr.BF16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def xent_back_args(**kw):
    a = tcr.tcr_xent_back_args(dloss=FAKE, inc_dloss=1, x=FAKE, ldx=64, weight=FAKE, ldw=64, target=FAKE, lse=FAKE,
                               dx=FAKE, lddx=64, dweight=FAKE, lddw=64, tokens=4, vocab=9, hidden=64,
                               ignore_index=-100, dtype=tcr.F16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BOTH = [dict(x=None), dict(x=FAKE + 1), dict(weight=None), dict(weight=FAKE + 1), dict(target=None),
        dict(target=FAKE + 4), dict(lse=FAKE + 2), dict(ldx=63), dict(ldw=63), dict(ldw=0), dict(vocab=0),
        dict(hidden=0), dict(dtype=tcr.F32), dict(dtype=tcr.I8), dict(tokens=1 << 23, vocab=1 << 17),
        dict(vocab=1 << 26, hidden=1 << 14, ldw=1 << 14, tokens=1)]


@pytest.mark.parametrize("change", BOTH + [dict(loss=None), dict(loss=FAKE + 1)])
def test_cross_entropy_refuses(lib, change):
    assert lib.tcr_cross_entropy(ctypes.byref(xent_args(**change)), None) == BAD


@pytest.mark.parametrize("change", BOTH + [
    dict(lse=None), dict(dloss=None), dict(dloss=FAKE + 1), dict(inc_dloss=2), dict(dx=FAKE + 1), dict(dweight=FAKE + 1),
    dict(lddx=63), dict(lddw=0)])
def test_cross_entropy_backward_refuses(lib, change):
    assert lib.tcr_cross_entropy_backward(ctypes.byref(xent_back_args(**change)), None) == BAD


@pytest.mark.parametrize("change", [dict(tokens=1 << 24), dict(vocab=1 << 27, hidden=1, ldw=1, ldx=1),
                                    dict(hidden=1 << 20, ldx=1 << 20, ldw=1 << 20)])
def test_cross_entropy_limits(lib, change):
    assert lib.tcr_cross_entropy(ctypes.byref(xent_args(**change)), None) == UNSUPPORTED
    assert lib.tcr_cross_entropy_backward(ctypes.byref(xent_back_args(**change)), None) == UNSUPPORTED


def test_cross_entropy_of_nothing(lib):
    assert lib.tcr_cross_entropy(None, None) == BAD and lib.tcr_cross_entropy_backward(None, None) == BAD
    assert lib.tcr_cross_entropy(ctypes.byref(xent_args(tokens=0, x=None, target=None)), None) == OK
    assert lib.tcr_cross_entropy_backward(ctypes.byref(xent_back_args(tokens=0, dweight=None)), None) == OK
    assert lib.tcr_cross_entropy_backward(ctypes.byref(xent_back_args(dx=None, dweight=None)), None) == OK


def test_calls_leave_the_interpreter_to_other_threads(lib, tmp_path):
    # as for the 8-bit path's calls, with the waiting function behind the five of these
    setup, calls = SLOW_PY.split("class Tensor:")[0], "class Tensor:" + SLOW_PY.split("class Tensor:")[1]
    head, tail = calls.split("for call in (")[0], calls.split("m.gemm(q, q, s, s, c, None)):")[1]
    code = setup + """
try:
    m.dropout(*[None] * 8)
except RuntimeError as e:
    assert "setup_training" in str(e)
m.setup_training("i64", *[slow] * 5)
""" + head + """
t = Tensor("i64", 4)
for call in (lambda: m.dropout(x, 0.1, 1, 2, None, None, x, None),
             lambda: m.layernorm(x, w, w, x, 1e-5, 0.1, 1, 2, None, x, x, None, s, s, None),
             lambda: m.layernorm_backward(x, x, w, s, s, None, 0.0, 0, 0, None, x, None, None, None, None),
             lambda: m.cross_entropy(x, c8, t, -100, s, s, None),
             lambda: m.cross_entropy_backward(s, x, c8, t, s, -100, x, c8, None)):
""".replace("t = Tensor", "c8 = Tensor(\"bf16\", 9, 8)\nt = Tensor") + tail
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    (tmp_path / "slow.c").write_text(SLOW_C)
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "slow.c"), "-o", str(tmp_path / "slow.so")], check=True)
    r = subprocess.run([sys.executable, "-c", code, BIND_PATH, str(tmp_path / "slow.so")], capture_output=True,
                       text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    counts = [int(n) for n in r.stdout.split()]
    assert len(counts) == 5 and min(counts) >= 1, counts


@pytest.mark.parametrize("p", [0.0, 0.1, 0.25, 0.5, 0.9999, 1.0])
def test_share_of_the_generators_bits_that_are_kept(p):
    k = spec.keep(64, 4096, p, 0x0123456789ABCDEF, 1 << 40)
    t = spec.threshold(p)
    assert abs(t / 65536 - p) <= 2.0 ** -17
    share = float(k.double().mean())
    assert abs(share - (1 - t / 65536)) <= 5 * (max(p * (1 - p), 1e-12) / k.numel()) ** 0.5
