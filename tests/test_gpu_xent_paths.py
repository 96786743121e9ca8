"""The cross entropy's paths that no other test takes: a device that could not be
asked at first, pieces of the vocabulary in every form of their rows."""
import os
import subprocess
import sys

import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests import rows_spec
from tests.test_gpu_xent import DTS, U, case, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)


FIRST = """
import os, torch, arithmetic_reduction_tensor_gb300 as tcr
x, w, t = torch.ones(4, 64, device="cuda").half(), torch.ones(9, 64, device="cuda").half(), torch.arange(4, device="cuda")
g = torch.ones(4, device="cuda")
for call in (lambda: tcr.tcr_cross_entropy(x, w, t), lambda: tcr.tcr_cross_entropy_backward(g, x, w, t, g)):
    os.environ["TCR_FAULT_INJECT"] = "query"
    try:
        call()
        raise SystemExit("a call whose device could not be asked went on")
    except tcr.TcrError as e:
        assert e.status == tcr.ERR_CUDA, e
del os.environ["TCR_FAULT_INJECT"]
loss = tcr.tcr_cross_entropy(x, w, t).loss
assert ((loss.double() - torch.tensor(9.0).log().item()).abs() < 1e-5).all()
"""


def test_a_failed_question_is_asked_again():
    # in a process of its own: the answer is kept
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, env={**os.environ, "PYTHONPATH": root},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,V,pitch", [(1030, 264, 300000, 264), (1030, 301, 300000, 307), (2000, 264, 150000, 269),
                                         (1030, 1, 300001, 1)])
def test_pieces_of_the_vocabulary_in_every_form(T, H, V, pitch, dt):
    # P of these does not fit one piece: later pieces add to dX and write their rows of dW,
    # by tensor-map stores or by threads, of a weight read where it lies or copied
    x, w, target, dloss = case(T, H, V, dt, ignored=0.3)
    ws = torch.full((V, pitch), float("nan"), dtype=w.dtype, device="cuda")[:, :H]
    ws.copy_(w)
    o = tcr.tcr_cross_entropy(x, ws, target, want_lse=True)
    wide = torch.full((V + 2, pitch + 3), 7, dtype=w.dtype, device="cuda")
    guarded = wide[1:V + 1, 2:2 + H]
    dx, _ = tcr.tcr_cross_entropy_backward(dloss, x, ws, target, o.lse, dweight=guarded)
    check(x, w, target, dloss, o.loss, o.lse, dx, guarded)
    frame = torch.ones_like(wide, dtype=torch.bool)
    frame[1:V + 1, 2:2 + H] = False
    assert (wide[frame] == 7).all()
    # the same bits where the rows are aligned (to a form that tensor maps take, if H is a multiple of 8)
    dx2, dw2 = tcr.tcr_cross_entropy_backward(dloss, x, w, target, o.lse)
    assert torch.equal(dx, dx2) and torch.equal(guarded, dw2)
    assert tcr.tcr_device_faults() == 0


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,H", [(16384 + 64, 8), (65536, 65), (262144, 64), (1 << 21, 16)])
def test_weight_gradients_of_many_tokens(T, H, dt):
    # logits of 0 over 256 entries, every token's target entry 0: P is 2^-8 of the common
    # dloss, exactly, so dW of the other entries is a sum of T terms of one sign, off
    # by the tensor cores' 2^-22 a step of 16 over 16384 tokens, the additions of
    # such chains (U each) and its rounding
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = (torch.rand(T, H, generator=gen, device="cuda") * 0.5 + 0.5).to(DTS[dt])
    w = torch.zeros(256, H, dtype=x.dtype, device="cuda")
    target = torch.zeros(T, dtype=torch.long, device="cuda")
    lse = tcr.tcr_cross_entropy(x, w, target, want_lse=True).lse
    g = torch.full((1,), 1 / T, device="cuda")
    _, dw = tcr.tcr_cross_entropy_backward(g.expand(T), x, w, target, lse, want_dx=False)
    want = x.double().sum(0) * float(g) / 256
    eps = rows_spec.EPS_OUT[x.dtype]
    # P: the exponential's 2^-22 and lse's rounding U log(256), then exact or one half step of a power of 2
    off = 2.0 ** -22 * -(-min(T, 16384) // 16) + (T // 16384 + 2) * U + 2.0 ** -21 + 8 * U
    assert ((dw[1:].double() - want).abs() <= (off + eps + eps * off) * want + rows_spec.TINY[x.dtype]).all()


def test_input_gradients_of_a_long_piece():
    # the same of dX: 2^19 entries in one piece, one split; the target entry's row is 0
    T, H, V = 512, 5120, 1 << 19
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1.0, generator=gen)
    w[0] = 0
    x = torch.zeros(T, H, dtype=w.dtype, device="cuda")
    target = torch.zeros(T, dtype=torch.long, device="cuda")
    lse = tcr.tcr_cross_entropy(x, w, target, want_lse=True).lse
    one = torch.ones(1, device="cuda")
    dx, _ = tcr.tcr_cross_entropy_backward(one.expand(T), x, w, target, lse, want_dweight=False)
    want = sum(b.double().sum(0) for b in w.split(1 << 15)) / V
    off = 2.0 ** -22 * 1024 + (V // 16384 + 2) * U + 2.0 ** -21 + 16 * U
    eps = rows_spec.EPS_OUT[w.dtype]
    assert ((dx.double() - want).abs() <= (off + eps + eps * off) * want).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("live", [0, 1, 70, 17000])
def test_few_of_many_tokens_count(live, dt):
    # the launch is the one for long sums, the sums are not: the same bits as without the ignored
    T, H, V = 40000, 72, 700
    x, w, target, dloss = case(T, H, V, dt, ignored=0.0)
    keep = torch.zeros(T, dtype=torch.bool, device="cuda")
    keep[torch.randperm(T, device="cuda")[:live]] = True
    target[~keep], x[~keep] = -100, float("nan")
    o = tcr.tcr_cross_entropy(x, w, target, want_lse=True)
    dx, dw = tcr.tcr_cross_entropy_backward(dloss, x, w, target, o.lse)
    assert (dx[~keep] == 0).all() and (o.loss[~keep] == 0).all()
    if live == 0:
        assert (dw == 0).all()
        return
    few = tcr.tcr_cross_entropy(x[keep], w, target[keep], want_lse=True)
    dx1, dw1 = tcr.tcr_cross_entropy_backward(dloss[keep], x[keep], w, target[keep], few.lse)
    assert torch.equal(o.loss[keep], few.loss) and torch.equal(dw, dw1)
    check(x[keep], w, target[keep], dloss[keep], few.loss, few.lse, dx1, dw1)
    check(x[keep], w, target[keep], dloss[keep], None, None, dx[keep], None)
