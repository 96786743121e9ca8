"""The cross entropy's paths that no other test takes: a device that could not be
asked at first, pieces of the vocabulary in every form of their rows."""
import os
import subprocess
import sys

import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests.test_gpu_xent import case, check

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
