"""The layer norm's gradient on rows of more than 8192 columns and more of them
than there are partial sums of the weight's and the bias' gradients, against
the declared operations on the CPU, bit for bit."""
import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests import train_spec as spec
from tests.test_gpu_layer import DROP, of
from tests.test_gpu_norm import DTS, rand, same

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)


def groups(rows, cols, dtype):
    """The partial sums of rows this long: as many blocks of 2048 columns as 152 SMs take in two rounds of three
    (binary32: one of four)."""
    return min(rows, max(1, 152 * (4 if dtype == torch.float32 else 6) // -(-cols // 2048)))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(183, 8193), (400, 8200), (131, 16384), (60, 40001), (5, 1 << 19), (3, (1 << 21) + 5)])
def test_gradient_bits_of_many_long_rows(rows, cols, dt, monkeypatch):
    monkeypatch.setattr(spec, "groups", groups)
    gen = torch.Generator().manual_seed(rows * cols)
    h, dy, dh = rand(gen, rows, cols, DTS[dt]), rand(gen, rows, cols, DTS[dt], 0.3), rand(gen, rows, cols, DTS[dt], 0.1)
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    mean, rstd = h.float().mean(1), 1 / h.float().std(1)
    dx, dr, dw, db = spec.layer_back(dy, h, w, mean, rstd, dh, DROP)
    g = tcr.tcr_layernorm_backward(dy.cuda(), h.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), dh=dh.cuda(), **of(DROP),
                                   want_dresidual=True)
    assert same(g.dx, dx.to(DTS[dt])) and same(g.dresidual, dr.to(DTS[dt]))
    assert same(g.dweight, dw) and same(g.dbias, db)
