"""The cross entropy on logits that no product rounds, against binary64: tokens
that are predicted well, logits of any size.

x holds ones in its first columns and the weight a few numbers of few bits, so
that every logit is a sum of two numbers that binary32 holds exactly.  What is
left are the errors of the loss itself, which are relative ones: with U = 2^-24,
the exponential's own is 2^-22, its argument d = l - m is rounded (U |d|) and
multiplied by a rounded constant (2 U |d|), once in a part of the vocabulary and
once where the parts are joined, where |d| is what both take together; the sums
have fewer than 100 levels, and the logarithm, the exponentials of the join and
the last additions 16 U in all.  Terms below 2^-126 count as 0.
"""
import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests import rows_spec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DTS = {"f16": torch.float16, "bf16": torch.bfloat16}
U = rows_spec.U
# one tile of tokens read where they lie; narrow tiles of a copy; wide tiles
SIZES = [(70, 300), (300, 300), (300, 9000)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)


def exact_case(T, V, dt, base, low=-40.0, high=-2.0, H=64, seed=0):
    """Logits base + (half a whole number in low .. high), 0 at each token's own best
    entry: (x, weight, best, logits in binary64).  Token t has columns 0 and 1 and
    column 2 + t % 50, which its best entry alone has in the weight."""
    gen = torch.Generator().manual_seed(seed + T + V)
    off = torch.randint(int(2 * low), int(2 * high) + 1, (V,), generator=gen) / 2
    x = torch.zeros(T, H)
    x[:, 0] = x[:, 1] = 1
    w = torch.zeros(V, H)
    w[:, 0], w[:, 1] = base, off
    kind = torch.arange(T) % 50
    best = torch.randperm(V, generator=gen)[:50][kind]
    x[torch.arange(T), 2 + kind] = 1
    w[best, 2 + kind] = -off[best]
    logits = base + off.double().repeat(T, 1)
    logits[torch.arange(T), best] = base
    a, b = x.to(DTS[dt]), w.to(DTS[dt])
    assert torch.equal(a.float(), x) and torch.equal(b.float(), w)
    assert torch.equal(a.double() @ b.double().t(), logits)
    return a.cuda(), b.cuda(), best.cuda(), logits.cuda()


def loss64(logits, target):
    """(loss, lse, lse - largest logit) in binary64, without differences of two large numbers."""
    m, top = logits.max(1, keepdim=True)
    log = torch.log1p(torch.exp(logits - m).scatter(1, top, 0.0).sum(1))
    return (m - logits.gather(1, target[:, None]))[:, 0] + log, m[:, 0] + log, log


def relative(logits):
    d = (logits.amax(1) - logits.amin(1)).clamp(max=90)          # further terms are 0
    return 2.0 ** -22 + 2 * 3 * U * d + 116 * U


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("base", [-256.0, -8.0, 0.0, 5.0, 30.0, 120.0, 256.0])
@pytest.mark.parametrize("T,V", SIZES)
def test_losses_of_tokens_predicted_well(T, V, base, dt):
    for low, high in ((-40.0, -2.0), (-20.0, -14.0), (-80.0, -30.0)):
        x, w, best, logits = exact_case(T, V, dt, base, low, high)
        other = torch.where(torch.arange(T, device="cuda") % 3 == 0, (best + 1) % V, best)
        for target in (best, other):
            o = tcr.tcr_cross_entropy(x, w, target, want_lse=True)
            loss, lse, log = loss64(logits, target)
            assert (o.loss >= 0).all()
            q = relative(logits)
            assert ((o.loss.double() - loss).abs() <= q * loss + 2.0 ** -100).all()
            assert ((o.lse.double() - lse).abs() <= q * log + U * lse.abs() + 2.0 ** -100).all()
