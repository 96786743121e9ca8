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


def probabilities(x, w, target, dloss, lse):
    """P read back through dx: entry v alone has column H + v of the weight, x 0 there."""
    (T, H), V = x.shape, len(w)
    xp, wp = x.new_zeros(T, H + V), w.new_zeros(V, H + V)
    xp[:, :H], wp[:, :H] = x, w
    wp[:, H:] = torch.eye(V, dtype=w.dtype, device=w.device)
    o = tcr.tcr_cross_entropy(xp, wp, target, want_lse=True)
    assert torch.equal(o.lse, lse)
    return tcr.tcr_cross_entropy_backward(dloss, xp, wp, target, lse, want_dweight=False)[0][:, H:]


def check_probabilities(P, logits, target, dloss, dt):
    """P against binary64: p = exp(d) is off by the exponential's share of `relative`
    and by lse's own error, a rounding of U |lse| and that of its logarithm; then
    (p - [target]) g and its rounding, in units of the largest |g| (2^15 smaller in
    binary16), and dx's.  Every product but one of dx's sum is 0."""
    _, lse, log = loss64(logits, target)
    d = (logits - lse[:, None]).abs().clamp(max=90)
    p = torch.exp(logits - lse[:, None])
    hit = torch.zeros_like(p).scatter_(1, target[:, None], 1.0)
    g = dloss.double()[:, None]
    q = 2.0 ** -22 + 3 * U * d + ((U * lse.abs()) + relative(logits) * log)[:, None] + 4 * U
    err = (p * q + 2 * U * (p + hit)) * g.abs()
    want = (p - hit) * g
    eps, tiny = rows_spec.EPS_OUT[DTS[dt]], rows_spec.TINY[DTS[dt]]
    low = float(g.abs().max()) * (2.0 ** -25 * 2.0 ** -15 if dt == "f16" else 2.0 ** -126)
    err = err + eps * (want.abs() + err) + low
    assert ((P.double() - want).abs() <= err + eps * (want.abs() + err) + tiny).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("base", [-256.0, 0.0, 30.0, 256.0])
@pytest.mark.parametrize("T,V", [(70, 300), (300, 300), (5000, 600)])
def test_gradients_of_tokens_predicted_well(T, V, base, dt):
    for low, high in ((-40.0, -2.0), (-12.0, -6.0)):
        x, w, best, logits = exact_case(T, V, dt, base, low, high)
        target = torch.where(torch.arange(T, device="cuda") % 3 == 0, (best + 1) % V, best)
        lse = tcr.tcr_cross_entropy(x, w, target, want_lse=True).lse
        dloss = torch.full((T,), 0.125, device="cuda")
        dloss[::7] = -0.01
        check_probabilities(probabilities(x, w, target, dloss, lse), logits, target, dloss, dt)


@pytest.mark.parametrize("T,V", SIZES)
def test_logits_at_the_ends_of_the_types(T, V):
    # entries that are masked by the type's lowest value, some of them whole parts of the
    # vocabulary, in one column of the weight; the largest value in turn
    for dt, last in (("bf16", 3.3895313892515355e38), ("f16", 65504.0)):
        x, w, best, logits = exact_case(T, V, dt, 5.0, -9.0, -1.0)
        masked = torch.arange(V, device="cuda") % 3 == 1
        masked[:256] = True
        masked[best] = False
        w[masked], w[masked, 0] = 0, -last
        logits[:, masked] = -last
        loss, lse, log = loss64(logits, best)
        o = tcr.tcr_cross_entropy(x, w, best, want_lse=True)
        q = 2.0 ** -22 + 2 * 3 * U * 9 + 116 * U         # the others' differences are 9 or less
        assert ((o.loss.double() - loss).abs() <= q * loss).all()
        assert ((o.lse.double() - lse).abs() <= q * log + U * lse.abs()).all()
        if V <= 600:
            dloss = torch.full((T,), 1.0, device="cuda")
            check_probabilities(probabilities(x, w, best, dloss, o.lse), logits, best, dloss, dt)
        # a target that is masked: as far off as the type goes
        hidden = torch.full_like(best, int(masked.nonzero()[0, 0]))
        o = tcr.tcr_cross_entropy(x, w, hidden)
        assert ((o.loss.double() - loss64(logits, hidden)[0]).abs() <= 2 * U * last).all()
        # every logit at an end: the loss is that of equal ones
        for end in (last, -last):
            w[:], w[:, 0] = 0, end
            o = tcr.tcr_cross_entropy(x, w, best, want_lse=True)
            flat = torch.tensor(float(V), dtype=torch.float64).log()
            assert ((o.loss.double() - flat).abs() <= (2.0 ** -22 + 116 * U) * flat).all()
            assert ((o.lse.double() - (end + flat)).abs() <= U * last + 1e-5).all()
            if V <= 600:
                assert probabilities(x, w, best, torch.ones(T, device="cuda"), o.lse).isfinite().all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,H,V", [(64, 1096, 512), (64, 4096, 512), (1100, 4096, 1100), (300, 8200, 700)])
def test_both_passes_see_the_same_logits(T, H, V, dt):
    # positive products, whose sums lose their last bits all one way: a token's row of P
    # adds up to 0 all the same, but for what the exponentials, lse's rounding and P's
    # own roundings leave.  A column of ones in the weight, 0 in x, adds it up.
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randn(T, H + 8, generator=gen, device="cuda").abs()
    w = torch.randn(V, H + 8, generator=gen, device="cuda").abs() * (47.0 / H)
    target = torch.randperm(V, generator=gen, device="cuda")[torch.arange(T, device="cuda") % V]
    x[:, H:] = 0
    x = x.to(DTS[dt])
    few = min(T, V)
    w[target[:few]] += x[:few].float() * (30.0 / (x[:few].float() ** 2).sum(1, keepdim=True))
    w[:, H:] = 1
    w = w.to(DTS[dt])
    logits = x.double() @ w.double().t()
    loss, lse, log = loss64(logits, target)
    assert float(loss.median()) < 0.05 and float(lse.min()) > 20
    p = torch.exp(logits - lse[:, None])
    size = 2 * p.scatter(1, target[:, None], 0.0).sum(1)                 # sum of |P|
    d = (logits - lse[:, None]).abs()
    off = 2.0 ** -22 + 3 * U * (p * d).sum(1) + U * lse + relative(logits) * log + 4 * U
    eps = rows_spec.EPS_OUT[DTS[dt]]
    got = tcr.tcr_cross_entropy(x, w, target, want_lse=True)
    dx, _ = tcr.tcr_cross_entropy_backward(torch.ones(T, device="cuda"), x, w, target, got.lse, want_dweight=False)
    # (the logits' own errors, which `size` is taken without: a thousandth)
    bound = (1.001 * size * (eps + 2.0 ** -22 * -(-V // 16)) + 2 * off) * (1 + 2 * eps) + 2.0 ** -30
    assert (dx[:, H].double().abs() <= bound).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,V", [(300, 2500), (700, 2000), (520, 1985), (600, 1700), (300, 9000)])
def test_bits_of_a_token_do_not_depend_on_the_others(T, V, dt):
    # on both sides of where tiles of the vocabulary become narrow
    gen = torch.Generator(device="cuda").manual_seed(T + V)
    x = torch.randn(T, 72, generator=gen, device="cuda").to(DTS[dt])
    w = (torch.randn(V, 72, generator=gen, device="cuda") / 3).to(DTS[dt])
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    all_of = tcr.tcr_cross_entropy(x, w, target, want_lse=True)
    for n in (1, 64, 257, T // 2):
        few = tcr.tcr_cross_entropy(x[:n], w, target[:n], want_lse=True)
        assert torch.equal(few.loss, all_of.loss[:n]) and torch.equal(few.lse, all_of.lse[:n])
    # ignored tokens: the same numbers without them, dweight's too
    target[torch.rand(T, generator=gen, device="cuda") < 0.4] = -100
    live = target != -100
    dloss = torch.randn(T, generator=gen, device="cuda")
    dloss[~live] = 0
    a = tcr.tcr_cross_entropy(x, w, target, want_lse=True)
    b = tcr.tcr_cross_entropy(x[live], w, target[live], want_lse=True)
    assert torch.equal(a.loss[live], b.loss) and torch.equal(a.lse[live], b.lse)
    assert torch.equal(b.loss, all_of.loss[live])
    dw = [tcr.tcr_cross_entropy_backward(d, xx, w, t, o.lse, want_dx=False)[1]
          for d, xx, t, o in ((dloss, x, target, a), (dloss[live], x[live], target[live], b))]
    assert torch.equal(*dw)
