"""The softmax cross entropy over a vocabulary and its gradient, against
binary64.

With L the declared bound of a logit (2^-22 ceil(H / 16) times the largest sum of
magnitudes of a token's logits) and U = 2^-24: lse is off by at most L + 2^-20 (the
exponentials' and logarithm's own errors and the sum of at most 2^17 terms in
order-independent trees of 32 + V / 256 / 16 + 16 levels) + 4 U |lse|, the loss by
that + L + U |loss|.  p is off relatively by q = 2 L + 2^-19 + 8 U |lse|, P by
(p q + U) |g|, by its rounding (half a step of the type, and half its smallest
subnormal in units of the largest |g|, 2^15 below for binary16), the
products' sums by 2^-22 ceil(K / 16) of their magnitudes (+ U a piece), and
their results by the output's rounding.
"""
import threading

import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests import rows_spec, train_spec as spec
from tests.test_gpu_norm import same, strided

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DTS = {"f16": torch.float16, "bf16": torch.bfloat16}
U = rows_spec.U


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)


def case(T, H, V, dt, ignored=0.2, seed=0, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + T + 7 * H + 13 * V)
    x = torch.randn(T, H, generator=gen, device="cuda").to(DTS[dt])
    w = (torch.randn(V, H, generator=gen, device="cuda") * spread / H ** 0.5).to(DTS[dt])
    target = (V * torch.rand(T, generator=gen, device="cuda") ** 2).long().clamp_(0, V - 1)
    target[torch.rand(T, generator=gen, device="cuda") < ignored] = -100
    dloss = torch.randn(T, generator=gen, device="cuda")
    return x, w, target, dloss


def check(x, w, target, dloss, loss, lse, dx, dw, ignore=-100, inf_ok=False):
    """Every output within its bound (None: not looked at)."""
    H, V = w.shape[1], w.shape[0]
    eps, tiny = rows_spec.EPS_OUT[x.dtype], rows_spec.TINY[x.dtype]
    l64, s64, dx64, dw64, (size, p, hit, g, P, xd, wd, row) = spec.xent64(x, w, target, ignore, dloss)
    L = 2.0 ** -22 * -(-H // 16) * size + 1e-30
    off = L + 2.0 ** -20 + 4 * U * row.abs()
    live = target != ignore
    if loss is not None:
        assert ((loss.double() - l64).abs() <= off + L + U * l64.abs()).all()
        assert (loss[~live] == 0).all()
    if lse is not None:
        assert ((lse.double() - s64).abs() <= off).all()
    q = (2 * L + 2.0 ** -19 + 8 * U * row.abs())[:, None]
    top = g.abs().max()
    low = top * (2.0 ** -25 * 2.0 ** -15 if x.dtype == torch.float16 else 2.0 ** -134)
    eP = (p * q + U * (p + hit)) * g.abs()
    eP = eP + eps * (P.abs() + eP) + torch.where(g == 0, 0.0, low)
    pieces = 2
    for got, want, a, e, b, K in ((dx, dx64, P, eP, wd, V), (dw, dw64, P.t(), eP.t(), xd, len(x))):
        if got is None:
            continue
        mag = a.abs() @ b.abs()
        err = e @ b.abs() + (2.0 ** -22 * -(-K // 16) + (pieces + 34) * U) * mag
        assert ((got.double() - want).abs() <= err + eps * (want.abs() + err) + tiny).all()
    if dx is not None:
        assert (dx[~live] == 0).all()


def step(x, w, target, dloss, **kw):
    o = tcr.tcr_cross_entropy(x, w, target, want_lse=True, **kw)
    dx, dw = tcr.tcr_cross_entropy_backward(dloss, x, w, target, o.lse, **kw)
    return o.loss, o.lse, dx, dw


SIZES = [(1, 64, 256), (1, 1, 1), (2, 8, 2), (3, 64, 255), (5, 65, 257), (64, 128, 1000), (127, 200, 513),
         (128, 64, 300), (129, 512, 5003), (256, 256, 256), (257, 1001, 771), (300, 72, 4099), (700, 320, 2560),
         (1030, 136, 1300), (31, 2049, 640), (2, 4096, 20000), (513, 7, 9000),
         # on both sides of where tiles become narrow, and ends of narrow ones
         (64, 64, 4864), (64, 72, 4865), (200, 128, 4700), (300, 64, 2400), (300, 64, 2500), (70, 1032, 63), (70, 136, 65)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,H,V", SIZES)
def test_against_binary64(T, H, V, dt):
    a = case(T, H, V, dt)
    check(*a, *step(*a))
    assert tcr.tcr_device_faults() == 0


@pytest.mark.parametrize("dt", DTS)
def test_peaked_logits_and_gradients_of_many_sizes(dt):
    x, w, target, dloss = case(333, 256, 2000, dt, spread=12.0)
    dloss *= torch.exp2(torch.randint(-20, 10, dloss.shape, device="cuda").float())
    check(x, w, target, dloss, *step(x, w, target, dloss))
    # logits far below and above 0
    x[:, 0] = 40.0
    w[:, 0] = 3.0
    check(x, w, target, dloss, *step(x, w, target, dloss))
    w[:, 0] = -3.0
    check(x, w, target, dloss, *step(x, w, target, dloss))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,H,V", [(5, 65, 257), (200, 200, 600), (300, 1001, 1003), (64, 64, 512)])
def test_strides_and_alignment_do_not_change_bits(T, H, V, dt):
    x, w, target, dloss = case(T, H, V, dt)
    want = step(x, w, target, dloss)
    for pitch, off in ((H + 8 - H % 8, 8), (H + 3, 1), (H + 2, 2)):
        xs, ws = strided(x, pitch, off), strided(w, pitch, off)
        gx = torch.full((T, pitch + off), 7, dtype=x.dtype, device="cuda")
        gw = torch.full((V, pitch + off), 7, dtype=x.dtype, device="cuda")
        o = tcr.tcr_cross_entropy(xs, ws, target, want_lse=True)
        tcr.tcr_cross_entropy_backward(dloss, xs, ws, target, o.lse, dx=gx[:, off:off + H], dweight=gw[:, off:off + H])
        got = (o.loss, o.lse, gx[:, off:off + H], gw[:, off:off + H])
        assert all(same(a, b) for a, b in zip(want, got))
        for g in (gx, gw):
            assert (g[:, :off] == 7).all() and (g[:, off + H:] == 7).all()
    # what lies between the rows is not looked at
    for pitch in (H + 8 - H % 8, H + 24 - H % 8, H + 3):
        xn = torch.full((T, pitch), float("nan"), dtype=x.dtype, device="cuda")
        wn = torch.full((V, pitch), float("nan"), dtype=x.dtype, device="cuda")
        xn[:, :H], wn[:, :H] = x, w
        assert all(same(a, b) for a, b in zip(want, step(xn[:, :H], wn[:, :H], target, dloss)))
    # few tokens, more than a tile of them and unaligned ones: the same bits of each
    if T > 64:
        few = tcr.tcr_cross_entropy(x[:64], w, target[:64], want_lse=True)
        assert same(few.loss, want[0][:64]) and same(few.lse, want[1][:64])
    # one row of x for all; the gradient of a mean; dx over x
    xe = x[:1].expand(T, H)
    assert same(tcr.tcr_cross_entropy(xe, w, target).loss, tcr.tcr_cross_entropy(xe.contiguous(), w, target).loss)
    one = torch.full((1,), 1 / 7, device="cuda").expand(T)
    a = tcr.tcr_cross_entropy_backward(one, x, w, target, want[1])
    b = tcr.tcr_cross_entropy_backward(one.contiguous(), x, w, target, want[1])
    assert all(same(p, q) for p, q in zip(a, b))
    xc = x.clone()
    dx, _ = tcr.tcr_cross_entropy_backward(dloss, xc, w, target, want[1], dx=xc)
    assert same(dx, want[2])


@pytest.mark.parametrize("T", [200, 256, 257, 700])
def test_ignored_tokens_count_for_nothing_whatever_they_hold(T):
    x, w, target, dloss = case(T, 136, 1300, "bf16", ignored=0.4)
    want = step(x, w, target, dloss)
    live = target != -100
    assert 0 < int(live.sum()) < T
    xn, dn = x.clone(), dloss.clone()
    xn[~live] = float("nan")
    dn[~live] = float("inf")
    assert all(same(a, b) for a, b in zip(want, step(xn, w, target, dn)))
    # the tokens that count alone give the same bits
    o = step(x[live], w, target[live], dloss[live])
    assert same(want[0][live], o[0]) and same(want[2][live], o[2]) and same(want[3], o[3])
    # another index that is ignored, one inside the vocabulary
    t = torch.where(live, target, 5)
    hit5 = t == 5
    got = step(x, w, t, dloss, ignore_index=5)
    assert (got[0][hit5] == 0).all() and same(got[0][~hit5], want[0][~hit5])


@pytest.mark.parametrize("T", [1, 64, 700])
def test_no_token_counts(T):
    x, w, target, dloss = case(T, 72, 300, "f16")
    target[:] = -100
    x[:] = float("nan")
    loss, lse, dx, dw = step(x, w, target, dloss)
    assert (loss == 0).all() and (lse == 0).all() and (dx == 0).all() and (dw == 0).all()


def test_bad_targets_and_bad_values_are_loud_and_stay_in_their_rows():
    x, w, target, dloss = case(300, 64, 500, "bf16", ignored=0.0)
    want = step(x, w, target, dloss)
    for bad in (500, -1, 1 << 40, -(1 << 40)):
        t = target.clone()
        t[17] = bad
        loss, lse, dx, dw = step(x, w, t, dloss)
        rest = torch.arange(300, device="cuda") != 17
        assert loss[17].isnan() and same(loss[rest], want[0][rest]) and same(lse, want[1])
        assert dx[17].isnan().all() and same(dx[rest], want[2][rest]) and dw.isnan().all()
    xn = x.clone()
    xn[200, 3] = float("nan")
    loss, lse, dx, _ = step(xn, w, target, dloss)
    rest = torch.arange(300, device="cuda") != 200
    assert loss[200].isnan() and lse[200].isnan() and dx[200].isnan().all()
    assert same(loss[rest], want[0][rest]) and same(dx[rest], want[2][rest])
    for g in (float("nan"), float("inf")):
        d = dloss.clone()
        d[9] = g
        _, _, dx, _ = step(x, w, target, d)
        rest = torch.arange(300, device="cuda") != 9
        assert not dx[9].isfinite().any() and same(dx[rest], want[2][rest])
    # no gradient arrives: zeros
    assert all((t == 0).all() for t in step(x, w, target, torch.zeros_like(dloss))[2:])
    # an entry of the vocabulary at minus infinity
    wi, xi = w.clone(), x.clone()
    wi[7] = 0
    wi[7, 0] = float("-inf")
    xi[:, 0] = 1.0
    target[target == 7] = 8
    loss, lse, *_ = step(xi, wi, target, dloss)
    wf = wi.clone()
    wf[7, 0] = -1e30
    assert loss.isfinite().all() and same(loss, step(xi, wf, target, dloss)[0])


def test_pieces_of_the_vocabulary():
    # P of 1030 tokens over 300000 entries does not fit one piece
    x, w, target, dloss = case(1030, 64, 300000, "bf16")
    check(x, w, target, dloss, *step(x, w, target, dloss))
    # one product's share of both gradients, with and without the other
    o = tcr.tcr_cross_entropy(x, w, target, want_lse=True)
    both = tcr.tcr_cross_entropy_backward(dloss, x, w, target, o.lse)
    dx, none = tcr.tcr_cross_entropy_backward(dloss, x, w, target, o.lse, want_dweight=False)
    assert none is None and same(dx, both[0])
    none, dw = tcr.tcr_cross_entropy_backward(dloss, x, w, target, o.lse, want_dx=False)
    assert none is None and same(dw, both[1])


def test_many_tokens():
    # more tokens than one CTA's share of the compaction holds
    x, w, target, dloss = case(300000, 8, 300, "f16", ignored=0.5)
    o = tcr.tcr_cross_entropy(x, w, target, want_lse=True)
    dx, dw = tcr.tcr_cross_entropy_backward(dloss, x, w, target, o.lse)
    check(x, w, target, dloss, o.loss, o.lse, dx, dw)


def test_gradient_against_differences():
    # central differences of the binary64 loss along random directions
    x, w, target, dloss = case(90, 40, 700, "bf16")
    _, _, dx, dw = step(x, w, target, dloss)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(x, w):
        return (spec.xent64(x, w, target, -100, dloss)[0] * dloss.double()).sum()

    for k, got in enumerate((dx, dw)):
        a = [x.double(), w.double()]
        v = torch.randn(a[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = list(a), list(a)
        up[k], down[k] = a[k] + h * v, a[k] - h * v
        diff = float((loss(*up) - loss(*down)) / (2 * h))
        # P and the result are each off by half a step of bfloat16
        assert abs(float((got.double() * v).sum()) - diff) <= 3 * 2.0 ** -8 * float((got.double() * v).abs().sum()) + 1e-6


def test_nothing_and_refusals():
    x, w, target, dloss = case(8, 64, 300, "bf16")
    e = x[:0]
    assert tcr.tcr_cross_entropy(e, w, target[:0]).loss.shape == (0,)
    dx, dw = tcr.tcr_cross_entropy_backward(dloss[:0], e, w, target[:0], dloss[:0])
    assert dx.shape == (0, 64) and (dw == 0).all()
    lse = tcr.tcr_cross_entropy(x, w, target, want_lse=True).lse
    back = lambda *a, **k: (lambda: tcr.tcr_cross_entropy_backward(*a, **k))      # noqa: E731
    bad = [
        (TypeError, lambda: tcr.tcr_cross_entropy(x.float(), w.float(), target)),
        (TypeError, lambda: tcr.tcr_cross_entropy(x, w.half(), target)),
        (TypeError, lambda: tcr.tcr_cross_entropy(x, w, target.int())),
        (ValueError, lambda: tcr.tcr_cross_entropy(x, w, target[:7])),
        (ValueError, lambda: tcr.tcr_cross_entropy(x, w[:, :63], target)),
        (ValueError, lambda: tcr.tcr_cross_entropy(x, w.cpu(), target)),
        (ValueError, lambda: tcr.tcr_cross_entropy(x, w[:1].expand(300, 64), target)),
        (ValueError, lambda: tcr.tcr_cross_entropy(x, w, target.cpu())),
        (ValueError, lambda: tcr.tcr_cross_entropy(x[0], w, target)),
        (tcr.TcrError, lambda: tcr.tcr_cross_entropy(x, w[:0], target)),
        (tcr.TcrError, lambda: tcr.tcr_cross_entropy(x[:, :0], w[:, :0], target)),
        (ValueError, back(dloss[:7], x, w, target, lse)), (TypeError, back(dloss.double(), x, w, target, lse)),
        (ValueError, back(dloss.repeat(2)[::2], x, w, target, lse)), (ValueError, back(dloss, x, w, target, lse[:7])),
        (ValueError, back(dloss, x, w, target, lse, dx=x[:7])), (TypeError, back(dloss, x, w, target, lse, dx=x.float())),
        (TypeError, back(dloss, x, w, target, lse, dweight=w.float())),
        (ValueError, back(dloss, x, w, target, lse, dweight=w.t())),
        (ValueError, back(dloss.cpu(), x, w, target, lse)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_failed_calls_leave_outputs_alone(monkeypatch):
    x, w, target, dloss = case(8, 64, 300, "bf16")
    out, dx, dw = torch.full((8,), 5.0, device="cuda"), torch.full_like(x, 5), torch.full_like(w, 5)
    for what in ("launch", "alloc"):
        monkeypatch.setenv("TCR_FAULT_INJECT", what)
        with pytest.raises(tcr.TcrError):
            tcr.tcr_cross_entropy(x, w, target, loss=out)
        with pytest.raises(tcr.TcrError):
            tcr.tcr_cross_entropy_backward(dloss, x, w, target, out, dx=dx, dweight=dw)
    monkeypatch.delenv("TCR_FAULT_INJECT")
    assert (out == 5).all() and (dx == 5).all() and (dw == 5).all()


def test_wait_limit_reports_nan_and_fault_word_then_recovers(monkeypatch):
    a = case(700, 320, 2560, "bf16")
    want = step(*a)
    torch.cuda.synchronize()
    tcr.tcr_device_faults(clear=True)
    monkeypatch.setenv("TCR_FAULT_INJECT", "stall")
    loss = tcr.tcr_cross_entropy(*a[:3]).loss
    torch.cuda.synchronize()
    assert loss.isnan().any() and tcr.tcr_device_faults(clear=True) & tcr.FAULT_PIPELINE_WAIT
    dx, dw = tcr.tcr_cross_entropy_backward(a[3], *a[:3], want[1])
    torch.cuda.synchronize()
    monkeypatch.delenv("TCR_FAULT_INJECT")
    assert dx.isnan().any() and dw.isnan().any() and tcr.tcr_device_faults(clear=True) & tcr.FAULT_PIPELINE_WAIT
    assert all(same(p, q) for p, q in zip(want, step(*a)))
    assert tcr.tcr_device_faults() == 0


def test_streams_graphs_and_threads():
    a, b = case(300, 200, 1000, "bf16"), case(129, 512, 3001, "f16")
    wa, wb = step(*a), step(*b)
    assert all(same(p, q) for p, q in zip(wa, step(*a)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(*a, stream=s)
    s.synchronize()
    assert all(same(p, q) for p, q in zip(wa, got))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        oa = step(*a)
    with torch.cuda.graph(g2):
        ob = step(*b)
    for _ in range(3):
        for t in (*oa, *ob):
            t.zero_()
        g1.replay()
        g2.replay()
        assert all(same(p, q) for p, q in zip(wa, oa)) and all(same(p, q) for p, q in zip(wb, ob))
    # replayed on other tokens, of another number
    a[0].copy_(a[0].flip(0))
    a[2][:150] = -100
    g1.replay()
    assert all(same(p, q) for p, q in zip(step(*a), oa))
    wa = step(*a)
    wrong = []

    def work(c, want):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(6):
                got = step(*c)
                st.synchronize()
                if not all(same(p, q) for p, q in zip(want, got)):
                    wrong.append(1)

    ts = [threading.Thread(target=work, args=c) for c in ((a, wa), (b, wb), (a, wa), (b, wb))]
    torch.cuda.synchronize()
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong


def test_a_training_step_of_the_operators_together():
    # x -> dropout, residual, layer norm -> loss, and back, against autograd in binary64
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, H, V, dt = 260, 192, 900, torch.bfloat16
    x, r = (torch.randn(T, H, generator=gen, device="cuda").to(dt) for _ in range(2))
    w = (torch.rand(H, generator=gen, device="cuda") + 0.5).to(dt)
    b = (torch.randn(H, generator=gen, device="cuda") * 0.1).to(dt)
    head = (torch.randn(V, H, generator=gen, device="cuda") / H ** 0.5).to(dt)
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    target[::7] = -100
    drop = dict(p=0.1, seed=11, offset=5)
    n = int((target != -100).sum())
    o = tcr.tcr_layernorm(x, w, b, residual=r, **drop, want_stats=True)
    l = tcr.tcr_cross_entropy(o.y, head, target, want_lse=True)
    dy, dhead = tcr.tcr_cross_entropy_backward(torch.full((1,), 1 / n, device="cuda").expand(T), o.y, head, target, l.lse)
    g = tcr.tcr_layernorm_backward(dy, o.h, w, o.mean, o.rstd, **drop, want_dresidual=True)
    leaves = [t.double().requires_grad_() for t in (x, r, w, b, head)]
    k = spec.keep(T, H, 0.1, 11, 5).cuda()
    h = leaves[1] + torch.where(k, leaves[0] * spec.factor(0.1), 0.0)
    var, mean = torch.var_mean(h, 1, unbiased=False, keepdim=True)
    y = (h - mean) / torch.sqrt(var + 1e-5) * leaves[2] + leaves[3]
    loss = torch.nn.functional.cross_entropy(y @ leaves[4].t(), target, ignore_index=-100)
    loss.backward()
    # five roundings to bfloat16 on the way (h, y, P, dy, the result), half a step of 2^-8 each, in
    # the norm of a gradient; the loss: y's rounding, averaged
    assert abs(float(l.loss.sum()) / n - float(loss.detach())) <= 2.0 ** -8 * 2
    for got, leaf in zip((g.dx, g.dresidual, g.dweight, g.dbias, dhead), leaves):
        err = (got.double() - leaf.grad).norm() / leaf.grad.norm()
        assert err <= 5 * 2.0 ** -8, float(err)
