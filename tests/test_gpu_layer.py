"""Dropout, the layer norm with it and the layer norm's gradient.

Two references: the declared binary32 operations restated on the CPU
(tests/train_spec.py), which results match bit for bit, and the definitions in
binary64.  There, with U = 2^-24 and d tree levels over a row: the mean is off
by at most e = (d + 1) U mean|h| + U |mean|, so h - mean by e + U |h - mean|; the
variance, a sum of squares, relatively by (d + 3) U + (e rstd)^2 + 2 e rstd U, rstd
by half that + 2 U; then four roundings and the output's own.
"""
import threading

import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests import rows_spec, train_spec as spec
from tests.test_gpu_norm import DTS, rand, same, strided

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = rows_spec.U
DROP = (0.3, 0x1234567890ABCDEF, (7 << 32) + 3)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)


def of(drop):
    return {} if drop is None else dict(zip(("p", "seed", "offset"), drop))


COLS = [1, 2, 7, 8, 9, 31, 100, 255, 256, 257, 500, 512, 513, 1001, 1024, 1025, 1400, 2048, 2049, 2999, 4096, 4099,
        5120, 5121, 6000, 7168, 7170, 8192, 8200, 12000, 16384, 16391, 32769, 40000]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999, 1.0])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (9, 255), (33, 257), (7, 1000), (4, 2049), (2, 20001)])
def test_dropout_bits(rows, cols, p, dt):
    gen = torch.Generator().manual_seed(cols)
    x, r = rand(gen, rows, cols, DTS[dt]), rand(gen, rows, cols, DTS[dt])
    drop = (p,) + DROP[1:]
    want = spec.dropped(x.float(), drop)
    assert same(tcr.tcr_dropout(x.cuda(), **of(drop)), want.to(DTS[dt]))
    both = (r.float() + want).to(DTS[dt])
    assert same(tcr.tcr_dropout(x.cuda(), **of(drop), residual=r.cuda()), both)
    # rows of any alignment, in place, and a row for all
    for pitch, off in ((cols + 3, 1), (cols + 8, 8)):
        guard = torch.full((rows, pitch + off), 7, dtype=DTS[dt], device="cuda")
        tcr.tcr_dropout(strided(x, pitch, off), **of(drop), residual=strided(r, pitch, off),
                        out=guard[:, off:off + cols])
        assert same(guard[:, off:off + cols], both)
        assert (guard[:, :off] == 7).all() and (guard[:, off + cols:] == 7).all()
    xc, rc = x.cuda(), r.cuda()
    assert same(tcr.tcr_dropout(xc, **of(drop), residual=rc, out=rc), both)
    assert same(tcr.tcr_dropout(xc, **of(drop), out=xc), want.to(DTS[dt]))
    one = spec.dropped(x[:1].float().expand(rows, cols), drop).to(DTS[dt])
    assert same(tcr.tcr_dropout(x[:1].cuda().expand(rows, cols), **of(drop)), one)


def test_dropout_masks_infinities_and_counts():
    x = torch.full((512, 4096), float("inf"), device="cuda")
    x[:, ::2] = float("nan")
    k = spec.keep(512, 4096, *DROP).cuda()
    y = tcr.tcr_dropout(x, **of(DROP))
    assert (y[~k] == 0).all() and (y[k].isnan() | y[k].isinf()).all()
    # 2^21 draws: 5 standard deviations of the share kept
    share = k.double().mean().item()
    assert abs(share - 0.7) < 5 * (0.21 / k.numel()) ** 0.5
    # of another seed, offset or row: other masks, as far apart as independent ones
    for other in ((0.3, DROP[1] + 1, DROP[2]), (0.3, DROP[1], DROP[2] + 1), (0.3, DROP[1], DROP[2] + (1 << 32))):
        both = (k & (tcr.tcr_dropout(torch.ones_like(x), **of(other)) > 0)).double().mean().item()
        assert abs(both - 0.49) < 5 * (0.25 / k.numel()) ** 0.5


def test_dropout_of_many_rows_and_wide_ones():
    # the last rows of a call against the rows alone would draw another mask:
    # their counter is the row
    for rows, cols in ((300000, 9), (70000, 257), (3, 1 << 20)):
        x = torch.ones(rows, cols, dtype=torch.float16, device="cuda")
        y = tcr.tcr_dropout(x, **of(DROP))
        first = rows - min(rows, 64)
        k = spec.keep(rows - first, cols, *DROP, first=first)
        assert torch.equal((y[first:] > 0).cpu(), k)


def test_state_replaces_seed_and_offset():
    x = torch.randn(37, 1000, device="cuda")
    state = torch.tensor([DROP[1], DROP[2]], dtype=torch.int64, device="cuda")
    want = tcr.tcr_dropout(x, **of(DROP))
    assert same(tcr.tcr_dropout(x, p=DROP[0], seed=5, offset=6, state=state), want)
    w = torch.ones(1000, device="cuda")
    a = tcr.tcr_layernorm(x, w, **of(DROP), want_stats=True)
    b = tcr.tcr_layernorm(x, w, p=DROP[0], state=state, want_stats=True)
    assert same(a.y, b.y) and same(a.h, b.h)
    ga = tcr.tcr_layernorm_backward(x, a.h, w, a.mean, a.rstd, **of(DROP))
    gb = tcr.tcr_layernorm_backward(x, a.h, w, a.mean, a.rstd, p=DROP[0], state=state)
    assert same(ga.dx, gb.dx)
    # a captured graph draws the mask that the state says at its replay
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = tcr.tcr_dropout(x, p=DROP[0], state=state)
    for offset in (DROP[2], 11, 12):
        state[1] = offset
        g.replay()
        assert same(y, tcr.tcr_dropout(x, p=DROP[0], seed=DROP[1], offset=offset))
    # negative and large numbers count modulo 2^64
    assert same(tcr.tcr_dropout(x, p=0.3, seed=-1, offset=-2),
                tcr.tcr_dropout(x, p=0.3, seed=(1 << 64) - 1, offset=(1 << 64) - 2))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("cols", COLS)
def test_layer_bits(cols, dt):
    gen = torch.Generator().manual_seed(cols)
    rows = 5
    x, r = rand(gen, rows, cols, DTS[dt]), rand(gen, rows, cols, DTS[dt], 2.0)
    x[2], r[2] = 0, 0                                   # an empty token
    x[3], r[3] = 3, 0                                   # one without variance
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    b = torch.randn(cols, generator=gen).to(DTS[dt])
    for drop in (None, DROP):
        h, mean, rstd, y = spec.layer(x, r, w, b, 1e-5, drop)
        o = tcr.tcr_layernorm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), **of(drop), want_stats=True)
        assert same(o.mean, mean) and same(o.rstd, rstd)
        assert same(o.h, h.to(DTS[dt])) and same(o.y, y.to(DTS[dt]))
        q, s = rows_spec.codes(y)
        o = tcr.tcr_layernorm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), **of(drop), out_dtype=torch.int8)
        assert same(o.scale, s) and same(o.y, q) and same(o.h, h.to(DTS[dt]))
    for wi, bi, ri in ((None, None, None), (w, None, r), (None, b, None)):
        h, mean, rstd, y = spec.layer(x, ri, wi, bi, 0.0)
        up = lambda t: None if t is None else t.cuda()      # noqa: E731
        o = tcr.tcr_layernorm(x.cuda(), up(wi), up(bi), residual=up(ri), eps=0.0, want_stats=True)
        assert same(o.mean, mean) and same(o.rstd, rstd) and same(o.y, y.to(DTS[dt]))
        assert (o.h is None) == (ri is None)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 4096), (3, 77), (4, 5001), (640, 768), (401, 2051), (33, 20000)])
def test_layer_against_binary64(rows, cols, dt):
    gen = torch.Generator().manual_seed(rows + cols)
    x, r = rand(gen, rows, cols, DTS[dt]) + 2, rand(gen, rows, cols, DTS[dt])
    x = x.to(DTS[dt])
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    b = torch.randn(cols, generator=gen).to(DTS[dt])
    eps = 1e-5
    h, mean, rstd, y = spec.layer64(x, r, w, b, eps, DROP)
    o = tcr.tcr_layernorm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), eps=eps, **of(DROP), want_stats=True)
    d = rows_spec.depth(cols)
    # h = r + x s: the factor s is rounded (U |x s|), the product (U |x s|), the sum (U of
    # it, |h| and the two errors before)
    xs = (h - r.double()).abs()
    eh = U * (2 * xs + h.abs()) * (1 + 4 * U)
    e = (d + 1) * U * h.abs().mean(1) + U * mean.abs() + eh.mean(1)
    ed = e[:, None] + eh + U * (h - mean[:, None]).abs()
    # the variance: its terms' errors by Cauchy, then the sum's roundings
    rel = (d + 3) * U + 2 * rstd * (ed * ed).mean(1).sqrt() + (rstd * rstd) * (ed * ed).mean(1)
    assert ((o.mean.cpu().double() - mean).abs() <= e).all()
    assert ((o.rstd.cpu().double() - rstd).abs() <= rstd * (rel / 2 + 3 * U)).all()
    wd = w.double().abs()
    off = wd * rstd[:, None] * (ed + (h - mean[:, None]).abs() * (rel[:, None] / 2 + 6 * U)) + 2 * U * (y.abs() + b.double().abs())
    out = rows_spec.EPS_OUT[DTS[dt]]
    assert ((o.y.cpu().double() - y).abs() <= off + out * (y.abs() + off) + rows_spec.TINY[DTS[dt]]).all()
    assert ((o.h.cpu().double() - h).abs() <= eh + out * (h.abs() + eh) + rows_spec.TINY[DTS[dt]]).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(5, 1), (9, 31), (11, 255), (9, 257), (20, 500), (9, 513), (13, 1023), (7, 1999),
                                       (5, 2049), (1300, 2051), (4, 3001), (9, 4095), (7, 4097), (320, 8191),
                                       (4, 8193), (3, 12001), (3, 16383), (3, 33000)])
def test_strides_and_alignment_do_not_change_bits(rows, cols, dt):
    gen = torch.Generator().manual_seed(rows + cols)
    x, r, dy = (rand(gen, rows, cols, DTS[dt]) for _ in range(3))
    x[1], r[1] = 0, 0                                    # with eps = 0: an infinite rstd
    x[2, cols // 2] = float("inf")
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    b = torch.randn(cols, generator=gen).to(DTS[dt])
    even, wide = (cols + 15) // 16 * 16, cols + 3
    for i8 in (False, True):
        t = torch.int8 if i8 else DTS[dt]
        got = []
        for pitch, off in ((even, 0), (wide, 1)):
            out = torch.full((rows, pitch + off), 7, dtype=t, device="cuda")
            h = torch.full((rows, pitch + off), 7, dtype=DTS[dt], device="cuda")
            o = tcr.tcr_layernorm(strided(x, pitch, off), strided(w[None], cols, off)[0],
                                  strided(b[None], cols, 2 * off)[0], residual=strided(r, pitch, off), eps=0.0,
                                  **of(DROP), h=h[:, off:off + cols], out=out[:, off:off + cols], want_stats=True)
            for g in (out, h):                           # nothing beside the rows was written
                assert (g[:, :off] == 7).all() and (g[:, off + cols:] == 7).all()
            got.append(o)
        a, c = got
        assert same(a.y, c.y) and same(a.h, c.h) and same(a.mean, c.mean) and same(a.rstd, c.rstd)
        assert not i8 or same(a.scale, c.scale)
    mean, rstd = torch.randn(rows, generator=gen).cuda(), (torch.rand(rows, generator=gen) + 0.5).cuda()
    rstd[0] = float("inf")
    got = []
    for pitch, off in ((even, 0), (wide, 1)):
        dx = torch.full((rows, pitch + off), 7, dtype=DTS[dt], device="cuda")
        dr = torch.full((rows, pitch + off), 7, dtype=DTS[dt], device="cuda")
        g = tcr.tcr_layernorm_backward(strided(dy, pitch, off), strided(x, pitch, off), strided(w[None], cols, off)[0],
                                       mean, rstd, dh=strided(r, pitch, off), **of(DROP), dx=dx[:, off:off + cols],
                                       dresidual=dr[:, off:off + cols])
        for t in (dx, dr):
            assert (t[:, :off] == 7).all() and (t[:, off + cols:] == 7).all()
        got.append(g)
    assert all(same(p, q) for p, q in zip(*got))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("cols", [9, 128, 255, 1000, 1501, 2560, 5001, 9000])
def test_every_tensor_at_an_alignment_of_its_own(cols, dt):
    gen = torch.Generator().manual_seed(cols)
    rnd = lambda n: int(torch.randint(0, n, (1,), generator=gen))      # noqa: E731
    rows = 7
    x, r, dy, dh = (rand(gen, rows, cols, DTS[dt]) for _ in range(4))
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    b = torch.randn(cols, generator=gen).to(DTS[dt])

    def place(t):
        return strided(t, cols + rnd(9), rnd(9)) if t.dim() == 2 else strided(t[None], cols, rnd(9))[0]

    want = tcr.tcr_layernorm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), **of(DROP), want_stats=True)
    codes = tcr.tcr_layernorm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), **of(DROP), out_dtype=torch.int8)
    grad = tcr.tcr_layernorm_backward(dy.cuda(), want.h, w.cuda(), want.mean, want.rstd, dh=dh.cuda(), **of(DROP),
                                      want_dresidual=True)
    for _ in range(6):
        o = tcr.tcr_layernorm(place(x), place(w), place(b), residual=place(r), **of(DROP), h=place(x), out=place(x),
                              want_stats=True)
        assert same(o.y, want.y) and same(o.h, want.h) and same(o.mean, want.mean) and same(o.rstd, want.rstd)
        q = tcr.tcr_layernorm(place(x), place(w), place(b), residual=place(r), **of(DROP), h=place(x),
                              out=place(codes.y.cpu()))
        assert same(q.y, codes.y) and same(q.scale, codes.scale)
        g = tcr.tcr_layernorm_backward(place(dy), place(want.h.cpu()), place(w), want.mean, want.rstd, dh=place(dh),
                                       **of(DROP), dx=place(x), dresidual=place(x))
        assert all(same(p, q) for p, q in zip(g, grad))
        y = tcr.tcr_dropout(place(x), **of(DROP), residual=place(r), out=place(x))
        assert same(y, want.h)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 8), (3, 100), (200, 257), (700, 513), (5, 1000), (321, 2049), (157, 2600), (9, 4100), (401, 1400), (700, 5100),
                                       (7, 6000), (5, 7000),
                                       (4, 8192), (3, 8200), (2, 20003)])
def test_gradient_bits(rows, cols, dt):
    gen = torch.Generator().manual_seed(rows * cols)
    h, dy, dh = rand(gen, rows, cols, DTS[dt]), rand(gen, rows, cols, DTS[dt], 0.3), rand(gen, rows, cols, DTS[dt], 0.1)
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    _, mean, rstd, _ = spec.layer(h, None, None, None, 1e-5)
    for wi, dhi, drop in ((w, dh, DROP), (w, None, None), (None, dh, None)):
        dx, dr, dw, db = spec.layer_back(dy, h, wi, mean, rstd, dhi, drop)
        up = lambda t: None if t is None else t.cuda()      # noqa: E731
        g = tcr.tcr_layernorm_backward(dy.cuda(), h.cuda(), up(wi), mean.cuda(), rstd.cuda(), dh=up(dhi), **of(drop),
                                       want_dresidual=True)
        assert same(g.dx, dx.to(DTS[dt])) and same(g.dresidual, dr.to(DTS[dt]))
        assert same(g.dbias, db)
        assert g.dweight is None if wi is None else same(g.dweight, dw)
    # each output alone is the same; in place over dy, h and dh
    args = (dy.cuda(), h.cuda(), w.cuda(), mean.cuda(), rstd.cuda())
    want = tcr.tcr_layernorm_backward(*args, dh=dh.cuda(), **of(DROP), want_dresidual=True)
    g = tcr.tcr_layernorm_backward(*args, dh=dh.cuda(), **of(DROP), want_dweight=False, want_dbias=False)
    assert same(g.dx, want.dx) and g.dweight is None and g.dbias is None and g.dresidual is None
    g = tcr.tcr_layernorm_backward(*args, dh=dh.cuda(), **of(DROP), want_dbias=False)
    assert same(g.dweight, want.dweight)
    for k in range(3):
        a = [t.clone() for t in args]
        d = dh.cuda()
        into = (a[0], a[1], d)
        g = tcr.tcr_layernorm_backward(*a, dh=d, **of(DROP), dx=into[k], dresidual=into[(k + 1) % 3])
        assert same(g.dx, want.dx) and same(g.dresidual, want.dresidual) and same(g.dbias, want.dbias)


def test_gradient_against_differences_and_autograd():
    # central differences of the binary64 loss along random directions, whose own error is of
    # order step^2; the kernels' by binary32 roundings and the stored h's (binary32)
    gen = torch.Generator().manual_seed(2)
    rows, cols, eps = 6, 333, 1e-5
    x, r, dy = (torch.randn(rows, cols, generator=gen) for _ in range(3))
    w, b = torch.rand(cols, generator=gen) + 0.5, torch.randn(cols, generator=gen)
    o = tcr.tcr_layernorm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), eps=eps, **of(DROP), want_stats=True)
    g = tcr.tcr_layernorm_backward(dy.cuda(), o.h, w.cuda(), o.mean, o.rstd, **of(DROP), want_dresidual=True)

    def loss(x, r, w, b):
        return (spec.layer64(x, r, w, b, eps, DROP)[3] * dy.double()).sum()

    args = [t.double() for t in (x, r, w, b)]
    leaves = [t.clone().requires_grad_() for t in args]
    loss(*leaves).backward()
    for k, got in enumerate((g.dx, g.dresidual, g.dweight, g.dbias)):
        got = got.cpu().double()
        assert torch.allclose(got, leaves[k].grad, rtol=1e-4, atol=1e-5 * float(leaves[k].grad.abs().max()))
        v = torch.randn(args[k].shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + step * v, args[k] - step * v
        diff = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(float((got * v).sum()) - float(diff)) <= 1e-5 * float((got * v).abs().sum()) + 1e-6


def test_nothing_and_refusals():
    f = torch.float32
    empty = torch.empty(0, 64, device="cuda")
    assert tcr.tcr_dropout(empty, p=0.1).shape == (0, 64)
    assert tcr.tcr_layernorm(empty, want_stats=True).mean.shape == (0,)
    g = tcr.tcr_layernorm_backward(empty, empty, torch.ones(64, device="cuda"), empty[:, 0], empty[:, 0])
    assert (g.dweight == 0).all() and (g.dbias == 0).all()
    flat = torch.empty(3, 0, device="cuda")
    o = tcr.tcr_layernorm(flat, out_dtype=torch.int8, want_stats=True)
    assert (o.scale == 0).all() and o.mean.isnan().all() and o.rstd.isnan().all()
    assert tcr.tcr_layernorm_backward(flat, flat, None, o.mean, o.rstd).dx.shape == (3, 0)
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(4, device="cuda")
    bad = [
        (ValueError, lambda: tcr.tcr_dropout(x, p=-0.1)), (ValueError, lambda: tcr.tcr_dropout(x, p=1.5)),
        (ValueError, lambda: tcr.tcr_dropout(x, p=float("nan"))), (TypeError, lambda: tcr.tcr_dropout(x.int(), p=0.1)),
        (ValueError, lambda: tcr.tcr_dropout(x.cpu(), p=0.1)), (ValueError, lambda: tcr.tcr_dropout(x.t(), p=0.1)),
        (ValueError, lambda: tcr.tcr_dropout(x, p=0.1, residual=x[:3])),
        (TypeError, lambda: tcr.tcr_dropout(x, p=0.1, out=torch.zeros(4, 64, device="cuda"))),
        (ValueError, lambda: tcr.tcr_dropout(x, p=0.1, out=x[:1].expand(4, 64))),
        (TypeError, lambda: tcr.tcr_dropout(x, p=0.1, state=torch.zeros(2, device="cuda"))),
        (ValueError, lambda: tcr.tcr_dropout(x, p=0.1, state=torch.zeros(3, device="cuda", dtype=torch.int64))),
        (ValueError, lambda: tcr.tcr_dropout(x, p=0.1, state=torch.zeros(2, dtype=torch.int64))),
        (TypeError, lambda: tcr.tcr_dropout(x, p=0.1, seed=1.5)),
        (ValueError, lambda: tcr.tcr_layernorm(x, x[0, :63])), (ValueError, lambda: tcr.tcr_layernorm(x, None, x[0, :63])),
        (TypeError, lambda: tcr.tcr_layernorm(x, x[0].float())), (ValueError, lambda: tcr.tcr_layernorm(x, p=2.0)),
        (ValueError, lambda: tcr.tcr_layernorm(x, scale=v)), (TypeError, lambda: tcr.tcr_layernorm(x, out_dtype=f)),
        (tcr.TcrError, lambda: tcr.tcr_layernorm(x, eps=-1.0)), (tcr.TcrError, lambda: tcr.tcr_layernorm(x, eps=float("inf"))),
        (ValueError, lambda: tcr.tcr_layernorm(x, mean=v[:3])),
        (ValueError, lambda: tcr.tcr_layernorm_backward(x, x, None, v[:3], v)),
        (ValueError, lambda: tcr.tcr_layernorm_backward(x, x, None, v, v[:3])),
        (TypeError, lambda: tcr.tcr_layernorm_backward(x.float(), x, None, v, v)),
        (ValueError, lambda: tcr.tcr_layernorm_backward(x, x, None, v, v, dbias=v)),
        (TypeError, lambda: tcr.tcr_layernorm_backward(x, x, None, v, v, dbias=x[0])),
        (ValueError, lambda: tcr.tcr_layernorm_backward(x, x, None, v, v, dresidual=x[:2])),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_failed_calls_leave_outputs_alone(monkeypatch):
    x, v = torch.ones(4, 64, device="cuda"), torch.ones(4, device="cuda")
    out, d = torch.full((4, 64), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    for what in ("launch", "alloc"):
        monkeypatch.setenv("TCR_FAULT_INJECT", what)
        if what == "launch":
            with pytest.raises(tcr.TcrError):
                tcr.tcr_dropout(x, p=0.1, out=out)
            with pytest.raises(tcr.TcrError):
                tcr.tcr_layernorm(x, out=out)
        with pytest.raises(tcr.TcrError):
            tcr.tcr_layernorm_backward(x, x, None, v, v, dx=out, dbias=d)
    monkeypatch.delenv("TCR_FAULT_INJECT")
    assert (out == 5).all() and (d == 5).all()


def test_streams_graphs_and_threads():
    gen = torch.Generator().manual_seed(5)
    x, r = rand(gen, 640, 2048, torch.bfloat16).cuda(), rand(gen, 640, 2048, torch.bfloat16).cuda()
    w = torch.ones(2048, dtype=torch.bfloat16, device="cuda")

    def step(**kw):
        o = tcr.tcr_layernorm(x, w, residual=r, **of(DROP), want_stats=True, **kw)
        g = tcr.tcr_layernorm_backward(x, o.h, w, o.mean, o.rstd, **of(DROP), want_dresidual=True, **kw)
        return (*o[:1], *o[2:], *g)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    s.synchronize()
    assert all(same(a, b) for a, b in zip(want, got))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        a = step()
    with torch.cuda.graph(g2):
        b = step()
    for _ in range(3):
        for t in (*a, *b):
            t.zero_()
        g1.replay()
        g2.replay()
        assert all(same(p, q) for p, q in zip(want, a)) and all(same(p, q) for p, q in zip(want, b))
    wrong = []

    def work():
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(8):
                got = step()
                st.synchronize()
                if not all(same(p, q) for p, q in zip(want, got)):
                    wrong.append(1)

    ts = [threading.Thread(target=work) for _ in range(4)]
    torch.cuda.synchronize()
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("cols", [1, 31, 256, 500, 1000, 1001, 2560, 5001, 7168, 16384, 16391, 40000])
def test_outputs_over_the_inputs(cols, dt):
    gen = torch.Generator().manual_seed(cols)
    x, r = rand(gen, 9, cols, DTS[dt]), rand(gen, 9, cols, DTS[dt])
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt]).cuda()
    b = torch.randn(cols, generator=gen).to(DTS[dt]).cuda()
    want = tcr.tcr_layernorm(x.cuda(), w, b, residual=r.cuda(), **of(DROP), want_stats=True)
    codes = tcr.tcr_layernorm(x.cuda(), w, b, residual=r.cuda(), **of(DROP), out_dtype=torch.int8)
    alone = tcr.tcr_layernorm(x.cuda(), w, b)
    for pitch, off in (((cols + 7) // 8 * 8, 0), (cols + 3, 1)):
        def xr():
            return strided(x, pitch, off), strided(r, pitch, off)

        for over_x in (True, False):                     # h over one, y over the other
            xs, rs = xr()
            o = tcr.tcr_layernorm(xs, w, b, residual=rs, **of(DROP), h=xs if over_x else rs, out=rs if over_x else xs,
                                  want_stats=True)
            assert same(o.h, want.h) and same(o.y, want.y) and same(o.mean, want.mean) and same(o.rstd, want.rstd)
            xs, rs = xr()
            o = tcr.tcr_layernorm(xs, w, b, residual=rs, **of(DROP), h=xs if over_x else rs, out_dtype=torch.int8)
            assert same(o.h, want.h) and same(o.y, codes.y) and same(o.scale, codes.scale)
        xs, _ = xr()
        assert same(tcr.tcr_layernorm(xs, w, b, out=xs).y, alone.y)


def test_the_widest_rows():
    # 2^27 columns, the documented limit; every sum a power of two or exact
    cols = 1 << 27
    h = torch.zeros(1, cols, dtype=torch.float16, device="cuda")
    h[0, ::2] = 2.0                                      # mean 1, variance 1
    o = tcr.tcr_layernorm(h, eps=0.0, want_stats=True)
    assert o.mean.item() == 1.0 and o.rstd.item() == 1.0 and torch.equal(o.y, h - 1)
    dy = torch.ones(1, cols, dtype=torch.float16, device="cuda")
    dy[0, ::4] = 3.0                                     # mean 1.5, mean of dy * xh 0.5
    g = tcr.tcr_layernorm_backward(dy, h, None, o.mean, o.rstd)
    assert torch.equal(g.dx, dy - 1.5 - (h - 1) * 0.5) and torch.equal(g.dbias, dy[0].float())
    k = spec.keep(1, 1 << 16, *DROP)
    assert torch.equal((tcr.tcr_dropout(dy, **of(DROP)) > 0)[:, :1 << 16].cpu(), k)
