"""The norm with the residual's addition, its gradient, the 8-bit row
quantiser and the reader of its codes.

Two references: the declared binary32 operations restated on the CPU
(tests/rows_spec.py), which results match bit for bit, and the definitions in
binary64, within bounds that follow from the roundings: a row sum of
non-negative terms over d tree levels is within (d + 1) U, so rstd and y are
within (d/2 + 8) U <= 2^-20 relative before the output's own rounding.
"""
import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests import rows_spec as spec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BITS = {2: torch.int16, 4: torch.int32, 1: torch.int8}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)


def same(a, b):
    """Bit equality, all NaNs alike."""
    a, b = a.detach().cpu().contiguous(), b.detach().cpu().contiguous()
    assert a.dtype == b.dtype and a.shape == b.shape
    if a.dtype.is_floating_point:
        na, nb = torch.isnan(a), torch.isnan(b)
        assert torch.equal(na, nb)
        a, b = a.masked_fill(na, 0), b.masked_fill(nb, 0)
    return torch.equal(a.view(BITS[a.element_size()]), b.view(BITS[b.element_size()]))


def rand(gen, rows, cols, dt, scale=1.0):
    return (torch.randn(rows, cols, generator=gen) * scale).to(dt)


def strided(t, pitch, offset):
    """t on the GPU as a slice of a wider matrix: rows `pitch` apart, starting
    `offset` elements into it."""
    rows, cols = t.shape
    base = torch.zeros(rows, pitch + offset, dtype=t.dtype, device="cuda")
    v = base[:, offset:offset + cols]
    v.copy_(t)
    return v


COLS = [1, 2, 7, 8, 9, 31, 100, 255, 256, 257, 500, 512, 513, 1001, 1024, 1025, 2048, 2049, 4096, 4099,
        8192, 8200, 16384, 16391, 32768, 32769, 40000]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("cols", COLS)
def test_norm_bits(cols, dt):
    gen = torch.Generator().manual_seed(cols)
    rows = 5
    x, r = rand(gen, rows, cols, DTS[dt]), rand(gen, rows, cols, DTS[dt], 2.0)
    x[2], r[2] = 0, 0                                   # an empty token
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    h, rstd, y = spec.norm(x, r, w, 1e-6)
    o = tcr.tcr_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-6, want_rstd=True)
    assert same(o.rstd, rstd)
    assert same(o.h, h.to(DTS[dt]))
    assert same(o.y, y.to(DTS[dt]))
    q, s = spec.codes(y)
    o = tcr.tcr_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-6, out_dtype=torch.int8)
    assert same(o.scale, s)
    assert same(o.y, q)
    assert same(o.h, h.to(DTS[dt]))
    assert same(tcr.tcr_dequantize_rows_i8(o.y, o.scale, dtype=DTS[dt]),
                (q.float() * s[:, None]).to(DTS[dt]))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 4096), (3, 77), (4, 5001), (640, 768), (401, 2051), (320, 20000)])
def test_norm_against_binary64(rows, cols, dt):
    gen = torch.Generator().manual_seed(rows + cols)
    x, r = rand(gen, rows, cols, DTS[dt]), rand(gen, rows, cols, DTS[dt])
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    h, y = spec.norm64(x, r, w, 1e-5)
    o = tcr.tcr_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-5)
    rel = 2.0 ** -20 + spec.EPS_OUT[DTS[dt]]
    assert ((o.y.cpu().double() - y).abs() <= rel * y.abs() + spec.TINY[DTS[dt]]).all()
    assert ((o.h.cpu().double() - h).abs() <= rel * h.abs() + spec.TINY[DTS[dt]]).all()
    o = tcr.tcr_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-5, out_dtype=torch.int8)
    s = y.abs().amax(1) / 127
    assert ((o.scale.cpu().double() - s).abs() <= 2.0 ** -19 * s).all()
    assert ((o.y.cpu().double() - y / s[:, None]).abs() <= 0.5 + 127 * 2.0 ** -18).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols,pitch,off", [(7, 500, 503, 1), (5, 4096, 4104, 3), (401, 1001, 1001, 5),
                                                 (3, 9000, 9001, 0), (6, 33000, 33003, 2), (9, 64, 200, 8)])
def test_strides_and_alignment_do_not_change_bits(rows, cols, pitch, off, dt):
    gen = torch.Generator().manual_seed(rows)
    x, r, dy = (rand(gen, rows, cols, DTS[dt]) for _ in range(3))
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    ws = strided(w[None], cols, 1)[0]
    for i8 in (False, True):
        out_t = torch.int8 if i8 else DTS[dt]
        a = tcr.tcr_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), out_dtype=out_t, want_rstd=True)
        guard = torch.full((rows, pitch + off), 7, dtype=out_t, device="cuda")
        hg = torch.full((rows, pitch + off), 7, dtype=DTS[dt], device="cuda")
        b = tcr.tcr_rmsnorm(strided(x, pitch, off), ws, residual=strided(r, pitch + 1, off), want_rstd=True,
                            out=guard[:, off:off + cols], h=hg[:, off:off + cols])
        assert same(a.y, b.y) and same(a.h, b.h) and same(a.rstd, b.rstd)
        for g in (guard, hg):                            # nothing beside the rows was written
            assert (g[:, :off] == 7).all() and (g[:, off + cols:] == 7).all()
    q, s = tcr.tcr_quantize_rows_i8(x.cuda(), gate=r.cuda())
    qs, ss = tcr.tcr_quantize_rows_i8(strided(x, pitch, off), gate=strided(r, pitch, off))
    assert same(q, qs) and same(s, ss)
    assert same(tcr.tcr_dequantize_rows_i8(q, s, dtype=DTS[dt]),
                tcr.tcr_dequantize_rows_i8(strided(q.cpu(), pitch, off), s,
                                           out=strided(torch.zeros(rows, cols, dtype=DTS[dt]), pitch, off)))
    dx, dw = tcr.tcr_rmsnorm_backward(dy.cuda(), a.h, w.cuda(), a.rstd, dh=r.cuda())
    dxs, dws = tcr.tcr_rmsnorm_backward(strided(dy, pitch, off), b.h, ws, b.rstd, dh=strided(r, pitch, off),
                                        dx=strided(torch.zeros(rows, cols, dtype=DTS[dt]), pitch, off))
    assert same(dx, dxs) and same(dw, dws)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(5, 1), (9, 31), (11, 255), (9, 257), (20, 500), (9, 513), (13, 1023), (7, 1999),
                                       (5, 2049), (1300, 2051), (1300, 2560), (6, 2561), (4, 3001), (9, 4095),
                                       (7, 4097), (5, 6145), (320, 8191), (4, 8193), (3, 12001), (3, 16383)])
def test_unaligned_rows_have_the_bits_of_aligned_ones(rows, cols, dt):
    gen = torch.Generator().manual_seed(rows + cols)
    x, r, dy = (rand(gen, rows, cols, DTS[dt]) for _ in range(3))
    x[1], r[1] = 0, 0                                    # with eps = 0: an infinite rstd
    x[2, cols // 2] = float("inf")
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    rstd = (torch.rand(rows, generator=gen) + 0.5).cuda()
    even = (cols + 15) // 16 * 16
    odd = even + 1

    def guarded(dtype, pitch, off):
        g = torch.full((rows, pitch + off), 7, dtype=dtype, device="cuda")
        return g, g[:, off:off + cols]

    # (inputs, outputs) aligned, both not, and either alone
    got = []
    for pi, po in ((even, even), (odd, odd), (odd, even), (even, odd)):
        oi, oo = (1 if pi == odd else 0), (1 if po == odd else 0)
        xs, rs, dys = (strided(t, pi, oi) for t in (x, r, dy))
        ws = strided(w[None], even, oi)[0]
        guards, outs = zip(*(guarded(t, po, oo) for t in (DTS[dt], DTS[dt], torch.int8, DTS[dt], torch.int8, DTS[dt],
                                                          DTS[dt])))
        a = tcr.tcr_rmsnorm(xs, ws, residual=rs, out=outs[0], h=outs[1], want_rstd=True)
        b = tcr.tcr_rmsnorm(xs, ws, residual=rs, eps=0.0, out=outs[2], h=outs[3])
        q, s = tcr.tcr_quantize_rows_i8(xs, gate=rs, out=outs[4])
        tcr.tcr_dequantize_rows_i8(strided(q.cpu(), pi, oi), s, out=outs[5])
        _, dw = tcr.tcr_rmsnorm_backward(dys, rs, ws, rstd, dh=rs, dx=outs[6])
        for g in guards:                                 # nothing beside the rows was written
            pad = g.clone()
            pad[:, oo:oo + cols] = 7
            assert (pad == 7).all()
        got.append([*outs, a.rstd, b.scale, s, dw])
    for other in got[1:]:
        assert all(same(u, v) for u, v in zip(got[0], other))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(4, 1), (4, 100), (5, 1001), (4, 1500), (1300, 2560), (9, 2560), (4, 2561), (4, 5001),
                                       (4, 7000), (3, 8192), (4, 8200), (4, 12289)])
def test_gradient_of_an_infinite_rstd(rows, cols, dt):
    # what a forward pass with eps = 0 returns where a row's squares vanish: the
    # row's sum is of its own elements, whatever lanes and vectors stay empty
    gen = torch.Generator().manual_seed(rows + cols)
    h, dy = rand(gen, rows, cols, DTS[dt]), rand(gen, rows, cols, DTS[dt])
    h[1], dy[1] = 1e-7, 1.0                              # products of one sign: the sum is infinite, not NaN
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    rstd = torch.rand(rows, generator=gen) + 0.5
    rstd[1] = float("inf")
    dxc, dwc = spec.back(dy, h, w, rstd, None)
    assert (dxc[1] == -float("inf")).all() and torch.isinf(dwc).all() and torch.isfinite(dxc[[0, 2]]).all()
    wide, ld = w.cuda(), (cols + 15) // 16 * 16
    for pitch, off in ((ld, 0), (ld + 1, 1)):
        dx, dw = tcr.tcr_rmsnorm_backward(strided(dy, pitch, off), strided(h, pitch, off), wide, rstd.cuda())
        assert same(dx, dxc.to(DTS[dt])) and same(dw, dwc)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 12000])
def test_a_row_does_not_depend_on_the_others(cols):
    gen = torch.Generator().manual_seed(1)
    x = rand(gen, 700, cols, torch.bfloat16).cuda()
    all_rows = tcr.tcr_rmsnorm(x, out_dtype=torch.int8, want_rstd=True)
    few = tcr.tcr_rmsnorm(x[123:126], out_dtype=torch.int8, want_rstd=True)
    assert same(all_rows.y[123:126], few.y) and same(all_rows.scale[123:126], few.scale)
    assert same(all_rows.rstd[123:126], few.rstd)
    q, s = tcr.tcr_quantize_rows_i8(x)
    q1, s1 = tcr.tcr_quantize_rows_i8(x[699:])
    assert same(q[699:], q1) and same(s[699:], s1)


def test_in_place_and_optional_arguments():
    gen = torch.Generator().manual_seed(3)
    for cols in (300, 4096, 4099, 40000):
        x, r = rand(gen, 9, cols, torch.float16), rand(gen, 9, cols, torch.float16)
        want = tcr.tcr_rmsnorm(x.cuda(), residual=r.cuda())
        xs, rs = x.cuda(), r.cuda()
        got = tcr.tcr_rmsnorm(xs, residual=rs, h=rs, out=xs)      # residual stream updated in place
        assert got.h is rs and same(want.h, rs) and same(want.y, xs)
        plain = tcr.tcr_rmsnorm(x.cuda())
        assert plain.h is None and plain.scale is None and plain.rstd is None
        assert same(plain.y, spec.norm(x, None, None, 1e-6)[2].half())
        # one row for all: an expanded residual
        one = tcr.tcr_rmsnorm(x.cuda(), residual=r[:1].cuda().expand(9, cols))
        assert same(one.y, tcr.tcr_rmsnorm(x.cuda(), residual=r[:1].repeat(9, 1).cuda()).y)


def test_empty_sizes():
    dev = dict(device="cuda", dtype=torch.bfloat16)
    o = tcr.tcr_rmsnorm(torch.empty(0, 64, **dev), out_dtype=torch.int8)
    assert o.y.shape == (0, 64) and o.scale.shape == (0,)
    o = tcr.tcr_rmsnorm(torch.empty(3, 0, **dev), out_dtype=torch.int8, want_rstd=True)
    assert (o.scale == 0).all() and torch.isnan(o.rstd).all()
    q, s = tcr.tcr_quantize_rows_i8(torch.empty(2, 0, **dev))
    assert (s == 0).all()
    dx, dw = tcr.tcr_rmsnorm_backward(torch.empty(0, 40, **dev), torch.empty(0, 40, **dev),
                                      torch.ones(40, **dev), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 40) and (dw == 0).all()


def test_rows_that_are_not_finite_or_vanish():
    cols = 200
    x = torch.ones(6, cols)
    x[0, 7] = float("nan")
    x[1, 100] = float("inf")
    x[2] = 0
    x[3] = 1e-39                                          # scale below the normal numbers
    x[4] = 0
    x[4, 3] = -3e38
    q, s = tcr.tcr_quantize_rows_i8(x.cuda())
    qc, sc = spec.codes(x)
    assert same(q, qc) and same(s, sc)
    assert torch.isnan(s[0]) and torch.isnan(s[1]) and s[2] == 0 and s[3] == 0 and q[4, 3] == -127
    back = tcr.tcr_dequantize_rows_i8(q, s)
    assert torch.isnan(back[:2]).all() and (back[2:4] == 0).all()
    for dt in (torch.float16, torch.bfloat16):            # the type's lowest value in a masked place
        y = torch.zeros(1, 64, dtype=dt)
        y[0, 1], y[0, 2] = torch.finfo(dt).min, 1.0
        q, s = tcr.tcr_quantize_rows_i8(y.cuda())
        assert same(q, spec.codes(y.float())[0]) and q[0, 1] == -127 and q[0, 2] == 0
    o = tcr.tcr_rmsnorm(x[:3].cuda(), out_dtype=torch.int8)
    assert torch.isnan(o.scale[:2]).all() and (o.y == 0).all() and o.scale[2] == 0


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 333), (300, 4096), (7, 17000), (2, 35001)])
def test_gated_quantiser(rows, cols, dt):
    gen = torch.Generator().manual_seed(cols)
    both = rand(gen, rows, 2 * cols, DTS[dt], 3.0)
    both[0, 0] = -90.0                                    # exp overflows on the way to silu = -0
    gate, up = both[:, :cols], both[:, cols:]
    y = gate.double() * torch.sigmoid(gate.double()) * up.double()
    b = both.cuda()
    q, s = tcr.tcr_quantize_rows_i8(b[:, cols:], gate=b[:, :cols])
    want = y.abs().amax(1, keepdim=True) / 127
    # CUDA's fast exponential is within 2 + 1.173 |g| ulp and counts where it
    # is not small beside 1 (g < 0), its quotient within 2; three roundings;
    # below exp(-87) the quotient gives 0
    err = (8 + 1.2 * (-gate.double()).clamp(min=0)) * 2.0 ** -23 * y.abs() + 1e-30
    serr = err.amax(1, keepdim=True) / 127 + 2.0 ** -22 * want
    assert ((s.cpu().double()[:, None] - want).abs() <= serr).all()
    assert ((q.cpu().double() - y / want).abs() <= 0.5 + (err + 127 * serr) / want).all()
    q, s = tcr.tcr_quantize_rows_i8(both.cuda())
    qc, sc = spec.codes(both.float())
    assert same(q, qc) and same(s, sc)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [1, 100, 1001, 9001, 40000])
def test_gate_where_its_factor_vanishes(cols, dt):
    # rows of one gate and values near the type's largest.  Down to -87.33 the
    # declared bound holds; from -87.34 on the quotient's denominator is past
    # 2^126 and the factor 0
    small, zero = ([-80.0, -86.5, -87.0], [-87.5, -88.0, -89.0, -100.0]) if dt == "bf16" else \
        ([-80.0, -87.0, -87.2, -87.33], [-87.34, -87.5, -88.5, -89.0, -200.0])
    gen = torch.Generator().manual_seed(cols)
    gates = torch.tensor(small + zero + [float("inf"), -float("inf")])
    x = ((torch.rand(len(gates), cols, generator=gen) + 1) * 1e38).to(DTS[dt])
    g = gates[:, None].expand(len(gates), cols).to(DTS[dt])
    y = g.double() / (1 + torch.exp(-g.double())) * x.double()
    q, s = (t.cpu() for t in tcr.tcr_quantize_rows_i8(x.cuda(), gate=g.cuda()))
    n, m = len(small), len(small) + len(zero)
    want = y.abs().amax(1) / 127
    # the declared bound, and the scale's own quotient
    err = (8 + 1.2 * -g[:n, 0].double()) * 2.0 ** -23 + 2.0 ** -23
    assert ((s[:n].double() - want[:n]).abs() <= err * want[:n]).all() and (s[:n] > 0).all()
    assert ((q[:n].double() - y[:n] / want[:n, None]).abs() <= 0.5 + 2 * 127 * err[:, None]).all()
    assert (s[n:m] == 0).all() and torch.isnan(s[m:]).all() and (q[n:] == 0).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 9), (33, 500), (310, 513), (700, 1024), (40, 2047), (9, 4096),
                                       (160, 4100), (5, 8192), (20, 16384), (12, 16385), (310, 17001)])
def test_backward(rows, cols, dt):
    gen = torch.Generator().manual_seed(rows * 7 + cols)
    h, dy, dh = (rand(gen, rows, cols, DTS[dt]) for _ in range(3))
    if rows > 2:
        h[1] = 0
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt])
    rstd = spec.norm(h, None, None, 1e-6)[1]
    cu = [t.cuda() for t in (dy, h, w, rstd, dh)]
    dx, dw = tcr.tcr_rmsnorm_backward(cu[0], cu[1], cu[2], cu[3], dh=cu[4])
    dxc, dwc = spec.back(dy, h, w, rstd, dh)
    assert same(dx, dxc.to(DTS[dt])) and same(dw, dwc)
    # binary64: the row sum is within (depth + 2) U of its terms' sizes, four
    # roundings follow; a column's sum has at most rows/G + G/32 + 6 levels
    dx64, dw64, size, wsize = spec.back64(dy, h, w, rstd, dh)
    bound = (spec.depth(cols) + 10) * spec.U * size + spec.EPS_OUT[DTS[dt]] * dx64.abs() + spec.TINY[DTS[dt]]
    assert ((dx.cpu().double() - dx64).abs() <= bound * 1.01).all()
    levels = rows / 152 + 304 / 32 + 10
    assert ((dw.cpu().double() - dw64).abs() <= levels * spec.U * wsize + 1e-40).all()
    # without the optional arguments
    dx, none = tcr.tcr_rmsnorm_backward(cu[0], cu[1], None, cu[3])
    assert none is None and same(dx, spec.back(dy, h, None, rstd, None)[0].to(DTS[dt]))
    # over its own inputs, and with one gradient row for all
    buf = cu[4].clone()
    dx2, _ = tcr.tcr_rmsnorm_backward(cu[0], cu[1], cu[2], cu[3], dh=buf, dx=buf)
    assert same(buf, dxc.to(DTS[dt]))
    one = dy[:1].expand(rows, cols)
    dx3, dw3 = tcr.tcr_rmsnorm_backward(cu[0][:1].expand(rows, cols), cu[1], cu[2], cu[3])
    a, b = spec.back(one, h, w, rstd, None)
    assert same(dx3, a.to(DTS[dt])) and same(dw3, b)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,cols", [(3, 9), (40, 500), (700, 1024), (401, 1001), (9, 4096), (160, 4099), (20, 8192),
                                       (7, 12289)])
def test_a_gradient_without_the_weights(rows, cols, dt, monkeypatch):
    # a frozen or absent weight: the same dx, and no scratch but for long rows
    gen = torch.Generator().manual_seed(rows + cols)
    dy, h, dh = (rand(gen, rows, cols, DTS[dt]).cuda() for _ in range(3))
    w = (torch.rand(cols, generator=gen) + 0.5).to(DTS[dt]).cuda()
    rstd = (torch.rand(rows, generator=gen) + 0.5).cuda()
    want, dw = tcr.tcr_rmsnorm_backward(dy, h, w, rstd, dh=dh)
    # a gradient asked for without a weight: that of a weight of ones
    dx1, dw1 = tcr.tcr_rmsnorm_backward(dy, h, None, rstd, dweight=torch.empty(cols, device="cuda"))
    dx2, dw2 = tcr.tcr_rmsnorm_backward(dy, h, torch.ones_like(w), rstd)
    assert same(dw1, dw2) and same(dw1, dw) and same(dx1, dx2)
    if cols <= 8192:
        monkeypatch.setenv("TCR_FAULT_INJECT", "alloc")
    dx, none = tcr.tcr_rmsnorm_backward(dy, h, w, rstd, dh=dh, want_dweight=False)
    assert none is None and same(dx, want)
    dx, none = tcr.tcr_rmsnorm_backward(dy, h, None, rstd)
    assert none is None and same(dx, dx1)


def test_backward_against_differences():
    # central differences of L = sum(dy * y) through the forward call in
    # binary32: step d = 2^-6; the quotient is off by the forward's roundings
    # (2^-20 of sum|dy y| over d) and d^2 / 6 of the third derivative, which
    # for h of unit size is below 15 sum|dy w| rstd^3 * 6
    gen = torch.Generator().manual_seed(11)
    rows, cols, d = 3, 6, 2.0 ** -6
    h, dy = torch.randn(rows, cols, generator=gen), torch.randn(rows, cols, generator=gen)
    w = torch.rand(cols, generator=gen) + 0.5
    o = tcr.tcr_rmsnorm(h.cuda(), w.cuda(), want_rstd=True)
    dx, dw = tcr.tcr_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), o.rstd)

    def loss(hh, ww):
        return (tcr.tcr_rmsnorm(hh.cuda(), ww.cuda()).y.cpu().double() * dy.double()).sum().item()
    size = (dy.double() * o.y.cpu().double()).abs().sum().item()
    third = 15 * (dy * w).abs().sum().item() * max(1.0, o.rstd.max().item() ** 3)
    tol = 2.0 ** -20 * size / d + d * d * third
    for i in range(rows):
        for j in range(cols):
            e = torch.zeros(rows, cols)
            e[i, j] = d
            num = (loss(h + e, w) - loss(h - e, w)) / (2 * d)
            assert abs(num - dx[i, j].item()) <= tol
    for j in range(cols):
        e = torch.zeros(cols)
        e[j] = d
        num = (loss(h, w + e) - loss(h, w - e)) / (2 * d)
        assert abs(num - dw[j].item()) <= 2.0 ** -20 * size / d + 1e-6


def test_wide_pitch_past_32_bits():
    # rows 2^30 elements apart: offsets pass 32 bits
    base = torch.empty((3 << 30) + 64, dtype=torch.int8, device="cuda")
    q = base.as_strided((4, 64), (1 << 30, 1))
    gen = torch.Generator().manual_seed(2)
    x = rand(gen, 4, 64, torch.float32)
    s = torch.empty(4, device="cuda")
    tcr.tcr_quantize_rows_i8(x.cuda(), out=q, scale=s)
    assert same(q.contiguous(), spec.codes(x)[0])
    assert same(tcr.tcr_dequantize_rows_i8(q, s), spec.codes(x)[0].float() * s.cpu()[:, None])


def test_streams_and_graphs():
    gen = torch.Generator().manual_seed(5)
    x, r = rand(gen, 64, 2048, torch.bfloat16).cuda(), rand(gen, 64, 2048, torch.bfloat16).cuda()
    w = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    want = tcr.tcr_rmsnorm(x, w, residual=r, out_dtype=torch.int8, want_rstd=True)
    wdx, wdw = tcr.tcr_rmsnorm_backward(x, want.h, w, want.rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tcr.tcr_rmsnorm(x, w, residual=r, out_dtype=torch.int8, want_rstd=True, stream=s)
    s.synchronize()
    assert same(want.y, got.y) and same(want.scale, got.scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = tcr.tcr_rmsnorm(x, w, residual=r, out_dtype=torch.int8, want_rstd=True)
        dx, dw = tcr.tcr_rmsnorm_backward(x, o.h, w, o.rstd)
    for _ in range(2):
        o.y.zero_()
        dw.zero_()
        g.replay()
        assert same(want.y, o.y) and same(wdx, dx) and same(wdw, dw)


def test_refusals_of_the_binding():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tcr.tcr_rmsnorm(x.int())
    with pytest.raises(ValueError):
        tcr.tcr_rmsnorm(x.cpu())
    with pytest.raises(ValueError):
        tcr.tcr_rmsnorm(x.t())
    with pytest.raises(ValueError):
        tcr.tcr_rmsnorm(x, residual=x[:3])
    with pytest.raises(TypeError):
        tcr.tcr_rmsnorm(x, weight=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        tcr.tcr_rmsnorm(x, weight=x[0, :63])
    with pytest.raises(TypeError):
        tcr.tcr_rmsnorm(x, out_dtype=torch.float32)
    with pytest.raises(ValueError):
        tcr.tcr_rmsnorm(x, out=x[:1].expand(4, 64))       # rows on top of each other
    with pytest.raises(tcr.TcrError):
        tcr.tcr_rmsnorm(x, eps=-1.0)
    with pytest.raises(tcr.TcrError):
        tcr.tcr_rmsnorm(x, eps=float("nan"))
    with pytest.raises(TypeError):
        tcr.tcr_rmsnorm_backward(x.float(), x, None, torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        tcr.tcr_rmsnorm_backward(x, x, None, torch.zeros(5, device="cuda"))
    with pytest.raises(TypeError):
        tcr.tcr_quantize_rows_i8(x, out=torch.zeros(4, 64, device="cuda", dtype=torch.uint8))
    with pytest.raises(ValueError):
        tcr.tcr_dequantize_rows_i8(torch.zeros(4, 64, device="cuda", dtype=torch.int8),
                                   torch.zeros(3, device="cuda"))


def test_failed_calls_leave_outputs_alone(monkeypatch):
    x = torch.ones(4, 64, device="cuda")
    out, dw = torch.full((4, 64), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    for what in ("launch", "alloc"):
        monkeypatch.setenv("TCR_FAULT_INJECT", what)
        if what == "launch":
            with pytest.raises(tcr.TcrError):
                tcr.tcr_rmsnorm(x, out=out)
        with pytest.raises(tcr.TcrError):
            tcr.tcr_rmsnorm_backward(x, x, x[0], torch.ones(4, device="cuda"), dx=out, dweight=dw)
    monkeypatch.delenv("TCR_FAULT_INJECT")
    assert (out == 5).all() and (dw == 5).all()


def test_the_widest_rows():
    # 2^27 columns, the documented limit: 65536 blocks of 2048 columns in the
    # gradient, more than a grid's y or z holds
    cols = 1 << 27
    one = torch.ones(1, cols, dtype=torch.float16, device="cuda")
    h = torch.zeros(1, cols, dtype=torch.float16, device="cuda")
    h[0, ::4] = 2.0                                      # mean square 1
    h[0, -1] = 2.0
    o = tcr.tcr_rmsnorm(h, eps=0.0, want_rstd=True)
    # S = 2^27 + 4, whose sums of halves are ties to 2^27: rstd 1
    assert o.rstd.item() == 1.0 and torch.equal(o.y, h)
    dx, dw = tcr.tcr_rmsnorm_backward(one, h, one[0], o.rstd)
    # S' = 2^26 + 2, likewise: c = 0.5, dx = 1 - h / 2
    assert torch.equal(dx, 1 - h / 2) and torch.equal(dw, h[0].float())
