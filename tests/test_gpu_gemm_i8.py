"""The 8-bit product with scales for each token and channel.

The sums are exact, so int32 outputs equal the product in 64-bit arithmetic
and floating outputs equal (float(S) * sa) * sw, each step rounded once, bit
for bit -- on every path, size, alignment and split.
"""
import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library
from tests.test_gpu_norm import same

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

OUT = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)
    yield
    assert tcr.tcr_device_faults(clear=True) == 0


def codes(gen, rows, cols, lo=-128, hi=128):
    return torch.randint(lo, hi, (rows, cols), generator=gen, device="cuda", dtype=torch.int8)


def sums(a, w):
    # binary64 holds every partial sum (|S| < 2^31) exactly
    return (a.double() @ w.double().t()).to(torch.int32)


def check(a, w, gen, out=None):
    M, N = a.shape[0], w.shape[0]
    s = sums(a, w)
    assert torch.equal(tcr.tcr_gemm_i8(a, w, out_dtype=torch.int32), s)
    sa = torch.rand(M, generator=gen, device="cuda") + 0.1
    sw = torch.rand(N, generator=gen, device="cuda") * 1e-3
    for dt in OUT:
        got = tcr.tcr_gemm_i8(a, w, sa, sw, out_dtype=dt)
        assert same(got, (s.float() * sa[:, None] * sw[None, :]).to(dt))


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(17)


@pytest.mark.parametrize("K", [1, 16, 100, 1024, 1025, 3000])
@pytest.mark.parametrize("N", [1, 7, 130, 256, 300])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 17, 33, 64, 161, 1025, 1057, 1300])
def test_every_small_shape(M, N, K, gen):
    check(codes(gen, M, K), codes(gen, N, K), gen)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (8, 5001, 8192), (9, 8192, 8192), (16, 4096, 4097),
                                   (64, 1000, 16384), (97, 257, 131071), (333, 2051, 4100), (640, 512, 1040),
                                   (1000, 3001, 2064), (33, 8192, 8192), (100, 5000, 8200), (65, 6001, 8191),
                                   (2048, 4096, 4096), (4099, 777, 1536), (7000, 256, 64)])
def test_larger_shapes(M, N, K, gen):
    check(codes(gen, M, K), codes(gen, N, K), gen)


@pytest.mark.parametrize("M", [1, 2, 8, 9, 30, 64, 300, 1100])
@pytest.mark.parametrize("K", [1024, 8192, 131071])
def test_the_largest_sums(M, K, gen):
    # every product 2^14 and of one sign: a chunk's sum is the accumulator's
    # last exact integer, the whole sum the largest that 32 bits hold
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    w[2, ::2] = 127
    w[3] = codes(gen, 1, K)[0]
    w[4] = 0
    check(a, w, gen)


@pytest.mark.parametrize("M", [1, 2, 6, 20, 40, 100, 1030])
@pytest.mark.parametrize("pitch_a,off_a,pitch_w,off_w,K", [(640, 16, 656, 32, 512), (515, 3, 512, 0, 512),
                                                          (512, 0, 600, 5, 500), (1041, 1, 1043, 7, 1037)])
def test_strides_and_alignment(M, pitch_a, off_a, pitch_w, off_w, K, gen):
    N = 300
    a = codes(gen, M, pitch_a + off_a)[:, off_a:off_a + K]
    w = codes(gen, N, pitch_w + off_w)[:, off_w:off_w + K]
    check(a, w, gen)
    c = torch.full((M, N + 9), 7.0, device="cuda")
    tcr.tcr_gemm_i8(a, w, out=c[:, 4:4 + N])
    assert torch.equal(c[:, 4:4 + N], sums(a, w).float())
    assert (c[:, :4] == 7).all() and (c[:, 4 + N:] == 7).all()


def test_empty_sizes(gen):
    a, w = codes(gen, 12, 64), codes(gen, 20, 64)
    assert tcr.tcr_gemm_i8(a[:0], w).shape == (0, 20)
    assert tcr.tcr_gemm_i8(a, w[:0]).shape == (12, 0)
    c = torch.full((12, 30), 7.0, device="cuda")
    tcr.tcr_gemm_i8(a[:, :0], w[:, :0], out=c[:, :20])
    assert (c[:, :20] == 0).all() and (c[:, 20:] == 7).all()


@pytest.mark.parametrize("M", [4, 40])
def test_scales_that_are_not_finite(M, gen):
    a, w = codes(gen, M, 256), codes(gen, 70, 256)
    sa, sw = torch.ones(M, device="cuda"), torch.ones(70, device="cuda")
    sa[1] = float("nan")                                  # a token with a NaN: its row of C only
    sw[5] = float("inf")
    got = tcr.tcr_gemm_i8(a, w, sa, sw, out_dtype=torch.float32)
    assert same(got, sums(a, w).float() * sa[:, None] * sw[None, :])
    assert torch.isnan(got[1]).all() and not torch.isnan(got[0, :5]).any()
    assert same(tcr.tcr_gemm_i8(a, w, scale_w=sw, out_dtype=torch.float32), sums(a, w).float() * sw[None, :])


def test_a_token_does_not_depend_on_the_others(gen):
    a, w = codes(gen, 500, 2000), codes(gen, 999, 2000)
    sa, sw = torch.rand(500, generator=gen, device="cuda"), torch.rand(999, generator=gen, device="cuda")
    c = tcr.tcr_gemm_i8(a, w, sa, sw)
    for at in (slice(0, 1), slice(250, 255), slice(480, 500)):
        assert same(c[at], tcr.tcr_gemm_i8(a[at], w, sa[at], sw))


def test_streams_and_graphs(gen):
    a, w = codes(gen, 48, 4096), codes(gen, 1024, 4096)
    want = tcr.tcr_gemm_i8(a, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tcr.tcr_gemm_i8(a, w, stream=s)
    one = tcr.tcr_gemm_i8(a[:1], w, stream=s)
    s.synchronize()
    assert same(want, got) and same(want[:1], one)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tcr.tcr_gemm_i8(a, w, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert same(want, out)


def test_refusals(gen, monkeypatch):
    a, w = codes(gen, 12, 64), codes(gen, 20, 64)
    with pytest.raises(ValueError):
        tcr.tcr_gemm_i8(a, w[:, :63])
    with pytest.raises(ValueError):
        tcr.tcr_gemm_i8(a.cpu(), w)
    with pytest.raises(TypeError):
        tcr.tcr_gemm_i8(a.int(), w)
    with pytest.raises(TypeError):
        tcr.tcr_gemm_i8(a, w, out_dtype=torch.int16)
    with pytest.raises(ValueError):
        tcr.tcr_gemm_i8(a, w, torch.ones(12, device="cuda"), out_dtype=torch.int32)
    with pytest.raises(ValueError):
        tcr.tcr_gemm_i8(a, w, torch.ones(11, device="cuda"))
    with pytest.raises(TypeError):
        tcr.tcr_gemm_i8(a, w, torch.ones(12, device="cuda").double())
    with pytest.raises(ValueError):
        tcr.tcr_gemm_i8(a[:1].expand(12, 64), w)
    with pytest.raises(tcr.TcrError) as e:
        tcr.tcr_gemm_i8(torch.zeros(1, 131072, dtype=torch.int8, device="cuda"),
                        torch.zeros(1, 131072, dtype=torch.int8, device="cuda"))
    assert e.value.status == tcr.ERR_UNSUPPORTED
    a = codes(gen, 1100, 64)                              # enough tokens for scratch
    out = torch.full((1100, 20), 5.0, device="cuda")
    for what in ("alloc", "launch"):
        monkeypatch.setenv("TCR_FAULT_INJECT", what)
        with pytest.raises(tcr.TcrError):
            tcr.tcr_gemm_i8(a, w, out=out)
    monkeypatch.delenv("TCR_FAULT_INJECT")
    assert (out == 5).all()
