"""The 8-bit operators together: a stack of residual MLP blocks and the
norm's training step (examples/w8a8_mlp.py), and the product's failure path."""
import importlib.util
import os
import threading
import time

import pytest

import arithmetic_reduction_tensor_gb300 as tcr
from arithmetic_reduction_tensor_gb300.build import build_library

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    torch.cuda.set_device(0)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("w8a8_mlp", os.path.join(root, "examples", "w8a8_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("width,hidden,tokens", [(256, 512, 70), (200, 328, 33), (512, 1024, 1200)])
def test_stack_of_blocks(example, width, hidden, tokens):
    gen = torch.Generator(device="cuda").manual_seed(3)
    blocks = [example.Block(width, hidden, gen) for _ in range(3)]
    x = torch.randn(tokens, width, generator=gen, device="cuda").to(torch.bfloat16)
    y, want = example.forward(blocks, x), example.reference(blocks, x)
    # Four quantisers a block (two of activations, two of weights), each with
    # a step of amax / 127: for normal values amax is about 4 sigma, so an
    # error of 4 / 127 / sqrt(12) = 0.9% of sigma each, four of them 1.8%, and
    # 0.3% of bfloat16; three blocks' outputs against a residual stream that
    # holds them: below 4%.
    assert ((y.float() - want).norm() / want.norm()).item() < 0.04
    # a token alone, captured, gives the prompt's bits
    one, out, step = example.decoder(blocks, width)
    for i in (0, tokens - 1):
        one.copy_(x[i:i + 1])
        step()
        assert torch.equal(out, y[i:i + 1])


def test_norm_weight_is_fitted(example):
    losses = example.train_norm()
    assert losses[-1] < 1e-3 * losses[0]


@pytest.mark.parametrize("M,N,K", [(1100, 300, 2000), (1100, 300, 500), (3000, 2560, 1500)])
def test_a_wait_that_runs_out_reports_and_recovers(example, monkeypatch, M, N, K):
    # the MMA issuer withholds each pair's first sums: the epilogue's wait
    # gives up after about a second, on split tiles, single chunks and whole
    # tiles of several chunks
    gen = torch.Generator(device="cuda").manual_seed(4)
    a = torch.randint(-128, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    want = (a.double() @ w.double().t()).to(torch.int32)
    torch.cuda.synchronize()
    tcr.tcr_device_faults(clear=True)
    monkeypatch.setenv("TCR_FAULT_INJECT", "stall")
    t0 = time.time()
    c = tcr.tcr_gemm_i8(a, w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    monkeypatch.delenv("TCR_FAULT_INJECT")
    assert torch.isnan(c).all()
    assert tcr.tcr_device_faults(clear=True) & tcr.FAULT_PIPELINE_WAIT
    assert elapsed < 20
    assert torch.equal(tcr.tcr_gemm_i8(a, w, out_dtype=torch.int32), want)
    torch.cuda.synchronize()
    assert tcr.tcr_device_faults() == 0


def test_threads_on_their_own_streams(example):
    # the calls leave the interpreter to each other: first uses, scratch and
    # launches of several threads at once give what one thread's give
    gen = torch.Generator(device="cuda").manual_seed(9)
    blocks = [example.Block(256, 640, gen) for _ in range(2)]
    xs = [torch.randn(rows, 256, generator=gen, device="cuda").to(torch.bfloat16) for rows in (1, 7, 60, 300, 1100, 2100)]

    def step(x):
        y = example.forward(blocks, x)
        o = tcr.tcr_rmsnorm(x, blocks[0].norm, residual=y, want_rstd=True)
        return (y, *tcr.tcr_rmsnorm_backward(y, o.h, blocks[0].norm, o.rstd))
    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(25):
                    got = step(xs[k])
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                wrong.append(f"thread {k}: other results")
        except Exception as e:        # reported below
            wrong.append(f"thread {k}: {e!r}")
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    torch.cuda.synchronize()
    assert tcr.tcr_device_faults() == 0
