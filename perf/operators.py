"""What the 8-bit inference path and the norm's training pass are measured on.

Operators of one transformer linear path, chained as a model chains them:

  norm    h = x + residual, y = weight * h / sqrt(mean(h^2) + eps) by rows; y in the
          inputs' type, or in 8-bit integers with one scale a row (token)
  back    the norm's gradient: dx by rows and the weight's gradient summed over rows
  gated   silu(gate) * up by rows into 8-bit integers with one scale a row, gate and up
          being the two halves of one product's output
  gemm    C = (A W^T) * scale of the token * scale of the channel, A and W in 8-bit
          integers, their products summed exactly

A case is a dict of plain values; `prepare` makes its inputs from the seed alone, `run`
is one pass (elementary torch operations in 32 bits where `own` is false, the library's
calls where it is true), `exact` the definition in 64 bits, `work` what a pass cannot
do without.  8-bit outputs are read back into 16 bits, so a pass of those operators is
the quantising call and the call that reads the codes back.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # a decoding step of four sequences: the launch and one row's latency
        {"name": "norm i8 4x4096", "op": "norm", "rows": 4, "cols": 4096, "dtype": "bf16", "i8": True, "pad": 0},
        # a long prompt batch at the width of the row-reduction workload
        {"name": "norm i8 65536x4096", "op": "norm", "rows": 65536, "cols": 4096, "dtype": "f16", "i8": True, "pad": 0},
        # a training forward: 16-bit output, an odd width, rows that are slices of wider ones
        {"name": "norm 6151x5001 padded", "op": "norm", "rows": 6151, "cols": 5001, "dtype": "bf16", "i8": False, "pad": 7},
        # a training step's backward of one norm
        {"name": "back 16384x4096", "op": "back", "rows": 16384, "cols": 4096, "dtype": "bf16"},
        # the same in binary32 with ragged sizes
        {"name": "back 1001x1537 f32", "op": "back", "rows": 1001, "cols": 1537, "dtype": "f32"},
        # a decoding step's gated activation
        {"name": "gated 8x8192", "op": "gated", "rows": 8, "cols": 8192, "dtype": "bf16"},
        # a prompt batch's gated activation
        {"name": "gated 16384x8192", "op": "gated", "rows": 16384, "cols": 8192, "dtype": "bf16"},
        # one token through a projection: the weights are read once
        {"name": "gemm 1x4096x4096", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "out": "bf16"},
        # a decoding batch through a wide projection
        {"name": "gemm 48x8192x8192", "op": "gemm", "m": 48, "n": 8192, "k": 8192, "out": "bf16"},
        # ragged sizes, a row pitch that no wide load fits
        {"name": "gemm 333x2051x4100", "op": "gemm", "m": 333, "n": 2051, "k": 4100, "out": "f32"},
        # a short prompt
        {"name": "gemm 2048x4096x4096", "op": "gemm", "m": 2048, "n": 4096, "k": 4096, "out": "f16"},
        # a prompt batch: bound by the tensor cores
        {"name": "gemm 8192x8192x8192", "op": "gemm", "m": 8192, "n": 8192, "k": 8192, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """A size spread over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, unit, share):
    """The same, a multiple of `unit` for that share of the draws."""
    v = _log(rng, lo, hi)
    if rng.random() < share:
        v = max(lo, v // unit * unit)
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "back", "gated", "gemm", "gemm"])
    if op == "gemm":
        m, n = _size(rng, 1, 8192, 1, 1), _size(rng, 256, 8192, 64, 0.5)
        k = _size(rng, 64, 8192, 16, 0.7)      # most weights have a pitch of whole 16-byte words
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "f16", "f32"])}
    cols = _size(rng, 128, 16384, 64, 0.6)
    dtype = rng.choice(["bf16", "f16", "f32"])
    rows = _size(rng, 1, min(65536, (1 << 26) // cols), 1, 1)
    if op == "norm":
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "i8": rng.random() < 0.6,
                "pad": rng.choice([0, 0, 8, 5])}
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype}


def _acts(gen, rows, cols, dtype, last_zero, pitch=None):
    """Hidden states: normal values, a few channels far larger than the rest, and
    a padding token (a row of zeros) at the end of batches."""
    base = torch.empty(rows, pitch or cols, dtype=dtype, device="cuda").normal_(generator=gen)
    x = base[:, :cols]
    loud = torch.randint(0, cols, (max(1, cols // 512),), generator=gen, device="cuda")
    x[:, loud] = x[:, loud] * 12
    if last_zero and rows > 2:
        x[-1] = 0
    return x


def _codes(gen, rows, cols):
    """Symmetric 8-bit codes as the row quantiser leaves them."""
    q = torch.empty(rows, cols, dtype=torch.float16, device="cuda").normal_(0.0, 30.0, generator=gen)
    q.round_().clamp_(-127, 127)
    q[:, 0] = 127
    return q.to(torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = dict(case)
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"], st["w"] = _codes(gen, m, k), _codes(gen, n, k)
        st["sa"] = torch.rand(m, generator=gen, device="cuda") * 0.05 + 0.01
        st["sw"] = torch.rand(n, generator=gen, device="cuda") * 1e-3 + 1e-4
        st["c"] = torch.empty(m, n, dtype=DT[case["out"]], device="cuda")
        return st
    rows, cols, dt = case["rows"], case["cols"], DT[case["dtype"]]
    back16 = torch.bfloat16 if dt == torch.float32 else dt      # the type codes are read back into
    if op == "norm":
        pitch = cols + case["pad"]
        st["x"] = _acts(gen, rows, cols, dt, True, pitch)
        st["r"] = _acts(gen, rows, cols, dt, True, pitch)
        st["w"] = (torch.rand(cols, generator=gen, device="cuda") + 0.5).to(dt)
        st["h"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        st["y"] = torch.empty(rows, cols, dtype=back16 if case["i8"] else dt, device="cuda")
    elif op == "back":
        st["h"] = _acts(gen, rows, cols, dt, True)
        st["dy"] = torch.empty(rows, cols, dtype=dt, device="cuda").normal_(0.0, 0.1, generator=gen)
        st["dh"] = torch.empty(rows, cols, dtype=dt, device="cuda").normal_(0.0, 0.1, generator=gen)
        st["w"] = (torch.rand(cols, generator=gen, device="cuda") + 0.5).to(dt)
        # saved by the forward pass
        st["rstd"] = torch.rsqrt(torch.linalg.vector_norm(st["h"], dim=1, dtype=torch.float32) ** 2 / cols + EPS)
        st["dx"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        st["dw"] = torch.empty(cols, dtype=torch.float32, device="cuda")
    else:
        both = torch.empty(rows, 2 * cols, dtype=dt, device="cuda").normal_(0.0, 2.0, generator=gen)
        if rows > 2:
            both[-1] = 0
        st["gate"], st["up"] = both[:, :cols], both[:, cols:]
        st["y"] = torch.empty(rows, cols, dtype=back16, device="cuda")
    st["q"] = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    st["scale"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    return st


def _round_i8(y):
    """(values that the 8-bit codes stand for, scale of each row)"""
    scale = y.abs().amax(1) / 127
    per = torch.where(scale > 0, 1 / scale, 0)[:, None]
    return torch.round(y * per) * scale[:, None], scale


def run(st):
    op = st["op"]
    if own:
        import arithmetic_reduction_tensor_gb300 as tcr
        if op == "gemm":
            return tcr.tcr_gemm_i8(st["a"], st["w"], st["sa"], st["sw"], out=st["c"])
        if op == "back":
            dx, dw = tcr.tcr_rmsnorm_backward(st["dy"], st["h"], st["w"], st["rstd"], dh=st["dh"],
                                              dx=st["dx"], dweight=st["dw"])
            return {"dx": dx, "dw": dw}
        if op == "norm" and not st["i8"]:
            r = tcr.tcr_rmsnorm(st["x"], st["w"], residual=st["r"], eps=EPS, h=st["h"], out=st["y"])
            return {"h": r.h, "y": r.y}
        if op == "norm":
            r = tcr.tcr_rmsnorm(st["x"], st["w"], residual=st["r"], eps=EPS, h=st["h"], out=st["q"],
                                scale=st["scale"])
            return {"h": r.h, "y": tcr.tcr_dequantize_rows_i8(r.y, r.scale, out=st["y"]), "scale": r.scale}
        q, scale = tcr.tcr_quantize_rows_i8(st["up"], gate=st["gate"], out=st["q"], scale=st["scale"])
        return {"y": tcr.tcr_dequantize_rows_i8(q, scale, out=st["y"]), "scale": scale}
    if op == "gemm":
        acc = st["a"].float() @ st["w"].float().t()
        return (acc * st["sa"][:, None] * st["sw"][None, :]).to(DT[st["out"]])
    if op == "back":
        h, dy, rstd = st["h"].float(), st["dy"].float(), st["rstd"][:, None]
        xhat = h * rstd
        g = dy * st["w"].float()
        dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)) + st["dh"].float()
        return {"dx": dx.to(st["h"].dtype), "dw": (dy * xhat).sum(0)}
    if op == "norm":
        h = st["x"].float() + st["r"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["w"].float()
        out = {"h": h.to(st["h"].dtype)}
    else:
        g = st["gate"].float()
        y = g / (1 + torch.exp(-g)) * st["up"].float()
        out = {}
    if op == "gated" or st["i8"]:
        y, out["scale"] = _round_i8(y)
    out["y"] = y.to(st["y"].dtype)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = lambda t: t.to(torch.float64)      # noqa: E731
    if op == "gemm":
        parts = []                           # some columns of C at a time: float64 copies are large
        a = f64(st["a"])
        for j in range(0, case["n"], 2048):
            parts.append(a @ f64(st["w"][j:j + 2048]).T)
        return torch.cat(parts, 1) * torch.outer(f64(st["sa"]), f64(st["sw"]))
    rows, cols = case["rows"], case["cols"]
    step = max(1, (1 << 25) // cols)         # some rows at a time, for the same reason
    got = []
    dw = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, step):
        at = slice(i, i + step)
        if op == "back":
            h, dy, rs = f64(st["h"][at]), f64(st["dy"][at]), f64(st["rstd"][at])
            w = f64(st["w"])
            inner = torch.einsum("rc,rc,c->r", dy, h, w)
            dx = torch.einsum("rc,c,r->rc", dy, w, rs)
            dx -= torch.einsum("rc,r->rc", h, inner * rs ** 3 / cols)
            dw += torch.einsum("rc,rc,r->c", dy, h, rs)
            got.append({"dx": dx + f64(st["dh"][at])})
            continue
        d = {}
        if op == "norm":
            d["h"] = f64(st["x"][at]) + f64(st["r"][at])
            ms = torch.einsum("rc,rc->r", d["h"], d["h"]) / cols + EPS
            y = torch.einsum("rc,c,r->rc", d["h"], f64(st["w"]), ms ** -0.5)
        else:
            y = f64(st["gate"][at]) * torch.sigmoid(f64(st["gate"][at])) * f64(st["up"][at])
        if op == "gated" or case["i8"]:
            d["scale"] = torch.linalg.vector_norm(y, ord=float("inf"), dim=1) / 127
            unit = torch.where(d["scale"] == 0, 1.0, d["scale"])[:, None]
            y = torch.round(y / unit) * unit
        d["y"] = y
        got.append(d)
    out = {key: torch.cat([d[key] for d in got]) for key in got[0]}
    if op == "back":
        out["dw"] = dw
    return out


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * BYTES[case["out"]], "flops": 2.0 * m * n * k}
    rows, cols, b = case["rows"], case["cols"], BYTES[case["dtype"]]
    size = rows * cols
    if op == "back":            # dy, h, dh read, dx written; the weight, its gradient, one number a row
        return {"bytes": 4 * size * b + cols * (b + 4) + 4 * rows, "flops": 12.0 * size}
    if op == "norm":            # x and the residual read, h and y written (codes read back: 16 bits)
        y = 2 if case["i8"] else b
        return {"bytes": size * (3 * b + y) + cols * b + (4 * rows if case["i8"] else 0), "flops": 8.0 * size}
    return {"bytes": size * (2 * b + 2) + 4 * rows, "flops": 10.0 * size}
