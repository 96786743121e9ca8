"""What dropout, the layer norm's training pass and the loss over a vocabulary are measured on.

Operators of one training step beside the norm and products that the library has:

  dropout  y = residual + dropout(x); the mask comes from a counter-based generator
           (Philox4x32-10) and is never stored.  Counter: vector of 8 columns, row,
           the call's 64-bit offset; key: the 64-bit seed; 16 bits an element, which
           is kept where they are at least t = rint(65536 p), times 65536 / (65536 - t)
  layer    h = residual + dropout(x), y = weight * (h - mean) * rstd + bias by rows; y in
           the inputs' type, or in 8-bit integers with one scale a row (token)
  back     the layer norm's gradient: that of x (through the dropout), of the residual,
           and the weight's and the bias' summed over rows
  loss     softmax cross entropy of x W^T against one target a token, the logits not kept;
           tokens whose target is -100 count for nothing; with the logarithm of each
           token's sum of exponentials, which the gradient takes
  step     the same and its gradient of x and of W

A case is a dict of plain values; `prepare` makes its inputs from the seed alone, `run`
is one pass (elementary torch operations in 32 bits where `own` is false, the library's
calls where it is true), `exact` the definition in 64 bits, `work` what a pass cannot
do without.  8-bit outputs are read back into 16 bits, so such a pass is the
norm's call and the call that reads the codes back.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5
IGNORED = -100


def listed():
    return [
        # one token a sequence of a small batch: the launch alone
        {"name": "dropout 8x1000", "op": "dropout", "rows": 8, "cols": 1000, "dtype": "f32", "p": 0.1, "add": False, "pad": 3},
        # a block's output onto the residual, a large batch
        {"name": "dropout 65536x4096", "op": "dropout", "rows": 65536, "cols": 4096, "dtype": "f16", "p": 0.1, "add": True, "pad": 0},
        # a decoding step of four sequences, codes for the next product
        {"name": "layer i8 4x4096", "op": "layer", "rows": 4, "cols": 4096, "dtype": "bf16", "i8": True, "p": 0.0, "pad": 0},
        # a training forward of one block
        {"name": "layer 16384x4096", "op": "layer", "rows": 16384, "cols": 4096, "dtype": "bf16", "i8": False, "p": 0.1, "pad": 0},
        # an odd width, rows that are slices of wider ones
        {"name": "layer 6151x5001 padded", "op": "layer", "rows": 6151, "cols": 5001, "dtype": "bf16", "i8": False, "p": 0.0, "pad": 7},
        # its backward
        {"name": "back 16384x4096", "op": "back", "rows": 16384, "cols": 4096, "dtype": "bf16", "p": 0.1},
        # the same in binary32 with ragged sizes
        {"name": "back 1001x1537 f32", "op": "back", "rows": 1001, "cols": 1537, "dtype": "f32", "p": 0.0},
        # scoring a few tokens: the vocabulary's matrix is read once
        {"name": "loss 16x4096 of 131072", "op": "loss", "tokens": 16, "hidden": 4096, "vocab": 131072, "dtype": "bf16", "ignored": 0.0},
        # scoring a batch of text
        {"name": "loss 4096x4096 of 65536", "op": "loss", "tokens": 4096, "hidden": 4096, "vocab": 65536, "dtype": "bf16", "ignored": 0.0},
        # a small model's step: ragged sizes, rows that no wide load fits
        {"name": "step 333x1001 of 5003", "op": "step", "tokens": 333, "hidden": 1001, "vocab": 5003, "dtype": "f16", "ignored": 0.2},
        # a training step of one micro-batch
        {"name": "step 4096x4096 of 32768", "op": "step", "tokens": 4096, "hidden": 4096, "vocab": 32768, "dtype": "bf16", "ignored": 0.0},
        # a tuning step: the prompts' tokens, a third of them, are not learnt
        {"name": "step 8192x4096 of 65536", "op": "step", "tokens": 8192, "hidden": 4096, "vocab": 65536, "dtype": "bf16", "ignored": 0.34},
    ]


def _log(rng, lo, hi):
    """A size spread over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, unit, share):
    """The same, a multiple of `unit` for that share of the draws."""
    v = _log(rng, lo, hi)
    if rng.random() < share:
        v = max(lo, v // unit * unit)
    return v


def draw(rng):
    op = rng.choice(["dropout", "layer", "back", "loss", "step", "step"])
    if op in ("loss", "step"):
        hidden, vocab = _size(rng, 64, 8192, 64, 0.7), _size(rng, 256, 131072, 64, 0.6)
        most = 8192 * 65536 * 4096 // (hidden * vocab)
        return {"op": op, "tokens": _log(rng, 1, min(8192, most)), "hidden": hidden, "vocab": vocab,
                "dtype": rng.choice(["bf16", "bf16", "f16"]), "ignored": rng.choice([0.0, 0.0, 0.1, 0.5])}
    cols = _size(rng, 128, 16384, 64, 0.6)
    dtype = rng.choice(["bf16", "f16", "f32"])
    case = {"op": op, "rows": _log(rng, 1, min(65536, (1 << 26) // cols)), "cols": cols, "dtype": dtype}
    if op == "dropout":
        case.update(p=rng.choice([0.1, 0.25, 0.5]), add=rng.random() < 0.7, pad=rng.choice([0, 0, 8, 5]))
    elif op == "layer":
        case.update(p=rng.choice([0.0, 0.0, 0.1]), i8=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 5]))
    else:
        case.update(p=rng.choice([0.0, 0.1]))
    return case


def _acts(gen, rows, cols, dtype, pitch=None):
    """Hidden states: normal values with a mean, a few channels far larger than
    the rest."""
    base = torch.empty(rows, pitch or cols, dtype=dtype, device="cuda").normal_(0.25, 1.0, generator=gen)
    x = base[:, :cols]
    loud = torch.randint(0, cols, (max(1, cols // 512),), generator=gen, device="cuda")
    x[:, loud] = x[:, loud] * 12
    return x


def _prepare_loss(case, gen, st):
    t, h, v, dt = case["tokens"], case["hidden"], case["vocab"], DT[case["dtype"]]
    st["x"] = torch.empty(t, h, dtype=dt, device="cuda").normal_(generator=gen)
    # logits of a few units; low ids are the frequent ones
    st["w"] = torch.empty(v, h, dtype=dt, device="cuda").normal_(0.0, 2.0 / math.sqrt(h), generator=gen)
    u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    st["target"] = (v * u ** 3).long().clamp_(0, v - 1)
    if case["ignored"]:
        st["target"][torch.rand(t, generator=gen, device="cuda") < case["ignored"]] = IGNORED
    count = (st["target"] != IGNORED).sum().clamp(min=1)
    st["dloss"] = (1.0 / count.float()).expand(t)        # of the mean over the tokens that count
    st["loss"] = torch.empty(t, device="cuda")
    st["lse"] = torch.empty(t, device="cuda")
    if case["op"] == "step":
        st["dx"], st["dw"] = torch.empty_like(st["x"]), torch.empty_like(st["w"])
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = dict(case)
    op = case["op"]
    if op in ("loss", "step"):
        return _prepare_loss(case, gen, st)
    rows, cols, dt = case["rows"], case["cols"], DT[case["dtype"]]
    st["seed"], st["offset"] = (0x9E3779B97F4A7C15 ^ int(seed)) & (1 << 64) - 1, (int(seed) + 1 << 20) & (1 << 64) - 1
    if op == "back":
        st["h"] = _acts(gen, rows, cols, dt)
        st["dy"] = torch.empty(rows, cols, dtype=dt, device="cuda").normal_(0.0, 0.1, generator=gen)
        st["dh"] = torch.empty(rows, cols, dtype=dt, device="cuda").normal_(0.0, 0.1, generator=gen)
        st["w"] = (torch.rand(cols, generator=gen, device="cuda") + 0.5).to(dt)
        # saved by the forward pass
        st["mean"] = torch.mean(st["h"], 1, dtype=torch.float32)
        var = torch.linalg.vector_norm(st["h"], dim=1, dtype=torch.float32) ** 2 / cols - st["mean"] ** 2
        st["rstd"] = torch.rsqrt(var + EPS)
        st["dx"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        st["dr"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        st["dw"], st["db"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        return st
    pitch = cols + case["pad"]
    st["x"] = _acts(gen, rows, cols, dt, pitch)
    if op == "dropout":
        st["r"] = _acts(gen, rows, cols, dt, pitch) if case["add"] else None
        st["y"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        return st
    back16 = torch.bfloat16 if dt == torch.float32 else dt      # the type codes are read back into
    st["r"] = _acts(gen, rows, cols, dt, pitch)
    st["w"] = (torch.rand(cols, generator=gen, device="cuda") + 0.5).to(dt)
    st["b"] = torch.empty(cols, dtype=dt, device="cuda").normal_(0.0, 0.5, generator=gen)
    st["h"] = torch.empty(rows, cols, dtype=dt, device="cuda")
    st["y"] = torch.empty(rows, cols, dtype=back16 if case["i8"] else dt, device="cuda")
    st["mean"], st["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    st["q"] = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    st["scale"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    return st


LOW = 0xFFFFFFFF


def _philox_bits(rows, cols, seed, offset, device):
    """The 16 bits of each element."""
    nvec = (cols + 7) // 8
    c = [torch.arange(nvec, device=device).expand(rows, nvec),
         torch.arange(rows, device=device)[:, None].expand(rows, nvec),
         torch.tensor(offset & LOW, device=device).expand(rows, nvec),
         torch.tensor(offset >> 32 & LOW, device=device).expand(rows, nvec)]
    k0, k1 = seed & LOW, seed >> 32 & LOW
    for _ in range(10):             # the generator's rounds; products wrap at 64 bits
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & LOW) ^ c[1] ^ k0, b & LOW, (a >> 32 & LOW) ^ c[3] ^ k1, a & LOW]
        k0, k1 = k0 + 0x9E3779B9 & LOW, k1 + 0xBB67AE85 & LOW
    words = torch.stack(c, 2)
    return torch.stack([words & 0xFFFF, words >> 16], 3).view(rows, nvec * 8)[:, :cols]


def _dropped(x, st):
    """dropout(x) in 32 bits; x where p is 0."""
    t = round(65536 * st["p"])
    if t == 0:
        return x
    keep = _philox_bits(x.shape[0], x.shape[1], st["seed"], st["offset"], x.device) >= t
    return torch.where(keep, x * (65536 / (65536 - t)), 0.0)


def _round_i8(y):
    """(values that the 8-bit codes stand for, scale of each row)"""
    scale = y.abs().amax(1) / 127
    per = torch.where(scale > 0, 1 / scale, 0)[:, None]
    return torch.round(y * per) * scale[:, None], scale


def _plain_loss(st):
    x, w, target = st["x"].float(), st["w"].float(), st["target"]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(1))
    live = target != IGNORED
    at = target.clamp(min=0)[:, None]
    loss = torch.where(live, lse - logits.gather(1, at)[:, 0], 0.0)
    if st["op"] == "loss":
        return {"loss": loss, "lse": torch.where(live, lse, 0.0)}
    p = torch.exp(logits - lse[:, None])
    p.scatter_add_(1, at, torch.full(at.shape, -1.0, device=x.device))
    p *= torch.where(live, st["dloss"], 0.0)[:, None]
    return {"loss": loss, "dx": (p @ w).to(st["x"].dtype), "dw": (p.t() @ x).to(st["w"].dtype)}


def _own(st):
    import arithmetic_reduction_tensor_gb300 as tcr
    op = st["op"]
    if op in ("loss", "step"):
        o = tcr.tcr_cross_entropy(st["x"], st["w"], st["target"], ignore_index=IGNORED, loss=st["loss"], lse=st["lse"])
        if op == "loss":
            return {"loss": o.loss, "lse": o.lse}
        dx, dw = tcr.tcr_cross_entropy_backward(st["dloss"], st["x"], st["w"], st["target"], o.lse,
                                                ignore_index=IGNORED, dx=st["dx"], dweight=st["dw"])
        return {"loss": o.loss, "dx": dx, "dw": dw}
    drop = {"p": st["p"], "seed": st["seed"], "offset": st["offset"]}
    if op == "dropout":
        return tcr.tcr_dropout(st["x"], **drop, residual=st["r"], out=st["y"])
    if op == "back":
        g = tcr.tcr_layernorm_backward(st["dy"], st["h"], st["w"], st["mean"], st["rstd"], dh=st["dh"], **drop,
                                       dx=st["dx"], dresidual=st["dr"] if st["p"] else None, dweight=st["dw"],
                                       dbias=st["db"])
        out = {"dx": g.dx, "dw": g.dweight, "db": g.dbias}
        return {**out, "dr": g.dresidual} if st["p"] else out
    if st["i8"]:
        o = tcr.tcr_layernorm(st["x"], st["w"], st["b"], residual=st["r"], eps=EPS, **drop, h=st["h"], out=st["q"],
                              scale=st["scale"])
        return {"h": o.h, "y": tcr.tcr_dequantize_rows_i8(o.y, o.scale, out=st["y"]), "scale": o.scale}
    o = tcr.tcr_layernorm(st["x"], st["w"], st["b"], residual=st["r"], eps=EPS, **drop, h=st["h"], out=st["y"],
                          mean=st["mean"], rstd=st["rstd"])
    return {"h": o.h, "y": o.y, "mean": o.mean, "rstd": o.rstd}


def run(st):
    if own:
        return _own(st)
    op = st["op"]
    if op in ("loss", "step"):
        return _plain_loss(st)
    if op == "dropout":
        y = _dropped(st["x"].float(), st)
        return (y if st["r"] is None else st["r"].float() + y).to(st["y"].dtype)
    if op == "back":
        h, dy, rstd = st["h"].float(), st["dy"].float(), st["rstd"][:, None]
        xhat = (h - st["mean"][:, None]) * rstd
        g = dy * st["w"].float()
        dr = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) + st["dh"].float()
        out = {"dx": _dropped(dr, st).to(st["h"].dtype),
               "dw": (dy * xhat).sum(0), "db": dy.sum(0)}
        return {**out, "dr": dr.to(st["h"].dtype)} if st["p"] else out
    h = st["r"].float() + _dropped(st["x"].float(), st)
    mean = h.mean(1, keepdim=True)
    rstd = torch.rsqrt(((h - mean) * (h - mean)).mean(1, keepdim=True) + EPS)
    y = (h - mean) * rstd * st["w"].float() + st["b"].float()
    out = {"h": h.to(st["h"].dtype)}
    if st["i8"]:
        y, out["scale"] = _round_i8(y)
    else:
        out["mean"], out["rstd"] = mean[:, 0], rstd[:, 0]
    out["y"] = y.to(st["y"].dtype)
    return out


def _exact_keep(st, first, rows, cols):
    """The kept elements times their factor, from the generator computed in
    numpy's unsigned 64-bit integers."""
    import numpy as np
    t = round(65536 * st["p"])
    v = np.arange((cols + 7) // 8, dtype=np.uint64)[None, :]
    r = np.arange(first, first + rows, dtype=np.uint64)[:, None]
    low, half = np.uint64(LOW), np.uint64(32)
    x0, x1 = np.broadcast_arrays(v, r)
    x2 = np.full(x0.shape, st["offset"] & LOW, dtype=np.uint64)
    x3 = np.full(x0.shape, st["offset"] >> 32 & LOW, dtype=np.uint64)
    for i in range(10):
        k0 = np.uint64((st["seed"] & LOW) + i * 0x9E3779B9 & LOW)
        k1 = np.uint64((st["seed"] >> 32 & LOW) + i * 0xBB67AE85 & LOW)
        p0, p1 = np.uint64(0xD2511F53) * x0, np.uint64(0xCD9E8D57) * x2
        x0, x1, x2, x3 = (p1 >> half) ^ x1 ^ k0, p1 & low, (p0 >> half) ^ x3 ^ k1, p0 & low
    bits = np.stack([x0, x1, x2, x3], 2).astype("<u4").view("<u2").reshape(rows, -1)[:, :cols]
    return torch.from_numpy((bits >= t).astype(np.float64)).cuda() * (65536.0 / (65536 - t))


def _exact_loss(case, st):
    x, target = st["x"].double(), st["target"]
    t, v, step = case["tokens"], case["vocab"], 8192
    live = target >= 0
    lse = torch.full((t,), -math.inf, dtype=torch.float64, device="cuda")
    for j in range(0, v, step):                      # some of the vocabulary at a time: float64 is large
        lse = torch.logaddexp(lse, torch.logsumexp(torch.einsum("th,vh->tv", x, st["w"][j:j + step].double()), 1))
    hit = torch.einsum("th,th->t", x, st["w"][target.clamp(min=0)].double())
    out = {"loss": torch.where(live, lse - hit, 0)}
    if case["op"] == "loss":
        return {**out, "lse": torch.where(live, lse, 0)}
    g = torch.where(live, st["dloss"].double(), 0)
    dx, dw = torch.zeros_like(x), []
    for j in range(0, v, step):
        w = st["w"][j:j + step].double()
        p = torch.einsum("th,vh->tv", x, w).sub_(lse[:, None]).exp_()
        p = (p - torch.nn.functional.one_hot((target - j).clamp(-1, len(w)) + 1, len(w) + 2)[:, 1:-1]) * g[:, None]
        dx += torch.einsum("tv,vh->th", p, w)
        dw.append(torch.einsum("tv,th->vh", p, x))
        del p, w
    out["dx"], out["dw"] = dx, torch.cat(dw)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("loss", "step"):
        return _exact_loss(case, st)
    rows, cols = case["rows"], case["cols"]
    step = max(1, (1 << 24) // cols)
    got = []
    dw = torch.zeros(2, cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, step):
        f64 = lambda name: st[name][i:i + step].double()      # noqa: E731
        n = min(step, rows - i)
        keep = _exact_keep(st, i, n, cols) if case["p"] else 1.0
        if op == "dropout":
            y = f64("x") * keep
            got.append({"": y if st["r"] is None else y + f64("r")})
            continue
        w = st["w"].double()
        if op == "back":
            dy, rs = f64("dy"), f64("rstd")
            xhat = torch.einsum("rc,r->rc", f64("h") - f64("mean")[:, None], rs)
            a = torch.einsum("rc,c->r", dy, w) / cols
            b = torch.einsum("rc,c,rc->r", dy, w, xhat) / cols
            dr = (dy * w - a[:, None] - torch.einsum("rc,r->rc", xhat, b)) * rs[:, None] + f64("dh")
            dw[0] += torch.einsum("rc,rc->c", dy, xhat)
            dw[1] += dy.sum(0)
            got.append({"dx": dr * keep, "dr": dr} if case["p"] else {"dx": dr})
            continue
        h = f64("r") + f64("x") * keep
        var, mean = torch.var_mean(h, 1, unbiased=False)
        d = {"h": h}
        y = torch.addcmul(st["b"].double(), (h - mean[:, None]) / torch.sqrt(var + EPS)[:, None], w)
        if case["i8"]:
            d["scale"] = torch.linalg.vector_norm(y, ord=float("inf"), dim=1) / 127
            unit = torch.where(d["scale"] == 0, 1.0, d["scale"])[:, None]
            y = torch.round(y / unit) * unit
        else:
            d["mean"], d["rstd"] = mean, (var + EPS) ** -0.5
        d["y"] = y
        got.append(d)
    out = {key: torch.cat([d[key] for d in got]) for key in got[0]}
    if op == "back":
        out["dw"], out["db"] = dw[0], dw[1]
    return out[""] if op == "dropout" else out


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op in ("loss", "step"):
        h, v = case["hidden"], case["vocab"]
        t = max(1, round(case["tokens"] * (1 - case["ignored"])))      # those that count
        # x and the matrix read; a step writes a gradient of each, and forms two more products
        size = (t + v) * h * b
        return {"bytes": size * (2 if op == "step" else 1) + 16 * case["tokens"],
                "flops": 2.0 * t * h * v * (3 if op == "step" else 1)}
    rows, cols = case["rows"], case["cols"]
    size = rows * cols
    if op == "dropout":
        return {"bytes": size * b * (3 if case["add"] else 2), "flops": 2.0 * size}
    if op == "layer":               # x and the residual read, h and y written (codes read back: 16 bits)
        y = 2 if case["i8"] else b
        return {"bytes": size * (3 * b + y) + 2 * cols * b + 8 * rows, "flops": 10.0 * size}
    # dy, h, dh read, dx (and the residual's) written; the weight, two gradients, two numbers a row
    return {"bytes": (5 if case["p"] else 4) * size * b + cols * (b + 8) + 8 * rows, "flops": 16.0 * size}
