"""Dropout's generator, the layer norm and its gradient restated on the CPU,
operation for operation in binary32, and in binary64 from their definitions;
the cross entropy in binary64."""
import numpy as np
import torch

from tests.rows_spec import F32, row_sums


def philox(c, k):
    """Philox4x32-10 of counters c (..., 4) and a key of two words (Salmon et
    al., 2011), in 64-bit unsigned integers."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [np.asarray(c[..., i], dtype=np.uint64) for i in range(4)]
    k = [np.uint64(k[0]), np.uint64(k[1])]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        x = [(b >> half) ^ x[1] ^ k[0], b & low, (a >> half) ^ x[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(x, -1).astype(np.uint32)


def threshold(p):
    return int(np.rint(65536.0 * p))


def keep(rows, cols, p, seed, offset, first=0):
    """Which elements of rows first, first + 1, .. are kept."""
    nvec = max(1, -(-cols // 8))
    c = np.zeros((rows, nvec, 4), dtype=np.uint64)
    c[..., 0] = np.arange(nvec)
    c[..., 1] = np.arange(first, first + rows)[:, None]
    c[..., 2], c[..., 3] = offset & 0xFFFFFFFF, offset >> 32 & 0xFFFFFFFF
    w = philox(c, (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
    bits = np.stack([w & 0xFFFF, w >> 16], -1).reshape(rows, nvec * 8)[:, :cols]
    return torch.from_numpy(bits >= threshold(p))


def factor(p):
    t = threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def dropped(x, drop):
    """dropout of the binary32 (or binary64) matrix x; drop = (p, seed, offset) or None."""
    if drop is None or threshold(drop[0]) == 0:
        return x
    s = torch.tensor(factor(drop[0]), dtype=x.dtype)
    return torch.where(keep(*x.shape, *drop), x * s, torch.zeros((), dtype=x.dtype))


def layer(x, r, w, b, eps, drop=None):
    """(h, mean, rstd, y) in binary32, each before its output's rounding."""
    h = dropped(x.float(), drop)
    if r is not None:
        h = r.float() + h
    n = torch.tensor(float(h.shape[1]))
    mean = row_sums(h) / n
    d = h - mean[:, None]
    t = row_sums(d * d) / n + torch.tensor(eps, dtype=F32)
    rstd = (1.0 / torch.sqrt(t.double())).float()
    y = d * rstd[:, None]
    if w is not None:
        y = y * w.float()
    if b is not None:
        y = y + b.float()
    return h, mean, rstd, y


def groups(rows, cols, dtype):
    """The partial sums of the gradients of weight and bias."""
    c = [(128, 12), (256, 6), (384, 4), (640, 3), (768, 2), (1 << 24, 1)] if dtype == torch.float32 else \
        [(128, 16), (192, 12), (320, 8), (384, 5), (640, 4), (768, 2), (896, 3), (1 << 24, 2)]
    c = next(n for most, n in c if -(-cols // 8) <= most)
    return min(rows, max(152, min(152 * c, -(-rows // 2))))


def column_sums(e, dtype):
    """The declared order of the gradients of weight and bias."""
    rows, cols = e.shape
    G = groups(rows, cols, dtype)
    part = torch.zeros(G, cols)
    for r in range(rows):
        part[r % G] = part[r % G] + e[r]
    s = torch.zeros(32, cols)
    for k in range(G):
        s[k % 32] = s[k % 32] + part[k]
    n = 32
    while n > 1:
        n //= 2
        s = s[:n] + s[n:]
    return s[0]


def layer_back(dy, h, w, mean, rstd, dh, drop=None):
    """(dx, dresidual, dweight, dbias) in binary32, in the declared orders."""
    dyf = dy.float()
    n = torch.tensor(float(h.shape[1]))
    xh = (h.float() - mean[:, None]) * rstd[:, None]
    g = dyf * w.float() if w is not None else dyf
    a, c = row_sums(g) / n, row_sums(g * xh) / n
    dr = rstd[:, None] * ((g - a[:, None]) - xh * c[:, None])
    if dh is not None:
        dr = dr + dh.float()
    return dropped(dr, drop), dr, column_sums(dyf * xh, dy.dtype), column_sums(dyf, dy.dtype)


def layer64(x, r, w, b, eps, drop=None):
    h = dropped(x.double(), drop)
    if r is not None:
        h = r.double() + h
    var, mean = torch.var_mean(h, 1, unbiased=False)
    rstd = 1 / torch.sqrt(var + eps)
    y = (h - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * w.double()
    return h, mean, rstd, y if b is None else y + b.double()


def xent64(x, w, target, ignore, dloss):
    """(loss, lse, dx, dw, sizes) in binary64 on x's device; sizes: what the
    error bounds are made of."""
    live = target != ignore
    xd, wd = x.double().clone(), w.double()
    xd[~live] = 0                              # what ignored tokens hold counts for nothing
    logits = xd @ wd.t()
    size = (xd.abs() @ wd.abs().t()).amax(1)   # largest sum of magnitudes of a token's logits
    lse = torch.logsumexp(logits, 1)
    at = target.clamp(0, len(w) - 1)[:, None]
    hit = torch.zeros_like(logits).scatter_(1, at, 1.0)
    loss = torch.where(live, lse - logits.gather(1, at)[:, 0], 0.0)
    g = torch.where(live, dloss.double(), 0.0)[:, None]
    p = torch.exp(logits - lse[:, None])
    P = (p - hit) * g
    return loss, torch.where(live, lse, 0.0), P @ wd, P.t() @ xd, (size, p, hit, g, P, xd, wd, lse)
