"""The row operators of the 8-bit path restated on the CPU, operation for
operation in binary32 (torch CPU arithmetic rounds each step to nearest), and
in binary64 from their definitions."""
import torch

F32, F64 = torch.float32, torch.float64
U = 2.0 ** -24                                  # half an ulp of 1 in binary32
EPS_OUT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def row_sums(e):
    """The declared sum of each row of the binary32 matrix e."""
    rows, cols = e.shape
    nvec = max(1, -(-cols // 8))
    p = 1
    while p < nvec:
        p *= 2
    x = torch.zeros(rows, p * 8, dtype=F32)
    x[:, :cols] = e
    x = x.view(rows, p, 4, 2)
    x = x[..., 0] + x[..., 1]
    x = x.view(rows, p, 2, 2)
    x = x[..., 0] + x[..., 1]
    x = x[..., 0] + x[..., 1]
    while p > 1:
        p //= 2
        x = x[:, :p] + x[:, p:]
    return x[:, 0]


def depth(cols):
    return 3 + max(1, -(-cols // 8)).bit_length()


def codes(y):
    amax = y.abs().amax(1) if y.shape[1] else torch.zeros(y.shape[0])
    bad = ~torch.isfinite(y).all(1)
    scale = amax / torch.tensor(127.0)
    tiny = scale < 2.0 ** -126
    per = torch.tensor(127.0) / amax
    per = torch.where(bad | tiny, torch.zeros(()), per)
    # the product is exact in binary64: one rounding, to the code
    q = torch.where((bad | tiny)[:, None], torch.zeros(()).double(), torch.round(y.double() * per.double()[:, None])).to(torch.int8)
    scale = torch.where(tiny, torch.zeros(()), scale)
    return q, torch.where(bad, torch.tensor(float("nan")), scale)


def norm(x, r, w, eps):
    """(h before rounding, rstd, y before rounding) in binary32."""
    h = x.float() + r.float() if r is not None else x.float()
    ms = row_sums(h * h) / torch.tensor(float(h.shape[1]))
    t = ms + torch.tensor(eps, dtype=F32)
    rstd = (1.0 / torch.sqrt(t.double())).float()
    y = h * rstd[:, None]
    if w is not None:
        y = y * w.float()
    return h, rstd, y


def norm64(x, r, w, eps):
    h = x.double() + (r.double() if r is not None else 0)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, y * w.double() if w is not None else y


def groups(rows, cols):
    """The partial sums of the weight's gradient."""
    team = min(1024, (-(-cols // 8) + 31) // 32 * 32)
    return min(rows, 152 * (1024 // team), max(152, -(-rows // 4)))


def back(dy, h, w, rstd, dh):
    """(dx before rounding, dw) in binary32, in the declared orders."""
    rows, cols = h.shape
    hf, dyf = h.float(), dy.float()
    g = dyf * w.float() if w is not None else dyf
    xh = hf * rstd[:, None]
    c = row_sums(g * xh) / torch.tensor(float(cols))
    dx = rstd[:, None] * (g - xh * c[:, None])
    if dh is not None:
        dx = dx + dh.float()
    e = dyf * xh
    G = groups(rows, cols)
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
    return dx, s[0]


def back64(dy, h, w, rstd, dh):
    hd, dyd, rs = h.double(), dy.double(), rstd.double()[:, None]
    g = dyd * w.double() if w is not None else dyd
    xh = hd * rs
    dx = rs * (g - xh * (g * xh).mean(1, keepdim=True))
    size = rs * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    return dx, (dyd * xh).sum(0), size, (dyd * xh).abs().sum(0)
