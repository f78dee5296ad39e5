"""The layer operators in 64 bits (torch on the CPU), each output with a bound
on how far a correct binary32 computation that rounds it once may be off.

Bounds are derived, not fitted. U[dtype] is the unit roundoff of an output
type (2^-8, 2^-11, 2^-24: a value v rounds to within U |v| + TINY), E = 2^-24 that of binary32. A
sum of n terms added as a tree of depth d is off by at most about d E times
the sum of the terms' absolute values; every kernel adds fewer than `depth`
levels, so depth * 2 E covers the sum and its terms' own roundings.
"""
import math

import numpy as np
import torch

E = 2.0 ** -24
U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def philox(counter, key):
    """Philox4x32-10 in Python integers: four 32-bit counter words, two key words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(rows, cols, p, seed, offset):
    """The kept elements, one Python call of the generator per group of eight."""
    at, groups = round(65536 * p), -(-cols // 8)
    out = np.zeros((rows, groups * 8), dtype=bool)
    for r in range(rows):
        for g in range(groups):
            n = r * groups + g
            w = philox((n & 0xFFFFFFFF, n >> 32, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
            for j in range(8):
                out[r, 8 * g + j] = (w[j // 2] >> 16 * (j % 2) & 0xFFFF) >= at
    return torch.from_numpy(out[:, :cols].copy())


def scale_of(p):
    at = round(65536 * p)
    return 65536.0 / (65536 - at) if at < 65536 else 0.0


def close(got, want, bound, what=""):
    """got (any type, any device) within bound of want (64 bits), elementwise."""
    g = got.detach().double().cpu()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    off = (g - want).abs() - (bound + U[got.dtype] * want.abs() * 1.01 + TINY[got.dtype])
    bad = ~(off <= 0)
    if bad.any():
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {g.numel()} outside their bound, first at flat index {i}: "
                             f"got {g.reshape(-1)[i]:.9g}, want {want.reshape(-1)[i]:.9g}, "
                             f"bound {torch.as_tensor(bound).expand_as(want).reshape(-1)[i]:.3g}")


def act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def act_error(z, kind):
    """Error of a binary32 activation or slope at an exact z: a few units of
    the exponential's argument (its relative error grows with it) on a result
    of at most about |z| + 1."""
    return 0.0 * z if kind in ("none", "relu") else 2.0 ** -20 * (1 + z.abs()) * (1 + z.abs())


def linear(x, w, bias, residual, kind):
    """(y, its bound, z, its bound) from CPU tensors of any type."""
    x, w = x.double(), w.double()
    k = x.shape[1]
    z = x @ w.t()
    size = x.abs() @ w.abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    ze = (k + 8) * 2 * E * size
    y = act(z, kind)
    ye = 1.2 * ze + act_error(z, kind)           # every slope is at most 1.13
    if residual is not None:
        y = y + residual.double()
        ye = ye + 2 * E * (y.abs() + residual.double().abs())
    return y, ye, z, ze


def linear_backward(dy, x, w, z, kind, dtype):
    """[(dx, bound), (dw, bound), (dbias, bound)]: g enters the products
    rounded to dtype when an activation's slope is in it."""
    dy, x, w = dy.double(), x.double(), w.double()
    g, ge = dy, 0.0 * dy
    if kind != "none":
        s = slope(z.double(), kind)
        g = dy * s
        ge = dy.abs() * act_error(z.double(), kind) + 2 * E * g.abs()
    gr = ge + (U[dtype] * g.abs() + TINY[dtype] if kind != "none" else 0.0)
    m, n = dy.shape

    def product(a, b, ae):
        return a @ b, ae @ b.abs() + (a.shape[1] + 8) * 2 * E * ((a.abs() + ae) @ b.abs())
    return [product(g, w, gr), product(g.t(), x, gr.t()),
            (g.sum(0), ge.sum(0) + (m + 8) * 2 * E * (g.abs() + ge).sum(0))]


def depth(cols):
    return 40 + cols // 8192


def norm(h, weight, shift, eps, he=None):
    """(y, bound), (mean, bound), (rstd, bound) of rows h known to within he."""
    h = h.double()
    he = torch.zeros_like(h) if he is None else he
    cols = h.shape[1]
    d = depth(cols) * 2 * E
    mean = h.mean(1, keepdim=True)
    me = d * h.abs().mean(1, keepdim=True) + he.mean(1, keepdim=True)
    c = h - mean
    ce = he + me + 2 * E * (h.abs() + mean.abs())
    var = (c * c).mean(1, keepdim=True)
    ve = d * var + (2 * c.abs() * ce + ce * ce).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    # relative error of rstd: half that of var + eps, and a few roundings
    low = (var + eps - ve).clamp(min=1e-300)
    rel = 0.5 * ve / low * (rstd * 0 + 1) + 6 * E
    re = rstd * rel
    xh = c * rstd
    xe = ce * rstd * (1 + rel) + xh.abs() * (rel + 2 * E)
    w = torch.ones(cols, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(cols, dtype=torch.float64) if shift is None else shift.double()
    y = xh * w + b
    ye = xe * w.abs() + 4 * E * (y.abs() + b.abs() + (xh * w).abs())
    return (y, ye), (mean[:, 0], me[:, 0]), (rstd[:, 0], re[:, 0])


def norm_backward(dy, x, mean, rstd, weight, dh=None):
    """(d, bound), (dweight, bound), (dshift, bound); d has dh in it."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, cols = dy.shape
    w = torch.ones(cols, dtype=torch.float64) if weight is None else weight.double()
    e = depth(cols) * 2 * E
    xh = (x - mean) * rstd
    xe = 4 * E * (x.abs() + mean.abs()) * rstd
    g = dy * w
    s1, s2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    s1e = e * g.abs().mean(1, keepdim=True)
    s2e = e * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * xe).mean(1, keepdim=True)
    d = rstd * (g - s1 - xh * s2)
    de = rstd * (8 * E * (g.abs() + s1.abs() + (xh * s2).abs()) + s1e + xh.abs() * s2e + xe * (s2.abs() + s2e))
    if dh is not None:
        d = d + dh.double()
        de = de + 2 * E * (d.abs() + dh.double().abs())
    r = (rows // 256 + 64) * 2 * E
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return ((d, de), (dw, r * (dy * xh).abs().sum(0) + (dy.abs() * xe).sum(0)), (db, r * dy.abs().sum(0)))


def column_sum(d, de):
    return d.sum(0), (d.shape[0] // 256 + 64) * 2 * E * (d.abs() + de).sum(0) + de.sum(0)


def dropout_add(x, residual, bias, mask, scale):
    """(h, bound); mask None: everything stays."""
    v = x.double()
    if bias is not None:
        v = v + bias.double()
    size = v.abs()
    if mask is not None:
        v, size = torch.where(mask, v * scale, torch.zeros_like(v)), size * scale
    e = 4 * E * size
    if residual is not None:
        v = v + residual.double()
        e = e + 2 * E * (v.abs() + residual.double().abs())
    return v, e
