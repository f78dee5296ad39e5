"""Cases for the operators around a tensor-parallel layer's all-reduce: the matrix product with its epilogue, dropout
with bias and residual, layer norm, and the last two in one pass, each forward and backward.

`run` computes them in elementary torch operations in 32 bits, or, with `own`, through signal_pad_sync_amd.arx.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # one token through a layer's first product at hidden size 4096: the weights are read once, latency counts
        {"name": "linear 1x4096x2048 gelu", "op": "linear", "m": 1, "k": 4096, "n": 2048, "act": "gelu",
         "bias": True, "residual": False, "save_z": False, "pad": 0, "dt": "bf16"},
        # the second product of a batch of 32 tokens: its output is the [32, 4096] partial that the ranks sum
        {"name": "linear 32x2048x4096", "op": "linear", "m": 32, "k": 2048, "n": 4096, "act": "none",
         "bias": False, "residual": False, "save_z": False, "pad": 0, "dt": "bf16"},
        # a ragged prompt and odd widths, rows that start on no 16-byte boundary
        {"name": "linear 333x1001x777 silu f16", "op": "linear", "m": 333, "k": 1001, "n": 777, "act": "silu",
         "bias": True, "residual": True, "save_z": True, "pad": 3, "dt": "f16"},
        # the largest: a training batch of 8192 tokens at hidden size 8192, z kept for the backward pass
        {"name": "linear 8192x8192x8192 gelu", "op": "linear", "m": 8192, "k": 8192, "n": 8192, "act": "gelu",
         "bias": True, "residual": True, "save_z": True, "pad": 0, "dt": "bf16"},
        # the backward pass of a training layer's first product at hidden size 4096
        {"name": "linear bwd 8192x4096x2048", "op": "linear_backward", "m": 8192, "k": 4096, "n": 2048,
         "act": "gelu_tanh", "bias": True, "pad": 0, "dt": "bf16"},
        # layer norm of a decode batch of 32 tokens
        {"name": "layer norm 32x4096", "op": "layer_norm", "rows": 32, "cols": 4096, "pad": 0, "dt": "bf16",
         "wt": "bf16"},
        # odd rows and columns in float32, rows cut out of a wider buffer
        {"name": "layer norm 4099x1023 f32", "op": "layer_norm", "rows": 4099, "cols": 1023, "pad": 5, "dt": "f32",
         "wt": "f32"},
        # the backward pass of a training batch at hidden size 8192, weights kept in float32
        {"name": "layer norm bwd 8192x8192", "op": "layer_norm_backward", "rows": 8192, "cols": 8192, "pad": 0,
         "dt": "bf16", "wt": "f32"},
        # bias, dropout and residual behind the sum of a training layer at hidden size 4096
        {"name": "dropout add 8192x4096", "op": "dropout_add", "rows": 8192, "cols": 4096, "bias": True,
         "residual": True, "p": 0.1, "pad": 0, "dt": "bf16"},
        # its backward pass with the bias's gradient, at odd sizes
        {"name": "dropout add bwd 3001x1025 f16", "op": "dropout_add_backward", "rows": 3001, "cols": 1025,
         "bias": True, "p": 0.25, "pad": 0, "dt": "f16"},
        # the summed partial of a decode batch joins the residual and is normalised for the next product
        {"name": "dropout add norm 32x4096", "op": "dropout_add_norm", "rows": 32, "cols": 4096, "bias": True,
         "p": 0.0, "pad": 0, "dt": "bf16", "wt": "bf16"},
        # the backward pass of the same join in training
        {"name": "dropout add norm bwd 8192x4096", "op": "dropout_add_norm_backward", "rows": 8192, "cols": 4096,
         "bias": True, "p": 0.1, "pad": 0, "dt": "bf16", "wt": "bf16"},
    ]


def draw(rng):
    def length(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return min(hi, max(lo, n))

    def width(lo, hi):
        n = length(lo, hi)
        if rng.random() < 0.6:  # a multiple of 64 or of 8, as most layers have
            n = max(lo, n // 64 * 64 if rng.random() < 0.6 else n // 8 * 8)
        return n if n != 3 << 10 else n + 64

    op = rng.choice(["linear", "linear", "linear", "linear_backward", "linear_backward", "layer_norm",
                     "layer_norm_backward", "dropout_add", "dropout_add_backward", "dropout_add_norm",
                     "dropout_add_norm_backward"])
    pad = rng.choice([0, 0, 0, 8, 3])
    if op.startswith("linear"):
        dt = rng.choice(["bf16", "bf16", "f16"])
        case = {"op": op, "m": length(1, 8192), "k": width(64, 8192), "n": width(64, 8192),
                "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "bias": rng.random() < 0.5}
        if op == "linear":
            case.update(residual=rng.random() < 0.5, save_z=rng.random() < 0.5)
        else:
            case["n"] = min(case["n"], 4096)
        return {**case, "pad": pad, "dt": dt}
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    cols = width(16, 16384)
    rows = length(1, min(16384, (1 << 25) // cols))
    case = {"op": op, "rows": rows, "cols": cols, "pad": pad, "dt": dt}
    if "norm" in op:
        case["wt"] = rng.choice([dt, "f32"])
    if op.startswith("dropout"):
        case.update(bias=rng.random() < 0.5, p=rng.choice([0.0, 0.1, 0.1, 0.25, 0.5]))
    if op == "dropout_add":
        case["residual"] = rng.random() < 0.7
    return case


def work(case):
    e, op = SIZE[case["dt"]], case["op"]
    if op.startswith("linear"):
        m, k, n = case["m"], case["k"], case["n"]
        if op == "linear":
            outs = 1 + case["residual"] + case["save_z"]
            return {"bytes": e * (m * k + n * k + n * case["bias"] + m * n * outs), "flops": 2 * m * n * k}
        reads = m * n * (1 if case["act"] == "none" else 2) + m * k + n * k
        return {"bytes": e * (reads + m * k + n * k + n * case["bias"]), "flops": 4 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    w = SIZE[case["wt"]] if "wt" in case else 0
    b = e * cols * case.get("bias", False)
    planes, flops, small = {
        "layer_norm": (2, 8, 2 * w * cols + 8 * rows),
        "layer_norm_backward": (3, 14, 3 * w * cols + 8 * rows),
        "dropout_add": (2 + case.get("residual", False), 4, b),
        "dropout_add_backward": (2, 3, b),
        "dropout_add_norm": (4, 12, b + 2 * w * cols + 8 * rows),
        "dropout_add_norm_backward": (5, 18, b + 3 * w * cols + 8 * rows),
    }[op]
    return {"bytes": e * planes * rows * cols + small, "flops": flops * rows * cols}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, pad = DTYPES[case["dt"]], case["pad"]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(shift).to(dtype)

    def rows_of(r, c, **kw):  # with a pad: the first columns of a wider buffer
        return normal(r, c + pad, **kw)[:, :c]

    s = {"case": case, "op": case["op"]}
    if case["op"].startswith("linear"):
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = rows_of(m, k)
        s["w"] = normal(n, k, scale=k ** -0.5)
        if case["op"] == "linear":
            s["bias"] = normal(n, scale=0.5) if case["bias"] else None
            s["residual"] = rows_of(m, n) if case["residual"] else None
        else:
            s["dy"] = rows_of(m, n, scale=0.1)
            s["z"] = normal(m, n) if case["act"] != "none" else None
        return s
    rows, cols = case["rows"], case["cols"]
    s["seed"], s["offset"] = (seed * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF, seed & 0xFFFF
    if "wt" in case:
        s["weight"] = normal(cols, scale=0.2, shift=1.0, dtype=DTYPES[case["wt"]])
        s["shift"] = normal(cols, scale=0.2, dtype=DTYPES[case["wt"]])
    if case["op"].startswith("dropout") and not case["op"].endswith("backward"):
        s["bias"] = normal(cols, scale=0.5) if case["bias"] else None
        s["residual"] = rows_of(rows, cols, scale=2.0) if case.get("residual", True) else None
    if case["op"] in ("layer_norm", "layer_norm_backward", "dropout_add", "dropout_add_norm"):
        s["x"] = rows_of(rows, cols, scale=1.5, shift=0.3)
    if case["op"] in ("layer_norm_backward", "dropout_add_norm_backward"):
        if "x" not in s:
            s["h"] = rows_of(rows, cols, scale=1.5, shift=0.3)
        x = s["x" if "x" in s else "h"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt()
        s["dy"] = rows_of(rows, cols, scale=0.1)
    if case["op"] in ("dropout_add_backward", "dropout_add_norm_backward"):
        s["dh"] = rows_of(rows, cols, scale=0.1)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from signal_pad_sync_amd import arx
    c, op = s["case"], s["op"]
    if op == "linear":
        return arx.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=c["act"], save_z=c["save_z"])
    if op == "linear_backward":
        return arx.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], act=c["act"], dbias=c["bias"])
    if op == "layer_norm":
        return arx.layer_norm(s["x"], s["weight"], s["shift"], eps=EPS)
    if op == "layer_norm_backward":
        return arx.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "dropout_add":
        return arx.dropout_add(s["x"], s["residual"], s["bias"], p=c["p"], seed=s["seed"], offset=s["offset"])
    if op == "dropout_add_backward":
        return arx.dropout_add_backward(s["dh"], p=c["p"], seed=s["seed"], offset=s["offset"], dbias=c["bias"])
    if op == "dropout_add_norm":
        return arx.dropout_add_norm(s["x"], s["residual"], s["weight"], s["shift"], bias=s["bias"], p=c["p"],
                                    seed=s["seed"], offset=s["offset"], eps=EPS)
    return arx.dropout_add_norm_backward(s["dy"], s["dh"], s["h"], s["mean"], s["rstd"], s["weight"], p=c["p"],
                                         seed=s["seed"], offset=s["offset"], dbias=c["bias"])


# ---- the plain forms -------------------------------------------------------


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * z * z)
    f = 1.0 / (1.0 + torch.exp(-z))
    return f * (1.0 + z * (1.0 - f))


def _keep(rows, cols, p, seed, offset, device):
    """The elements that stay: 16 of the generator's bits each, eight elements a counter."""
    low, groups = 0xFFFFFFFF, (cols + 7) // 8
    c0 = torch.arange(rows * groups, device=device)
    c0, c1 = c0 & low, c0 >> 32
    c2, c3 = torch.full_like(c0, offset & low), torch.full_like(c0, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2)
    return halves.reshape(rows, groups * 8)[:, :cols] >= int(round(p * 65536))


def _drop(v, s):
    p = s["case"]["p"]
    at = int(round(p * 65536))
    if at == 0:
        return v
    keep = _keep(v.shape[0], v.shape[1], p, s["seed"], s["offset"], v.device)
    return torch.where(keep, v * (65536.0 / (65536 - at)), 0.0)


def _norm(x, s):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
    return d * rstd[:, None] * s["weight"].float() + s["shift"].float(), mean, rstd


def _norm_grad(dy, x, s):
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0).to(s["weight"].dtype), dy.sum(0).to(s["weight"].dtype)


def _plain(s):
    c, op, dt = s["case"], s["op"], DTYPES[s["case"]["dt"]]
    if op == "linear":
        z = torch.matmul(s["x"].float(), s["w"].float().t())
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        return (y.to(dt), z.to(dt)) if c["save_z"] else y.to(dt)
    if op == "linear_backward":
        g = s["dy"].float()
        if c["act"] != "none":
            g = g * _act_grad(s["z"].float(), c["act"])
        dx, dw = torch.matmul(g, s["w"].float()), torch.matmul(g.t(), s["x"].float())
        return dx.to(dt), dw.to(dt), g.sum(0).to(dt) if c["bias"] else None
    if op == "layer_norm":
        y, mean, rstd = _norm(s["x"].float(), s)
        return y.to(dt), mean, rstd
    if op == "layer_norm_backward":
        dx, dw, db = _norm_grad(s["dy"].float(), s["x"].float(), s)
        return dx.to(dt), dw, db
    if op in ("dropout_add", "dropout_add_norm"):
        v = s["x"].float()
        if c["bias"]:
            v = v + s["bias"].float()
        h = _drop(v, s)
        if s["residual"] is not None:
            h = h + s["residual"].float()
        if op == "dropout_add":
            return h.to(dt)
        y, mean, rstd = _norm(h, s)
        return h.to(dt), y.to(dt), mean, rstd
    if op == "dropout_add_backward":
        dx = _drop(s["dh"].float(), s)
        return dx.to(dt), dx.sum(0).to(dt) if c["bias"] else None
    dh, dw, db = _norm_grad(s["dy"].float(), s["h"].float(), s)
    dh = dh + s["dh"].float()
    dx = _drop(dh, s)
    return dx.to(dt), dh.to(dt), dx.sum(0).to(dt) if c["bias"] else None, dw, db


# ---- the definitions in 64 bits ---------------------------------------------


def _exact_mask(rows, cols, p, seed, offset):
    """Multiplier of each element: 0 or 1/(1-p), from the generator in unsigned 64-bit host arithmetic."""
    import numpy as np
    per_row = -(-cols // 8)
    n = np.arange(rows * per_row, dtype=np.uint64)
    mask, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    ctr = [n & mask, n >> half, np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, offset >> 32)]
    for r in range(10):
        key0 = np.uint64((seed + r * 0x9E3779B9) & 0xFFFFFFFF)
        key1 = np.uint64(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        p0, p1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(p1 >> half) ^ ctr[1] ^ key0, p1 & mask, (p0 >> half) ^ ctr[3] ^ key1, p0 & mask]
    out = np.empty((len(n), 8), dtype=np.uint32)
    for j in range(8):
        out[:, j] = (ctr[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF)
    at = int(round(p * 65536))
    keep = out.reshape(rows, per_row * 8)[:, :cols] >= at
    return torch.from_numpy(keep).cuda().double() * (65536.0 / max(1, 65536 - at))


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op.startswith("linear"):
        if op == "linear":
            z = d["x"] @ d["w"].T
            if "bias" in d:
                z += d["bias"]
            f = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0),
                 "gelu": lambda t: t * (0.5 * torch.special.erfc(-t / 2 ** 0.5)),
                 "gelu_tanh": lambda t: t * torch.sigmoid((8 / math.pi) ** 0.5 * (t + 0.044715 * t ** 3)),
                 "silu": lambda t: t * torch.sigmoid(t)}[case["act"]]
            y = f(z)
            if "residual" in d:
                y = y + d["residual"]
            return (y, z) if case["save_z"] else y
        g = d["dy"]
        if case["act"] != "none":
            z = d["z"]
            if case["act"] == "relu":
                slope = (z > 0).double()
            elif case["act"] == "gelu":
                slope = 0.5 * torch.special.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
            elif case["act"] == "gelu_tanh":
                a = (8 / math.pi) ** 0.5
                f = torch.sigmoid(a * (z + 0.044715 * z ** 3))
                slope = f + z * f * (1 - f) * a * (1 + 3 * 0.044715 * z * z)
            else:
                f = torch.sigmoid(z)
                slope = f + z * f * (1 - f)
            g = g * slope
        return g @ d["w"], g.T @ d["x"], g.sum(0) if case["bias"] else None
    m = None
    if case.get("p", 0.0) > 0:
        m = _exact_mask(case["rows"], case["cols"], case["p"], s["seed"], s["offset"])
    if op == "dropout_add_backward":
        dx = d["dh"] if m is None else d["dh"] * m
        return dx, dx.sum(0) if case["bias"] else None
    if op in ("dropout_add", "dropout_add_norm", "layer_norm"):
        h = d["x"]
        if "bias" in d:
            h = h + d["bias"]
        if m is not None:
            h = h * m
        if "residual" in d:
            h = h + d["residual"]
        if op == "dropout_add":
            return h
        mean = h.mean(1, keepdim=True)
        rstd = (h.var(1, keepdim=True, correction=0) + EPS) ** -0.5
        y = (h - mean) * rstd * d["weight"] + d["shift"]
        return (y, mean[:, 0], rstd[:, 0]) if op == "layer_norm" else (h, y, mean[:, 0], rstd[:, 0])
    x = d["h"] if "h" in d else d["x"]
    rs, cols = d["rstd"][:, None], case["cols"]
    xh = (x - d["mean"][:, None]) * rs
    t = d["dy"] * d["weight"]
    grad = rs / cols * (cols * t - t.sum(1, keepdim=True) - xh * (t * xh).sum(1, keepdim=True))
    dw, db = (d["dy"] * xh).sum(0), d["dy"].sum(0)
    if op == "layer_norm_backward":
        return grad, dw, db
    grad = grad + d["dh"]
    dx = grad if m is None else grad * m
    return dx, grad, dx.sum(0) if case["bias"] else None, dw, db
