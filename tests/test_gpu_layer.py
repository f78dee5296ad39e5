"""GPU: the layer operators against their definitions in 64 bits
(tests/layer_ref.py), within bounds derived there, at the sizes, strides,
types and masks where they can go wrong; gradients also against differences
of the 64-bit forward pass; under graph replay, on other streams, in place."""
import numpy as np
import pytest
import torch

from signal_pad_sync_amd import arx
from tests import layer_ref as R
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SEED, OFFSET = 0x9E3779B97F4A7C15, (5 << 32) | 7


def rand(seed, *shape, dtype=BF16, scale=1.0, shift=0.0):
    """Seeded CPU tensor."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def dev(t, pad=0, lead=0):
    """t on the GPU; a plane with `pad` more columns a row and `lead` elements
    before its first, all of them NaN, which no result may show."""
    if t is None:
        return None
    if t.dim() == 1 or (pad == 0 and lead == 0):
        return t.cuda()
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + lead,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[lead:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def check_linear(m, n, k, dtype=BF16, act="none", bias=False, residual=False, save_z=False, pad=0, lead=0, seed=1):
    note(f"linear m={m} n={n} k={k} {dtype} {act} bias={bias} residual={residual} z={save_z} pad={pad} lead={lead}")
    x, w = rand(seed, m, k, dtype=dtype), rand(seed + 1, n, k, dtype=dtype, scale=max(k, 1) ** -0.5)
    b = rand(seed + 2, n, dtype=dtype) if bias else None
    r = rand(seed + 3, m, n, dtype=dtype) if residual else None
    got = arx.linear(dev(x, pad, lead), dev(w, pad, lead), bias=dev(b), residual=dev(r, pad, lead), act=act,
                     save_z=save_z)
    torch.cuda.synchronize()
    y, ye, z, ze = R.linear(x, w, b, r, act)
    R.close(got[0] if save_z else got, y, ye, "y")
    if save_z:
        R.close(got[1], z, ze, "z")


# lengths from one token on, at, below and above the edges of tiles and of
# groups of eight, and dimensions of one
SIZES = [(1, 1, 1), (1, 64, 8), (1, 2048, 512), (2, 100, 1000), (3, 17, 33), (5, 1, 300), (7, 4096, 64), (8, 129, 255),
         (15, 300, 100), (16, 256, 512), (17, 96, 72), (31, 33, 1024), (32, 512, 2048), (33, 64, 40), (63, 127, 129),
         (64, 64, 64), (65, 130, 96), (100, 1000, 77), (127, 255, 511), (128, 128, 128), (129, 257, 65), (200, 40, 4096),
         (255, 256, 64), (256, 512, 1024), (257, 300, 200), (300, 1, 65), (1, 300, 4096), (511, 513, 130), (1024, 8, 8)]


# up to 32 tokens: past weights streamed once, with the depth whole and split,
# and in tiles, which take weights on 16-byte boundaries only
@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 2048), (1, 512, 8192), (2, 500, 16384), (5, 300, 4096), (8, 5000, 2000),
                                   (16, 9000, 520), (16, 20000, 72), (3, 16384, 1024), (16, 2048, 8192),
                                   (16, 1024, 2056), (16, 1025, 4100), (7, 33000, 130),
                                   (17, 1024, 1024), (24, 4097, 1032), (31, 250, 520), (32, 700, 4096), (32, 40, 72),
                                   (32, 4096, 2048), (33, 1024, 1024)])
def test_few_tokens(m, n, k, pad):
    check_linear(m, n, k, F16 if n % 3 else BF16, "silu", bias=True, residual=True, save_z=True, pad=pad)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_linear_sizes(m, n, k, dtype):
    check_linear(m, n, k, dtype)
    check_linear(m, n, k, dtype, "gelu", True, True, True, pad=3, lead=1, seed=10)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("bias,residual,save_z", [(False, False, False), (True, False, True), (False, True, False),
                                                  (True, True, True)])
@pytest.mark.parametrize("m,n,k,pad", [(1, 333, 520, 0), (24, 160, 264, 8), (130, 200, 96, 5), (300, 260, 192, 0)])
def test_linear_epilogues(m, n, k, pad, act, bias, residual, save_z):
    check_linear(m, n, k, BF16, act, bias, residual, save_z, pad)


@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (2, 2), (4, 4), (8, 0), (0, 8), (64, 0)])
def test_linear_strides(pad, lead):
    for m, n, k in [(4, 128, 256), (40, 96, 320), (256, 256, 256), (260, 130, 64)]:
        check_linear(m, n, k, BF16, "silu", True, True, True, pad, lead)


def test_linear_of_nothing():
    x, w = torch.zeros(0, 16, dtype=BF16, device="cuda"), torch.zeros(8, 16, dtype=BF16, device="cuda")
    assert arx.linear(x, w).shape == (0, 8)
    b = rand(1, 8).cuda()
    y = arx.linear(torch.zeros(3, 0, dtype=BF16, device="cuda"), torch.zeros(8, 0, dtype=BF16, device="cuda"), bias=b)
    assert torch.equal(y, b.expand(3, 8))        # k = 0: the sum is empty, the epilogue is not
    dx, dw, db = arx.linear_backward(torch.zeros(0, 8, dtype=BF16, device="cuda"), x, w, dbias=True)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


def test_linear_infinities_stay_in_their_row():
    x, w = rand(1, 70, 200), rand(2, 90, 200)
    x[3, 199], x[68, 0] = float("inf"), float("nan")
    y = arx.linear(dev(x, 3), dev(w, 3)).float().cpu()
    rows = torch.isfinite(y).all(1)
    assert (rows == ~torch.isin(torch.arange(70), torch.tensor([3, 68]))).all()


def test_linear_in_place_residual():
    for m in (4, 200):
        x, w, r = rand(1, m, 96), rand(2, 136, 96, scale=0.1), rand(3, m, 136)
        out = dev(r, 8)
        got = arx.linear(x.cuda(), w.cuda(), residual=out, out=out)
        assert got is out
        y, ye, _, _ = R.linear(x, w, None, r, "none")
        R.close(out, y, ye)


def check_linear_backward(m, n, k, dtype, act, dbias, pad=0, lead=0, want=(True, True), seed=20):
    note(f"linear_backward m={m} n={n} k={k} {dtype} {act} dbias={dbias} pad={pad} lead={lead} {want}")
    dy, x = rand(seed, m, n, dtype=dtype), rand(seed + 1, m, k, dtype=dtype)
    w, z = rand(seed + 2, n, k, dtype=dtype, scale=k ** -0.5), rand(seed + 3, m, n, dtype=dtype, scale=1.5)
    got = arx.linear_backward(dev(dy, pad, lead), dev(x, pad, lead), dev(w, pad, lead),
                              z=None if act == "none" else dev(z, pad, lead), act=act, dx=want[0], dw=want[1],
                              dbias=dbias)
    torch.cuda.synchronize()
    for name, g, asked, (v, e) in zip(("dx", "dw", "dbias"), got, (*want, dbias),
                                      R.linear_backward(dy, x, w, z, act, dtype)):
        assert (g is not None) == asked
        if asked:
            R.close(g, v, e, name)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_backward_sizes(m, n, k):
    check_linear_backward(m, n, k, BF16, "none", True)
    check_linear_backward(m, n, k, F16, "gelu", True, pad=3, lead=1)


@pytest.mark.parametrize("act", R.ACTS)
def test_linear_backward_acts(act):
    check_linear_backward(130, 72, 264, BF16, act, True)
    check_linear_backward(64, 200, 96, BF16, act, False, pad=8)
    check_linear_backward(40, 65, 33, F16, act, True, 1, 0, (False, True))
    check_linear_backward(40, 64, 32, F16, act, True, 0, 0, (True, False))
    check_linear_backward(9, 64, 32, BF16, act, True, 0, 0, (False, False))


def differences(f, x, d, h=1e-4):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("act", R.ACTS)
def test_linear_gradient_against_differences(act):
    m, n, k = 24, 40, 56
    x, w, b = rand(1, m, k), rand(2, n, k, scale=k ** -0.5), rand(3, n)
    c = rand(4, m, n)
    _, z = arx.linear(x.cuda(), w.cuda(), bias=b.cuda(), act=act, save_z=True)
    dx, dw, db = arx.linear_backward(c.cuda(), x.cuda(), w.cuda(), z=z, act=act, dbias=True)

    def loss(x, w, b):
        return float((R.act(x @ w.t() + b, act) * c.double()).sum())
    xd, wd, bd = x.double(), w.double(), b.double()
    for g, f, at in ((dx, lambda v: loss(v, wd, bd), xd), (dw, lambda v: loss(xd, v, bd), wd),
                     (db, lambda v: loss(xd, wd, v), bd)):
        d = torch.randn(at.shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
        got = float((g.double().cpu() * d).sum())
        # z and g are rounded to bf16 (U each, slopes of slopes below 1.2),
        # and the gradient once more: 4 * 2^-9 of the terms' root mean square
        # sum, times 6 for chance; differences add h^2 of a third derivative
        size = float((g.double().cpu() * d).pow(2).sum().sqrt())
        assert abs(got - differences(f, at, d)) < 6 * 4 * R.U[BF16] * size + 1e-2 * (act == "relu") * size + 1e-4


# ---- row operators -----------------------------------------------------------

ROWS = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 64), (33, 100), (4, 511), (9, 512), (7, 513), (300, 130), (6, 1023),
        (5, 1024), (4, 1025), (3, 2048), (1000, 24), (3, 2050), (2, 4096), (600, 4096), (3, 4100), (2, 8192), (5, 8193),
        (3, 16384), (2, 16392), (2, 32768), (2, 40000), (3, 40001)]
TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]
IDS = ["bf16", "bf16-f32", "f16", "f16-f32", "f32"]


@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", ROWS)
def test_layer_norm(rows, cols, dtype, wdtype):
    for pad, lead, affine in ((0, 0, True), (3, 1, cols % 2 == 0)):
        note(f"layer_norm {rows}x{cols} {dtype} {wdtype} pad={pad} lead={lead}")
        x = rand(1, rows, cols, dtype=dtype, scale=2.0, shift=0.5)
        w = rand(2, cols, dtype=wdtype, shift=1.0) if affine else None
        b = rand(3, cols, dtype=wdtype) if affine else None
        got = arx.layer_norm(dev(x, pad, lead), dev(w), dev(b))
        for g, (v, e), name in zip(got, R.norm(x, w, b, 1e-5), ("y", "mean", "rstd")):
            R.close(g, v, e, name)


@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", ROWS)
def test_layer_norm_backward(rows, cols, dtype, wdtype):
    for pad, lead, affine in ((0, 0, True), (3, 1, cols % 2 == 0)):
        note(f"layer_norm_backward {rows}x{cols} {dtype} {wdtype} pad={pad} lead={lead}")
        x, dy = rand(1, rows, cols, dtype=dtype, scale=2.0, shift=0.5), rand(2, rows, cols, dtype=dtype)
        w = rand(3, cols, dtype=wdtype, shift=1.0) if affine else None
        mean = x.float().mean(1)
        rstd = (x.float().var(1, unbiased=False) + 1e-5).rsqrt()
        got = arx.layer_norm_backward(dev(dy, pad, lead), dev(x, pad, lead), mean.cuda(), rstd.cuda(), dev(w))
        assert got[1].dtype == (wdtype if affine else dtype)
        for g, (v, e), name in zip(got, R.norm_backward(dy, x, mean, rstd, w), ("dx", "dweight", "dshift")):
            R.close(g, v, e, name)


def test_layer_norm_of_hard_rows():
    """A constant row, a large mean beside a small spread, the largest and the
    smallest values, and rows that an infinity or a NaN spoils alone."""
    cols = 1000
    x = rand(1, 8, cols, dtype=F32)
    x[0] = 3.25
    x[1] = 1000.0 + 0.01 * x[1]
    x[2] = 1e15 * x[2]
    x[3] = 1e-30 * x[3]
    x[4, 999] = float("inf")
    x[5, 0] = float("nan")
    y, mean, rstd = arx.layer_norm(x.cuda())
    ok = [0, 1, 2, 3, 6, 7]
    for g, (v, e), name in zip((y, mean, rstd), R.norm(x[ok], None, None, 1e-5), ("y", "mean", "rstd")):
        R.close(g[ok], v, e, name)
    assert not y[0].any()
    assert torch.isnan(y[5]).all() and not torch.isfinite(y[4]).any()


def test_layer_norm_in_place():
    for cols in (100, 4096, 40000):
        x = rand(1, 5, cols, scale=2.0)
        buf = dev(x, 8)
        y, mean, rstd = arx.layer_norm(buf, out=buf)
        assert y is buf
        R.close(y, *R.norm(x, None, None, 1e-5)[0])


@pytest.mark.parametrize("kind", ["layer_norm", "dropout_add_norm"])
def test_norm_gradient_against_differences(kind):
    rows, cols, p = 6, 72, 0.25
    x, r = rand(1, rows, cols, dtype=F32), rand(2, rows, cols, dtype=F32)
    w, b, bias = rand(3, cols, dtype=F32, shift=1.0), rand(4, cols, dtype=F32), rand(5, cols, dtype=F32)
    cy, ch = rand(6, rows, cols, dtype=F32), rand(7, rows, cols, dtype=F32)
    mask = R.keep_mask(rows, cols, p, SEED, OFFSET)
    if kind == "layer_norm":
        _, mean, rstd = arx.layer_norm(x.cuda(), w.cuda(), b.cuda())
        dx, dw, db = arx.layer_norm_backward(cy.cuda(), x.cuda(), mean, rstd, w.cuda())
        grads = {"x": dx, "w": dw, "b": db}
    else:
        h, _, mean, rstd = arx.dropout_add_norm(x.cuda(), r.cuda(), w.cuda(), b.cuda(), bias=bias.cuda(), p=p,
                                                seed=SEED, offset=OFFSET)
        dx, dr, dbias, dw, db = arx.dropout_add_norm_backward(cy.cuda(), ch.cuda(), h, mean, rstd, w.cuda(), p=p,
                                                              seed=SEED, offset=OFFSET, dbias=True)
        grads = {"x": dx, "r": dr, "bias": dbias, "w": dw, "b": db}
    at = {"x": x.double(), "r": r.double(), "w": w.double(), "b": b.double(), "bias": bias.double()}

    def loss(v):
        h = v["x"]
        if kind != "layer_norm":
            h = torch.where(mask, (v["x"] + v["bias"]) * R.scale_of(p), torch.zeros_like(h)) + v["r"]
        d = h - h.mean(1, keepdim=True)
        y = d * ((d * d).mean(1, keepdim=True) + 1e-5) ** -0.5 * v["w"] + v["b"]
        return float((y * cy.double()).sum() + (kind != "layer_norm") * (h * ch.double()).sum())
    for name, g in grads.items():
        d = torch.randn(at[name].shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
        want = differences(lambda v: loss({**at, name: v}), at[name], d)
        terms = (g.double().cpu() * d)
        # binary32 roundings (a few hundred units at most) and h^2 = 1e-8 of a third derivative
        assert abs(float(terms.sum()) - want) < 512 * R.E * float(terms.abs().sum()) + 1e-5, name


DROPS = [0.0, 1e-6, 0.1, 0.5, 0.999, 1.0]


def test_generator_known_answers():
    """The published known-answer vectors of Philox4x32 with ten rounds."""
    ones = 0xFFFFFFFF
    assert R.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert R.philox((ones,) * 4, (ones, ones)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("rows,cols,pad", [(3, 8, 0), (5, 13, 0), (17, 100, 3), (2, 2050, 0), (40, 64, 8), (1, 1, 0)])
@pytest.mark.parametrize("p", DROPS)
def test_dropout_mask_is_the_generators(rows, cols, pad, p):
    note(f"dropout {rows}x{cols} p={p}")
    ones = torch.ones(rows, cols, dtype=F32)
    mask = R.keep_mask(rows, cols, p, SEED, OFFSET)
    want = torch.where(mask, torch.tensor(R.scale_of(p)), torch.tensor(0.0)).float()
    assert torch.equal(arx.dropout_add(dev(ones, pad), p=p, seed=SEED, offset=OFFSET).cpu(), want)
    assert torch.equal(arx.dropout_add_backward(dev(ones, pad), p=p, seed=SEED, offset=OFFSET)[0].cpu(), want)
    h, _, _, _ = arx.dropout_add_norm(dev(ones, pad), p=p, seed=SEED, offset=OFFSET)
    assert torch.equal(h.cpu(), want)


def test_no_dropout_copies_nothing():
    """p = 0 and a caller that lets them be shared: the dropout's gradient is its
    argument, the join's two gradients are one."""
    dh = rand(1, 33, 72).cuda()
    dx, db = arx.dropout_add_backward(dh, dbias=True, share=True)
    assert dx is dh
    R.close(db, *R.column_sum(dh.double().cpu(), torch.zeros(33, 72, dtype=torch.float64)))
    h, y, mean, rstd = arx.dropout_add_norm(dh, dh)
    dx, dr, _, _, _ = arx.dropout_add_norm_backward(dh, None, h, mean, rstd, share=True)
    assert dx is dr
    dx, dr, _, _, _ = arx.dropout_add_norm_backward(dh, None, h, mean, rstd, p=0.5, share=True)
    assert dx is not dr


def test_dropout_rate_and_independence():
    x = torch.ones(2048, 1024, dtype=BF16, device="cuda")
    n = x.numel()
    kept = [arx.dropout_add(x, p=0.3, seed=s, offset=o) != 0 for s, o in ((1, 0), (1, 1), (2, 0))]
    for a in kept:   # six standard deviations of a binomial
        assert abs(int(a.sum()) - 0.7 * n) < 6 * (0.21 * n) ** 0.5 + n * 2.0 ** -17
        both = (a[:, 1:] & a[:, :-1]).sum() / (n - 2048)
        assert abs(float(both) - 0.49) < 6 * (0.25 * 3 / n) ** 0.5 + 2.0 ** -16
    for a, b in ((0, 1), (0, 2), (1, 2)):
        assert abs(float((kept[a] & kept[b]).sum()) / n - 0.49) < 6 * (0.25 / n) ** 0.5 + 2.0 ** -16


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 9, 1), (70, 24, 0), (33, 300, 8), (9, 2056, 0), (300, 40, 3)])
def test_dropout_add(rows, cols, pad, dtype):
    x, r, b = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype), rand(3, cols, dtype=dtype)
    for p in (0.0, 0.2, 1.0):
        mask = R.keep_mask(rows, cols, p, SEED, OFFSET)
        for bias, res in ((None, None), (b, r), (None, r), (b, None)):
            got = arx.dropout_add(dev(x, pad), dev(res, pad), dev(bias), p=p, seed=SEED, offset=OFFSET)
            R.close(got, *R.dropout_add(x, res, bias, mask, R.scale_of(p)))
        dx, db = arx.dropout_add_backward(dev(x, pad), p=p, seed=SEED, offset=OFFSET, dbias=True)
        want, e = R.dropout_add(x, None, None, mask, R.scale_of(p))
        R.close(dx, want, e, "dx")
        R.close(db, *R.column_sum(want, e), "dbias")


def test_dropped_infinities_leave_no_nan():
    x = torch.full((64, 64), float("inf"), dtype=BF16, device="cuda")
    x[1] = float("nan")
    r = rand(1, 64, 64).cuda()
    assert torch.equal(arx.dropout_add(x, r, p=1.0), r)
    h, y, _, _ = arx.dropout_add_norm(x, r, p=1.0)
    assert torch.equal(h, r) and torch.isfinite(y).all()
    mask = R.keep_mask(64, 64, 0.5, 3, 4).cuda()
    got = arx.dropout_add(x, p=0.5, seed=3, offset=4)
    assert torch.equal(got[0] == float("inf"), mask[0]) and not got[~mask].any()


@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 13), (70, 64), (5, 1030), (4, 4096), (3, 8200), (2, 16400),
                                       (2, 33000)])
def test_dropout_add_norm(rows, cols, dtype, wdtype):
    x, r = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype, scale=2.0)
    w, b, bias = rand(3, cols, dtype=wdtype, shift=1.0), rand(4, cols, dtype=wdtype), rand(5, cols, dtype=dtype)
    dy, dh = rand(6, rows, cols, dtype=dtype), rand(7, rows, cols, dtype=dtype)
    for p, pad, full in ((0.0, 0, True), (0.3, 3, True), (0.3, 0, False)):
        note(f"dropout_add_norm {rows}x{cols} {dtype} {wdtype} p={p} pad={pad} full={full}")
        mask = R.keep_mask(rows, cols, p, SEED, OFFSET) if p else None
        kw = dict(p=p, seed=SEED, offset=OFFSET)
        res, bia = (r, bias) if full else (None, None)
        h, y, mean, rstd = arx.dropout_add_norm(dev(x, pad), dev(res, pad), dev(w), dev(b), bias=dev(bia), **kw)
        hv, he = R.dropout_add(x, res, bia, mask, R.scale_of(p))
        R.close(h, hv, he, "h")
        for g, (v, e), name in zip((y, mean, rstd), R.norm(hv, w, b, 1e-5, he), ("y", "mean", "rstd")):
            R.close(g, v, e, name)
        hc, mc, rc = h.cpu(), mean.cpu(), rstd.cpu()
        grad_h = dh if full else None
        dx, dr, db, dw, ds = arx.dropout_add_norm_backward(dev(dy, pad), dev(grad_h, pad), dev(hc, pad), mean, rstd,
                                                           dev(w), dbias=full, **kw)
        (d, de), vw, vs = R.norm_backward(dy, hc, mc, rc, w, grad_h)
        R.close(dr, d, de, "dresidual")
        v, e = R.dropout_add(d, None, None, mask, R.scale_of(p))
        e = e + de * (R.scale_of(p) if mask is not None else 1.0)
        R.close(dx, v, e, "dx")
        R.close(dw, *vw, "dweight")
        R.close(ds, *vs, "dshift")
        assert (db is not None) == full
        if full:
            R.close(db, *R.column_sum(v, e), "dbias")


@pytest.mark.parametrize("rows", [63, 64, 65, 128, 129])
@pytest.mark.parametrize("cols", [7, 136, 1001])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_column_sums_by_one_workgroup_and_by_several(rows, cols, dtype):
    """Bias gradients where their sums go from one kernel to two."""
    note(f"column sums {rows}x{cols} {dtype}")
    dh = rand(1, rows, cols, dtype=dtype)
    mask = R.keep_mask(rows, cols, 0.2, SEED, OFFSET)
    dx, db = arx.dropout_add_backward(dev(dh, 1), p=0.2, seed=SEED, offset=OFFSET, dbias=True)
    want, e = R.dropout_add(dh, None, None, mask, R.scale_of(0.2))
    R.close(dx, want, e, "dx")
    R.close(db, *R.column_sum(want, e), "dbias")
    x, w = rand(2, rows, 24, dtype=dtype), rand(3, cols, 24, dtype=dtype)
    none = torch.zeros(rows, cols, dtype=torch.float64)
    db = arx.linear_backward(dev(dh), dev(x), dev(w), dx=False, dw=False, dbias=True)[2]
    R.close(db, *R.column_sum(dh.double(), none), "dbias of linear")


@pytest.mark.parametrize("rows", [64, 65])
def test_wide_norm_gradients_by_one_workgroup_and_by_several(rows):
    cols = 8203
    x, dy, w = rand(1, rows, cols), rand(2, rows, cols), rand(3, cols, dtype=F32, shift=1.0)
    _, mean, rstd = arx.layer_norm(dev(x), dev(w))
    dx, dw, ds = arx.layer_norm_backward(dev(dy), dev(x), mean, rstd, dev(w))
    (d, de), vw, vs = R.norm_backward(dy, x, mean.cpu(), rstd.cpu(), w)
    R.close(dx, d, de, "dx")
    R.close(dw, *vw, "dweight")
    R.close(ds, *vs, "dshift")


def test_rows_of_nothing():
    x = torch.zeros(0, 24, dtype=BF16, device="cuda")
    assert arx.layer_norm(x)[0].shape == (0, 24)
    none = torch.zeros(0, dtype=F32, device="cuda")
    dx, dw, db = arx.layer_norm_backward(x, x, none, none)
    assert dx.shape == (0, 24) and not dw.any() and not db.any()
    wide = torch.zeros(0, 40000, dtype=BF16, device="cuda")
    assert not arx.layer_norm_backward(wide, wide, none, none)[1].any()
    assert arx.dropout_add(x, p=0.5).shape == (0, 24)
    assert not arx.dropout_add_backward(x, p=0.5, dbias=True)[1].any()
    assert not arx.dropout_add_norm_backward(x, None, x, none, none, dbias=True)[2].any()
    empty = torch.zeros(3, 0, dtype=BF16, device="cuda")
    assert arx.dropout_add(empty).shape == (3, 0) and arx.layer_norm(empty)[0].shape == (3, 0)


def test_same_call_same_bits():
    x, w, dy = rand(1, 700, 1000).cuda(), rand(2, 1000).cuda(), rand(3, 700, 1000).cuda()
    _, mean, rstd = arx.layer_norm(x, w)
    a, b = (arx.layer_norm_backward(dy, x, mean, rstd, w) for _ in range(2))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    p, q = (arx.linear_backward(dy, x, rand(4, 1000, 1000).cuda(), dbias=True) for _ in range(2))
    assert all(torch.equal(u, v) for u, v in zip(p, q))
    t, wt = rand(5, 3, 4096).cuda(), rand(6, 512, 4096).cuda()
    assert torch.equal(arx.linear(t, wt), arx.linear(t, wt))


def test_another_stream():
    """A call on a stream that is not the current one: its outputs and
    workspace belong to that stream."""
    x, w = rand(1, 40, 2048).cuda(), rand(2, 512, 2048, scale=0.02).cuda()
    want = arx.linear(x, w, act="gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append(arx.linear(x, w, act="gelu", stream=s))
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)   # the current stream's memory moves on
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with torch.cuda.stream(s):
        got = arx.layer_norm(x)[0]
    s.synchronize()
    assert torch.equal(got, arx.layer_norm(x)[0])


def test_graph_replays():
    """A layer's forward and backward calls captured in a hipGraph, replayed
    with eager work and new inputs between the replays."""
    m, d, f = 48, 512, 1024
    x, w1, w2 = rand(1, m, d).cuda(), rand(2, f, d, scale=0.05).cuda(), rand(3, d, f, scale=0.05).cuda()
    g, s = rand(4, d, shift=1.0).cuda(), rand(5, d).cuda()
    kw = dict(p=0.1, seed=11, offset=3)

    def step():
        u, z = arx.linear(x, w1, act="gelu", save_z=True)
        h, y, mean, rstd = arx.dropout_add_norm(arx.linear(u, w2), x, g, s, **kw)
        dx, dr, db, dw, ds = arx.dropout_add_norm_backward(y, None, h, mean, rstd, g, dbias=True, **kw)
        du, dw2, _ = arx.linear_backward(dx, u, w2)
        return h, y, dw, ds, db, dw2, *arx.linear_backward(du, x, w1, z=z, act="gelu", dbias=True)
    step()
    torch.cuda.synchronize()
    note("layer graph capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(3):
        x.copy_(rand(100 + rep, m, d))
        note(f"layer graph replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b), f"replay {rep}"
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements into their buffer."""
    ld, rows, cols = 1 << 28, 12, 520
    big = torch.zeros(ld * (rows - 1) + cols, dtype=torch.int16, device="cuda").view(BF16)
    x = torch.as_strided(big, (rows, cols), (ld, 1))
    t, w = rand(1, rows, cols), rand(2, 96, cols, scale=0.05)
    x.copy_(t)
    note("rows past 2^31 elements")
    y, ye, _, _ = R.linear(t, w, None, None, "none")
    R.close(arx.linear(x, w.cuda()), y, ye)
    R.close(arx.layer_norm(x)[0], *R.norm(t, None, None, 1e-5)[0])
    out = x
    mask = R.keep_mask(rows, cols, 0.5, 1, 2)
    arx.dropout_add(x, p=0.5, seed=1, offset=2, out=out)
    R.close(out, *R.dropout_add(t, None, None, mask, 2.0))
