"""GPU: the row operators where a team of lanes walks over several rows and a
launch has fewer teams than rows, against their definitions
(tests/layer_ref.py), over every width of a team."""
import numpy as np
import pytest
import torch

from signal_pad_sync_amd import arx
from tests import layer_ref as R
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SEED, OFFSET = 0xD1B54A32D192ED03, (9 << 32) | 2
TYPES = pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F16, F32), (F32, F32)], ids=["bf16", "f16-f32", "f32"])
# (rows, columns): a backward launch's 256 workgroups have 32768, 8192, 4096,
# 2048, 1024, 512 and 256 teams; past 8192 columns a column's rows are walked
WALKS = [(66000, 60), (16500, 250), (8300, 500), (4200, 1000), (2100, 1500), (1100, 2050), (600, 4100), (600, 8192), (300, 8203)]


def keep_mask(rows, cols, p, seed, offset):
    """layer_ref.keep_mask, all counters at a time."""
    groups = -(-cols // 8)
    n, low, half = np.arange(rows * groups, dtype=np.uint64), np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [n & low, n >> half, np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    bits = np.stack([w >> np.uint64(s) & np.uint64(0xFFFF) for w in c for s in (0, 16)], 1)
    return torch.from_numpy((bits >= round(65536 * p)).reshape(rows, groups * 8)[:, :cols].copy())


def test_mask_is_the_generators():
    assert torch.equal(keep_mask(7, 61, 0.3, SEED, OFFSET), R.keep_mask(7, 61, 0.3, SEED, OFFSET))


def close(got, want, bound, what):
    R.close(got, want.cpu(), bound.cpu(), what)


def normal(g, *shape, dtype, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


@TYPES
@pytest.mark.parametrize("rows,cols", WALKS)
def test_layer_norm_over_many_rows(rows, cols, dtype, wdtype):
    note(f"layer_norm {rows}x{cols} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = normal(g, rows, cols, dtype=dtype, scale=2.0, shift=0.5), normal(g, rows, cols, dtype=dtype)
    w, b = normal(g, cols, dtype=wdtype, shift=1.0), normal(g, cols, dtype=wdtype)
    got = arx.layer_norm(x, w, b)
    for t, (v, e), name in zip(got, R.norm(x, w, b, 1e-5), ("y", "mean", "rstd")):
        close(t, v, e, name)
    grads = arx.layer_norm_backward(dy, x, got[1], got[2], w)
    for t, (v, e), name in zip(grads, R.norm_backward(dy, x, got[1], got[2], w), ("dx", "dweight", "dshift")):
        close(t, v, e, name)


@TYPES
@pytest.mark.parametrize("rows,cols", WALKS)
def test_join_over_many_rows(rows, cols, dtype, wdtype):
    note(f"dropout_add_norm {rows}x{cols} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, r = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype, scale=2.0)
    w, b, bias = normal(g, cols, dtype=wdtype, shift=1.0), normal(g, cols, dtype=wdtype), normal(g, cols, dtype=dtype)
    dy, dh = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype)
    kw = dict(p=0.3, seed=SEED, offset=OFFSET)
    mask, scale = keep_mask(rows, cols, 0.3, SEED, OFFSET).cuda(), R.scale_of(0.3)
    h, y, mean, rstd = arx.dropout_add_norm(x, r, w, b, bias=bias, **kw)
    hv, he = R.dropout_add(x, r, bias, mask, scale)
    close(h, hv, he, "h")
    for t, (v, e), name in zip((y, mean, rstd), R.norm(hv, w, b, 1e-5, he), ("y", "mean", "rstd")):
        close(t, v, e, name)
    dx, dr, db, dw, ds = arx.dropout_add_norm_backward(dy, dh, h, mean, rstd, w, dbias=True, **kw)
    (d, de), vw, vs = R.norm_backward(dy, h, mean, rstd, w, dh)
    close(dr, d, de, "dresidual")
    v, e = R.dropout_add(d, None, None, mask, scale)
    e = e + de * scale
    for t, (want, bound), name in zip((dx, dw, ds, db), ((v, e), vw, vs, R.column_sum(v, e)),
                                      ("dx", "dweight", "dshift", "dbias")):
        close(t, want, bound, name)


def test_more_rows_than_a_launch_has_teams():
    """Narrow rows past 2^25, the teams of the largest forward launch."""
    rows, cols = (1 << 25) + 77, 7
    note(f"layer_norm {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = normal(g, rows, cols, dtype=BF16, scale=2.0)
    y, mean, rstd = arx.layer_norm(x)
    for part in (slice(0, 100), slice((1 << 25) - 100, None)):
        for t, (v, e), name in zip((y, mean, rstd), R.norm(x[part].cpu(), None, None, 1e-5), ("y", "mean", "rstd")):
            close(t[part], v, e, name)
