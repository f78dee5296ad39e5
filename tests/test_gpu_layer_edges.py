"""GPU: the layer operators where a dimension is zero, against their
definitions (tests/layer_ref.py)."""
import pytest
import torch

from signal_pad_sync_amd import arx
from tests import layer_ref as R
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("rows", [0, 1, 3, 300])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gradients_of_no_columns(rows, dtype):
    note(f"gradients {rows}x0 {dtype}")
    x, row = torch.zeros(rows, 0, dtype=dtype, device="cuda"), torch.zeros(rows, dtype=F32, device="cuda")
    dx, dw, ds = arx.layer_norm_backward(x, x, row, row)
    assert dx.shape == (rows, 0) and dw.shape == ds.shape == (0,)
    for p in (0.0, 0.5):
        dx, db = arx.dropout_add_backward(x, p=p, dbias=True)
        assert dx.shape == (rows, 0) and db.shape == (0,)
        dx, dr, db, dw, ds = arx.dropout_add_norm_backward(x, x, x, row, row, p=p, dbias=True)
        assert dx.shape == dr.shape == (rows, 0) and db.shape == dw.shape == ds.shape == (0,)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("m,n,k", [(5, 0, 16), (300, 0, 264), (0, 24, 16), (0, 0, 16), (5, 24, 0), (5, 0, 0), (0, 0, 0)])
def test_linear_gradients_with_a_dimension_of_zero(m, n, k, act):
    """Sums over nothing are zero, and a plane without elements stays one; the
    bias's gradient needs no depth."""
    note(f"linear_backward m={m} n={n} k={k} {act}")
    g = torch.Generator().manual_seed(1)
    dy, x, w, z = (torch.randn(*s, generator=g).to(BF16) for s in ((m, n), (m, k), (n, k), (m, n)))
    got = arx.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=None if act == "none" else z.cuda(), act=act, dbias=True)
    for name, t, (v, e) in zip(("dx", "dw", "dbias"), got, R.linear_backward(dy, x, w, z, act, BF16)):
        R.close(t, v, e, name)
    for want in ((True, False), (False, True)):
        part = arx.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=None if act == "none" else z.cuda(), act=act,
                                   dx=want[0], dw=want[1])
        for t, full, asked in zip(part, got, want):
            assert torch.equal(t, full) if asked else t is None
