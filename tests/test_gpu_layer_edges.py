"""GPU: the layer operators where a dimension is zero, against their
definitions (tests/layer_ref.py), and whose memory their results are."""
import pytest
import torch

from signal_pad_sync_amd import arx
from tests import layer_ref as R
from tests.gpu_util import library, note

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


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F16, F32), (F32, F32)], ids=["bf16", "f16-f32", "f32"])
@pytest.mark.parametrize("rows", [1, 5, 1000])
def test_statistics_of_no_columns(rows, dtype, wdtype):
    """The mean of nothing is NaN, and so is what follows from it; neither is
    what the memory held before."""
    note(f"norms {rows}x0 {dtype}")
    x, w = torch.zeros(rows, 0, dtype=dtype, device="cuda"), torch.zeros(0, dtype=wdtype, device="cuda")
    for call in (lambda: arx.layer_norm(x, w, w), lambda: arx.dropout_add_norm(x, x, w, w, bias=x[0], p=0.5)[1:],
                 lambda: arx.dropout_add_norm(x)[1:]):
        before = torch.full((2 * rows,), 7.0, device="cuda")
        del before                       # the statistics take its place
        y, mean, rstd = call()
        assert y.shape == (rows, 0) and torch.isnan(mean).all() and torch.isnan(rstd).all()
    stats = torch.full((2, rows), 7.0, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert arx.lib.arx_layer_norm(None, None, None, None, stats[0].data_ptr(), None, rows, 0, 0, 0, 1e-5, arx.BF16,
                                  arx.BF16, stream) == 0
    assert arx.lib.arx_dropout_add_norm(None, None, None, None, None, None, None, None, stats[1].data_ptr(), rows, 0,
                                        0, 0, 0, 0, 1e-5, 0.1, 1, 2, arx.F32, arx.F32, stream) == 0
    assert torch.isnan(stats).all()


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 0.25])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("other", [False, True], ids=["current", "stream"])
def test_gradients_own_their_memory(p, pad, other):
    """Whatever p is: each gradient contiguous and memory of its own, so that
    changing one in place changes neither another nor an argument."""
    note(f"gradients' memory p={p} pad={pad} other stream={other}")
    buf = torch.randn(33, 72 + pad, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    dh = buf[:, :72]
    h, y, mean, rstd = arx.dropout_add_norm(dh, dh)
    torch.cuda.synchronize()
    kept = buf.clone()
    s = torch.cuda.Stream() if other else None
    for dbias in (False, True):
        dx, _ = arx.dropout_add_backward(dh, p=p, dbias=dbias, stream=s)
        dxn, dr, _, _, _ = arx.dropout_add_norm_backward(dh, dh, h, mean, rstd, p=p, dbias=dbias, stream=s)
        torch.cuda.synchronize()
        outs = [dx, dxn, dr]
        want = [t.clone() for t in outs]
        if p < 2.0 ** -17:
            assert torch.equal(dx, dh) and torch.equal(dxn, dr)
        for i, t in enumerate(outs):
            assert t.is_contiguous()
            t.zero_()
            for j in range(i + 1, len(outs)):
                assert torch.equal(outs[j], want[j])
            assert torch.equal(buf, kept)
        torch.cuda.synchronize()


def test_gradients_of_no_dropout_take_the_all_reduce():
    """A column slice's gradient is a plane that arx.allreduce takes."""
    dh = torch.randn(8, 80, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()[:, :64]
    with library(2, 512):
        for src in (1,):
            arx.recv_view(1, src, 512).zero_()
        dx, _ = arx.dropout_add_backward(dh)
        out = torch.empty_like(dx)
        arx.allreduce(dx, out, 512)
        torch.cuda.synchronize()
        assert torch.equal(out, dh)


def test_column_sums_of_the_widest_plane():
    """2^31 - 1 columns, the largest size: one row's bias gradient is the row."""
    cols = (1 << 31) - 1
    note(f"dropout_add_backward 1x{cols}")
    dh = torch.empty(1, cols, dtype=BF16, device="cuda")
    dh.view(-1)[: 1 << 30].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    dh.view(-1)[1 << 30:] = dh.view(-1)[: cols - (1 << 30)].neg()
    dx, db = arx.dropout_add_backward(dh, dbias=True)
    assert torch.equal(db, dh[0]) and torch.equal(dx, dh)
