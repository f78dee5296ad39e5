"""The layer operators' argument checks, in the library and in the binding
(CPU only: every call below is refused before it reaches the device), and
their code objects: no packed fp32 instructions in the assembly."""
import os
import re

import pytest
import torch

from signal_pad_sync_amd import arx
from signal_pad_sync_amd import build as B
from tests.test_isa import assembly

L = arx.lib
A, S = 1 << 30, 1 << 24     # addresses that no call may touch, far enough apart
BIG = 1 << 31


def linear(x=A, w=A + S, bias=None, r=None, y=A + 2 * S, z=None, m=4, n=8, k=16, ldx=16, ldw=16, ldr=8, ldy=8, ldz=8,
           act=0, dtype=0, ws=None, nws=0):
    return L.arx_linear(x, w, bias, r, y, z, m, n, k, ldx, ldw, ldr, ldy, ldz, act, dtype, ws, nws, None)


def linear_backward(dy=A, x=A + S, w=A + 2 * S, z=None, dx=A + 3 * S, dw=A + 4 * S, db=None, m=4, n=8, k=16, lddy=8,
                    ldx=16, ldw=16, ldz=8, lddx=16, lddw=16, act=0, dtype=0, ws=A + 5 * S, nws=S):
    return L.arx_linear_backward(dy, x, w, z, dx, dw, db, m, n, k, lddy, ldx, ldw, ldz, lddx, lddw, act, dtype, ws,
                                 nws, None)


def norm(x=A, w=None, b=None, y=A + S, mean=None, rstd=None, rows=4, cols=8, ldx=8, ldy=8, eps=1e-5, dtype=0, wdtype=0):
    return L.arx_layer_norm(x, w, b, y, mean, rstd, rows, cols, ldx, ldy, eps, dtype, wdtype, None)


def norm_backward(dy=A, x=A + S, mean=A + 2 * S, rstd=A + 3 * S, w=None, dx=A + 4 * S, dw=None, db=None, rows=4,
                  cols=8, lddy=8, ldx=8, lddx=8, dtype=0, wdtype=0, ws=A + 5 * S, nws=S):
    return L.arx_layer_norm_backward(dy, x, mean, rstd, w, dx, dw, db, rows, cols, lddy, ldx, lddx, dtype, wdtype, ws,
                                     nws, None)


def drop(x=A, b=None, r=None, h=A + S, rows=4, cols=8, ldx=8, ldr=8, ldh=8, p=0.1, dtype=0):
    return L.arx_dropout_add(x, b, r, h, rows, cols, ldx, ldr, ldh, p, 1, 2, dtype, None)


def drop_backward(dh=A, dx=A + S, db=A + 2 * S, rows=4, cols=8, lddh=8, lddx=8, p=0.1, dtype=0, ws=A + 3 * S, nws=S):
    return L.arx_dropout_add_backward(dh, dx, db, rows, cols, lddh, lddx, p, 1, 2, dtype, ws, nws, None)


def join(x=A, bias=None, r=None, w=None, b=None, h=A + S, y=A + 2 * S, mean=None, rstd=None, rows=4, cols=8, ldx=8,
         ldr=8, ldh=8, ldy=8, eps=1e-5, p=0.1, dtype=0, wdtype=0):
    return L.arx_dropout_add_norm(x, bias, r, w, b, h, y, mean, rstd, rows, cols, ldx, ldr, ldh, ldy, eps, p, 1, 2,
                                  dtype, wdtype, None)


def join_backward(dy=A, dh=None, h=A + S, mean=A + 2 * S, rstd=A + 3 * S, w=None, dx=A + 4 * S, dr=None, db=None,
                  dw=None, ds=None, rows=4, cols=8, ld=8, p=0.1, dtype=0, wdtype=0, ws=A + 5 * S, nws=S):
    return L.arx_dropout_add_norm_backward(dy, dh, h, mean, rstd, w, dx, dr, db, dw, ds, rows, cols, ld, ld, ld, ld,
                                           ld, p, 1, 2, dtype, wdtype, ws, nws, None)


REFUSED = [
    (linear, dict(m=BIG), "size"), (linear, dict(dtype=2), "dtype"), (linear, dict(dtype=-1), "dtype"),
    (linear, dict(act=5), "act"), (linear, dict(act=-1), "act"), (linear, dict(x=None), "null x"),
    (linear, dict(w=None), "null w"), (linear, dict(y=None), "null y"), (linear, dict(x=A + 1), "aligned"),
    (linear, dict(ldx=15), "row distance"), (linear, dict(ldw=15), "row distance"),
    (linear, dict(ldy=7), "row distance"), (linear, dict(ldx=BIG), "row distance"),
    (linear, dict(y=A), "overlaps"), (linear, dict(y=A + S), "overlaps"), (linear, dict(z=A + 2 * S), "overlaps"),
    (linear, dict(r=A + 2 * S + 2), "overlaps"), (linear, dict(bias=A + 2 * S), "overlaps"),
    (linear, dict(r=A + 2 * S, ldr=9), "overlaps"), (linear, dict(z=A + 2 * S + 8 * 2 * 2), "overlaps"),
    (linear_backward, dict(dy=None), "null dy"), (linear_backward, dict(x=None), "null x"),
    (linear_backward, dict(w=None), "null w"), (linear_backward, dict(act=2), "null z"),
    (linear_backward, dict(dx=A), "overlaps"), (linear_backward, dict(dw=A + 3 * S), "overlaps"),
    (linear_backward, dict(act=2, z=A + 6 * S, nws=16), "workspace"),
    (linear_backward, dict(db=A + 6 * S, ws=None), "workspace"),
    (linear_backward, dict(db=A + 6 * S, ws=A + 5 * S + 8), "16-byte"), (linear_backward, dict(dtype=2), "dtype"),
    (norm, dict(rows=BIG), "size"), (norm, dict(dtype=3), "dtype"), (norm, dict(dtype=2), "wdtype"),
    (norm, dict(wdtype=1), "wdtype"), (norm, dict(eps=-1.0), "eps"), (norm, dict(eps=float("nan")), "eps"),
    (norm, dict(x=None), "null x"), (norm, dict(y=None), "null y"), (norm, dict(ldx=7), "row distance"),
    (norm, dict(y=A + 2), "overlaps"), (norm, dict(y=A, ldy=16), "overlaps"), (norm, dict(mean=A + S), "overlaps"),
    (norm, dict(mean=A + 2 * S, rstd=A + 2 * S + 4), "overlaps"), (norm, dict(mean=A + 2 * S + 2), "aligned"),
    (norm_backward, dict(mean=None), "null mean"), (norm_backward, dict(rstd=None), "null rstd"),
    (norm_backward, dict(dx=None), "null dx"), (norm_backward, dict(nws=8), "workspace"),
    (norm_backward, dict(dw=A + 6 * S, db=A + 6 * S), "overlaps"), (norm_backward, dict(wdtype=1), "wdtype"),
    (drop, dict(p=-0.1), "p "), (drop, dict(p=1.1), "p "), (drop, dict(p=float("nan")), "p "),
    (drop, dict(h=None), "null h"), (drop, dict(h=A + 16), "overlaps"), (drop, dict(b=A + S), "overlaps"),
    (drop, dict(dtype=9), "dtype"), (drop_backward, dict(p=2.0), "p "), (drop_backward, dict(dh=None), "null dh"),
    (drop_backward, dict(nws=8), "workspace"), (drop_backward, dict(db=A + S), "overlaps"),
    (join, dict(y=A + S), "overlaps"), (join, dict(eps=float("inf")), "eps"), (join, dict(p=7.0), "p "),
    (join, dict(y=None), "null y"), (join, dict(wdtype=1), "wdtype"),
    (join_backward, dict(dx=None), "null dx"), (join_backward, dict(dr=A + 4 * S), "overlaps"),
    (join_backward, dict(ld=4), "row distance"), (join_backward, dict(ws=None), "workspace"),
]


@pytest.mark.parametrize("call,args,why", REFUSED, ids=[f"{c.__name__}-{i}" for i, (c, _, _) in enumerate(REFUSED)])
def test_refused(call, args, why):
    assert call(**args) == arx.EINVAL
    assert why in L.arx_strerror(arx.EINVAL).decode()


def test_nothing_to_do_needs_no_device():
    assert linear(m=0, y=None) == 0 and linear(n=0) == 0
    assert linear_backward(m=0, n=0) == 0 and linear_backward(dx=None, dw=None) == 0
    assert norm(rows=0) == 0 and norm(cols=0, x=None, y=None) == 0
    assert norm_backward(cols=0) == 0 and drop(rows=0) == 0 and drop_backward(rows=0, db=None) == 0
    assert join(cols=0) == 0 and join_backward(cols=0) == 0


def test_column_slices_of_one_buffer_do_not_overlap():
    """Planes side by side in wider rows are let pass the overlap check (and
    refused afterwards for their workspace, before any launch)."""
    side = dict(rows=4, cols=8, lddy=16, ldx=8, lddx=16, nws=0)
    assert norm_backward(dy=A, dx=A + 16, **side) == arx.EINVAL
    assert "workspace" in L.arx_strerror(arx.EINVAL).decode()
    assert norm_backward(dy=A + 16, dx=A, **side) == arx.EINVAL
    assert "workspace" in L.arx_strerror(arx.EINVAL).decode()
    assert norm_backward(dy=A, dx=A + 14, **side) == arx.EINVAL
    assert "overlaps" in L.arx_strerror(arx.EINVAL).decode()
    assert norm_backward(dy=A, dx=A + 18, **side) == arx.EINVAL     # its rows reach into the next row's dy
    assert "overlaps" in L.arx_strerror(arx.EINVAL).decode()
    assert norm_backward(dy=A, dx=A + 16 + 16 * 2 * 100, **side) == arx.EINVAL   # and beyond the last row
    assert "workspace" in L.arx_strerror(arx.EINVAL).decode()


def test_workspace_sizes():
    assert L.arx_rows_workspace(100, 64, 0) == 0 and L.arx_rows_workspace(100, 64, 4) == 0
    assert L.arx_rows_workspace(BIG, 64, 1) == 0 and L.arx_linear_workspace(BIG, 1, 1, 0) == 0
    for rows, cols in ((1, 1), (100, 64), (10000, 4096), (3, 40000)):
        sizes = [L.arx_rows_workspace(rows, cols, k) for k in (1, 2, 3)]
        assert sizes[0] >= 4 * cols and sizes == sorted(sizes)
    # an activation's backward pass keeps one plane of gradients
    plain, gelu = (L.arx_linear_backward_workspace(100, 64, 32, act, 1) for act in (0, 2))
    assert gelu >= plain + 100 * 64 * 2
    # operands off 16-byte boundaries are copied onto them
    assert L.arx_linear_workspace(100, 64, 32, 0) >= L.arx_linear_workspace(100, 64, 32, 1) + (100 + 64) * 32 * 2
    assert L.arx_linear_workspace(100, 64, 33, 1) >= L.arx_linear_workspace(100, 64, 32, 1) + (100 + 64) * 40 * 2
    assert L.arx_linear_backward_workspace(100, 64, 32, 0, 0) >= plain + (100 * 64 + 100 * 32 + 64 * 32) * 2


@pytest.mark.parametrize("n", [8, 512, 4096, 5000, 32000])
@pytest.mark.parametrize("k", [1, 64, 1000, 8192, 16384])
def test_unaligned_workspace_serves_aligned_operands(n, k):
    for m in (1, 2, 8, 16, 17, 64, 300):
        assert L.arx_linear_workspace(m, n, k, 0) >= L.arx_linear_workspace(m, n, k, 1)


@pytest.mark.parametrize("sizes", [dict(m=(1 << 29) + 1), dict(n=1 << 22), dict(k=(1 << 22) - 7)])
def test_linear_size_limits(sizes):
    assert linear(**sizes) == arx.EINVAL and linear_backward(**sizes) == arx.EINVAL
    assert "size" in L.arx_strerror(arx.EINVAL).decode()


def T(*shape, dtype=torch.bfloat16, strides=None):
    """A CPU tensor: the binding looks at types and shapes first, so every
    other refusal shows without a GPU, and it is refused for its device last."""
    return torch.empty_strided(shape, strides, dtype=dtype) if strides else torch.empty(shape, dtype=dtype)


F16, F32, I16 = torch.float16, torch.float32, torch.int16
V = T(4, dtype=F32)
BAD = [
    (lambda: arx.linear(T(4, 8), T(6, 8)), "w must be a GPU tensor"),
    (lambda: arx.linear(None, T(6, 8)), "x must be a tensor"),
    (lambda: arx.linear(T(4, 8, dtype=F32), T(8, 8)), "Float"),
    (lambda: arx.linear(T(4, 8), T(8, 8, dtype=F16)), "w is of type"),
    (lambda: arx.linear(T(4, 8), T(8, 9)), "w has shape"),
    (lambda: arx.linear(T(4, 8), T(8)), "w has shape"),
    (lambda: arx.linear(T(4, 8), T(8, 8), act="swish"), "act"),
    (lambda: arx.linear(T(2, 4, 8), T(8, 8)), "two dimensions"),
    (lambda: arx.linear(T(4, 8), T(8, 8, strides=(1, 8))), "contiguous"),
    (lambda: arx.linear(T(4, 8), T(8, 8, strides=(0, 1))), "contiguous"),
    (lambda: arx.linear_backward(T(4, 6), T(4, 8), T(7, 8)), "w has shape"),
    (lambda: arx.linear_backward(T(4, 6), T(5, 8), T(6, 8)), "GPU tensor"),
    (lambda: arx.layer_norm(T(4, 8), T(8, dtype=F16)), "weight is of type"),
    (lambda: arx.layer_norm(T(4, 8), None, T(8, dtype=F16)), "shift is of type"),
    (lambda: arx.layer_norm(T(4, 8, dtype=F32), T(8)), "weight is of type"),
    (lambda: arx.layer_norm(T(4, 8), T(9)), "weight has shape"),
    (lambda: arx.layer_norm(T(4, 8), T(8, strides=(2,))), "weight has shape"),
    (lambda: arx.layer_norm(T(4, 8, dtype=I16)), "Short"),
    (lambda: arx.layer_norm(T(4, 8), out=T(4, 9)), "out has shape"),
    (lambda: arx.layer_norm_backward(T(4, 8), T(5, 8), V, V), "x has shape"),
    (lambda: arx.dropout_add(T(4, 8), seed=-1), "seed"),
    (lambda: arx.dropout_add(T(4, 8), seed=1.5), "seed"),
    (lambda: arx.dropout_add(T(4, 8), offset=1 << 64), "offset"),
    (lambda: arx.dropout_add(T(4, 8), T(4, 9)), "residual has shape"),
    (lambda: arx.dropout_add(T(4, 8), T(1, 8)), "residual has shape"),
    (lambda: arx.dropout_add(T(4, 8), T(4, 8, dtype=F16)), "residual is of type"),
    (lambda: arx.dropout_add(T(4, 8), None, T(9)), "bias has shape"),
    (lambda: arx.dropout_add_backward(T(4, 8), offset=-1), "offset"),
    (lambda: arx.dropout_add_norm(T(4, 8), None, T(8), T(8, dtype=F32)), "GPU tensor"),
    (lambda: arx.dropout_add_norm_backward(T(4, 8), T(3, 8), T(4, 8), V, V), "dh has shape"),
    (lambda: arx.dropout_add_norm_backward(T(4, 8), None, T(3, 8), V, V), "h has shape"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_binding_refuses(i, monkeypatch):
    monkeypatch.setattr(arx, "_current_device", lambda: 0)
    monkeypatch.setattr(arx, "_current_stream", lambda device: 0)
    call, why = BAD[i]
    with pytest.raises(arx.ArxError) as e:
        call()
    assert e.value.code == arx.EINVAL and why in str(e.value)


def test_binding_refuses_a_wrong_count():
    with pytest.raises(arx.ArxError):
        arx._binding.linear(0, 0, T(4, 8))
    with pytest.raises(TypeError):
        arx._binding.bind(arx.ArxError)


@pytest.mark.parametrize("src", ["arx_rows.hip", "arx_linear.hip"])
def test_no_packed_fp32(src, tmp_path):
    for i, line in enumerate(assembly(os.path.join(B.CSRC, src), tmp_path)):
        assert not re.match(r"^\s*v_pk_(add|mul|fma)_f32", line), f"{src}:{i + 1}: {line.strip()}"
