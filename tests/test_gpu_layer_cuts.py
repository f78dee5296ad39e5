"""GPU: every cut of the matrix products (tests/layer_cuts.py, pinned by
tests/test_layer_sizes_host.py), at sizes that end inside a tile.

Small whole numbers make the sums exact in binary32 in any order, so every
output has one right value, and a depth that is lost, doubled or taken from a
neighbour shows in most of them. The epilogues and gradients are then compared
with their definitions in 64 bits (tests/layer_ref.py)."""
import pytest
import torch

from signal_pad_sync_amd import arx
from tests import layer_cuts as C
from tests import layer_ref as R
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
AS_IS = pytest.mark.parametrize("as_is", [False, True], ids=["copied", "as_is"])
TILES = [pytest.param(s, id="%s-%d-%dx%dx%d" % (*c, *s)) for s, c in C.TILES.items()]
ROWS = [pytest.param(s, id="%dx%dx%d" % s) for s in C.ROWS]
PAIRS = [pytest.param(s, id="%s-%dx%dx%d" % ("dw_first" if w else "dx_first", *s)) for s, w in C.PAIRS.items()]


def place(t, as_is):
    """t as a plane of a wider buffer, on 16-byte boundaries or off them, with
    NaN between its rows, which no result may show."""
    pad, lead = (8, 0) if as_is else (3, 1)
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + lead,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[lead:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


class Numbers:
    def __init__(self, seed, dtype):
        self.g, self.dtype = torch.Generator(device="cuda").manual_seed(seed), dtype

    def whole(self, *shape):
        return torch.randint(-2, 3, shape, generator=self.g, device="cuda").to(self.dtype)

    def normal(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(self.dtype)


def close(got, want, bound, what):
    R.close(got, want.cpu(), bound.cpu(), what)


def exact_linear(m, n, k, dtype, as_is):
    f = Numbers(m + n + k, dtype)
    x, w, b, r = f.whole(m, k), f.whole(n, k), f.whole(n), f.whole(m, n)
    y, z = arx.linear(place(x, as_is), place(w, as_is), bias=b, residual=place(r, as_is), save_z=True)
    want = x.double() @ w.double().t() + b.double()
    assert torch.equal(z, want.to(dtype)), "z"
    assert torch.equal(y, (want + r.double()).to(dtype)), "y"


@AS_IS
@TYPES
@pytest.mark.parametrize("size", TILES)
def test_forward_is_exact(size, dtype, as_is):
    size = C.in_layout(size, "fwd", as_is)
    note(f"linear {size} {dtype} as_is={as_is}")
    exact_linear(*size, dtype, as_is)


@AS_IS
@TYPES
@pytest.mark.parametrize("size", ROWS)
def test_few_rows_are_exact(size, dtype, as_is):
    note(f"linear {size} {dtype} as_is={as_is}")
    exact_linear(*size, dtype, as_is)


@AS_IS
@TYPES
@pytest.mark.parametrize("size", TILES)
def test_gradients_are_exact(size, dtype, as_is):
    """Each product on its own: of x over the columns, of w over the rows."""
    m, k, n = C.in_layout(size, "dx", as_is)
    note(f"linear_backward dx m={m} n={n} k={k} {dtype} as_is={as_is}")
    f = Numbers(m + n + k, dtype)
    dy, x, w = f.whole(m, n), f.whole(m, k), f.whole(n, k)
    dx, _, _ = arx.linear_backward(place(dy, as_is), place(x, as_is), place(w, as_is), dw=False)
    assert torch.equal(dx, (dy.double() @ w.double()).to(dtype)), "dx"
    n, k, m = C.in_layout(size, "dw", as_is)
    note(f"linear_backward dw m={m} n={n} k={k} {dtype} as_is={as_is}")
    dy, x, w = f.whole(m, n), f.whole(m, k), f.whole(n, k)
    _, dw, _ = arx.linear_backward(place(dy, as_is), place(x, as_is), place(w, as_is), dx=False)
    assert torch.equal(dw, (dy.double().t().contiguous() @ x.double()).to(dtype)), "dw"


@AS_IS
@TYPES
@pytest.mark.parametrize("size", PAIRS)
def test_paired_gradients_are_exact(size, dtype, as_is):
    m, n, k = size if not as_is else (size[0], C.up8(size[1]), C.up8(size[2]))
    note(f"linear_backward pair m={m} n={n} k={k} {dtype} as_is={as_is}")
    f = Numbers(m + n + k, dtype)
    dy, x, w = f.whole(m, n), f.whole(m, k), f.whole(n, k)
    dx, dw, db = arx.linear_backward(place(dy, as_is), place(x, as_is), place(w, as_is), dbias=True)
    assert torch.equal(dx, (dy.double() @ w.double()).to(dtype)), "dx"
    assert torch.equal(dw, (dy.double().t().contiguous() @ x.double()).to(dtype)), "dw"
    assert torch.equal(db, dy.double().sum(0).to(dtype)), "dbias"


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("size", TILES)
def test_epilogues(size, act):
    dtype, as_is = (BF16, True) if act == "gelu" else (F16, False)
    m, n, k = C.in_layout(size, "fwd", as_is)
    note(f"linear {m}x{n}x{k} {dtype} {act}")
    f = Numbers(1, dtype)
    x, w, b, r = f.normal(m, k), f.normal(n, k, scale=k ** -0.5), f.normal(n), f.normal(m, n)
    y, z = arx.linear(place(x, as_is), place(w, as_is), bias=b, residual=place(r, as_is), act=act, save_z=True)
    yv, ye, zv, ze = R.linear(x, w, b, r, act)
    close(y, yv, ye, "y")
    close(z, zv, ze, "z")


@pytest.mark.parametrize("act", ["gelu_tanh", "relu"])
@pytest.mark.parametrize("size", PAIRS)
def test_paired_gradients(size, act):
    """With an activation's slope in front of the products, twice: the same call
    gives the same bits."""
    m, n, k = size
    dtype = BF16 if act == "relu" else F16
    note(f"linear_backward pair {m}x{n}x{k} {dtype} {act}")
    f = Numbers(2, dtype)
    dy, x, w, z = f.normal(m, n), f.normal(m, k), f.normal(n, k, scale=k ** -0.5), f.normal(m, n, scale=1.5)
    args = [place(t, False) for t in (dy, x, w)]
    got = [arx.linear_backward(*args, z=place(z, False), act=act, dbias=True) for _ in range(2)]
    for name, a, b, (v, e) in zip(("dx", "dw", "dbias"), *got, R.linear_backward(dy, x, w, z, act, dtype)):
        assert torch.equal(a, b), name
        close(a, v, e, name)


def test_a_large_pair_gives_the_same_bits():
    """Many workgroups of both products at once, eight times."""
    m, n, k = 4096, 2048, 4096
    f = Numbers(3, BF16)
    dy, x, w, z = f.normal(m, n), f.normal(m, k), f.normal(n, k, scale=k ** -0.5), f.normal(m, n)
    note(f"linear_backward pair {m}x{n}x{k} again and again")
    first = arx.linear_backward(dy, x, w, z=z, act="gelu_tanh", dbias=True)
    for _ in range(7):
        for a, b in zip(first, arx.linear_backward(dy, x, w, z=z, act="gelu_tanh", dbias=True)):
            assert torch.equal(a, b)
