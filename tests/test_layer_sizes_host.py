"""The layer operators' size queries and host-side shapes over all sizes, none
among them (CPU only: nothing here reaches the device)."""
import ctypes
import itertools
import os
import subprocess

import pytest

from signal_pad_sync_amd import arx
from signal_pad_sync_amd import build as B
from tests import layer_cuts as C

L = arx.lib
HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host")
SRC, OUT = os.path.join(HERE, "shapes_harness.cpp"), os.path.join(HERE, "_build")


@pytest.mark.parametrize("rows,cols", list(itertools.product((0, 1, 3, 64, 65, 5000), (0, 1, 8, 8192, 8193))))
def test_rows_workspace_of_any_size(rows, cols):
    sizes = [L.arx_rows_workspace(rows, cols, k) for k in (1, 2, 3)]
    assert sizes == sorted(sizes) and (sizes[0] >= 4 * cols if cols else not any(s > 8 * rows for s in sizes))


@pytest.mark.parametrize("m,n,k", list(itertools.product((0, 1, 70), repeat=3)))
def test_linear_workspaces_of_any_size(m, n, k):
    for aligned in (0, 1):
        assert L.arx_linear_workspace(m, n, k, aligned) >= 0
        for act in (0, 2):
            assert L.arx_linear_backward_workspace(m, n, k, act, aligned) >= (2 * m * n if act else 0)


@pytest.fixture(scope="module")
def shapes():
    """csrc/arx_shapes.h built with g++ (tests/host/shapes_harness.cpp)."""
    os.makedirs(OUT, exist_ok=True)
    so = os.path.join(OUT, "libshapes.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", B.CSRC, SRC, "-o", so],
                   check=True)
    return ctypes.CDLL(so)


def cut_of(shapes, size, layout="fwd", as_is=True):
    out = (ctypes.c_uint64 * 4)()
    shapes.cut_of(*map(ctypes.c_uint32, size), layout == "dw", layout != "fwd", as_is, out)
    assert 0 < size[2] - out[2] * (out[1] - 1) <= out[2] or size[2] == 0     # the splits cover the depth, none is empty
    return C.NAMES[out[0]], out[1]


@pytest.mark.parametrize("as_is", [False, True])
@pytest.mark.parametrize("layout", ["fwd", "dx", "dw"])
def test_tiles_that_the_gpu_tests_reach(shapes, layout, as_is):
    for size, want in C.TILES.items():
        assert cut_of(shapes, C.in_layout(size, layout, as_is), layout, as_is) == want, size
    for name in C.NAMES[2:]:
        assert {s > 1 for c, s in C.TILES.values() if c == name} == {False, True}


def test_few_rows_that_the_gpu_tests_reach(shapes):
    for size, (on, off) in C.ROWS.items():
        assert cut_of(shapes, size) == on and cut_of(shapes, size, as_is=False) == off, size


def test_pairs_that_the_gpu_tests_reach(shapes):
    for (m, n, k), dw_first in C.PAIRS.items():
        assert shapes.paired(m, n, k) and (m >= n) == dw_first


@pytest.mark.parametrize("m", [1, 16, 17, 32, 33, 4096, 1 << 29])
@pytest.mark.parametrize("n", [1, 63, 64, 129, 4096, (1 << 22) - 8])
@pytest.mark.parametrize("k", [0, 1, 64, 4096, (1 << 22) - 8])
def test_splits_cover_the_depth(shapes, m, n, k):
    for layout in ("fwd", "dx", "dw"):
        for as_is in (False, True):
            cut_of(shapes, (m, n, k), layout, as_is)


@pytest.mark.parametrize("rows", [0, 1, 17, 64, 65, 1025, 1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("cols", [1, 8, 127, 4096, 1 << 22, (1 << 28) + 8, (1 << 31) - 129, (1 << 31) - 1])
@pytest.mark.parametrize("sums", [False, True])
def test_column_walks_fit_a_launch(shapes, rows, cols, sums):
    """Every column has a lane, and a launch has fewer than 2^32 threads in x:
    256 a workgroup here, and 1024 for 64 columns where several workgroups'
    sums are added."""
    out = (ctypes.c_uint64 * 3)()
    shapes.columns_of(ctypes.c_uint32(rows), ctypes.c_uint32(cols), sums, out)
    lanes, x, y = out
    assert x * lanes * 8 >= cols and 1 <= y < 1 << 16
    assert x * 256 < 1 << 32
    assert not sums or y == 1 or -(-cols // 64) * 1024 < 1 << 32
