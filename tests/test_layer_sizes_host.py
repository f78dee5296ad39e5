"""The layer operators' size queries and host-side shapes over all sizes, none
among them (CPU only: nothing here reaches the device)."""
import itertools

import pytest

from signal_pad_sync_amd import arx

L = arx.lib


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
