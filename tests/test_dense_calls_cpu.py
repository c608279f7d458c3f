"""What the dense operators' calls promise and refuse, the parts that need no
GPU."""

import os

import pytest

from host_paged_expert_gb300 import _lib


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from host_paged_expert_gb300 import build

        build.build()
    return _lib.lib()


def up(n, of):
    return -(-n // of) * of


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 65, 1021, 7826, 1 << 20])
@pytest.mark.parametrize("out", [1, 8, 9, 64, 88, 1536, 1 << 20])
@pytest.mark.parametrize("act", [0, 1, 4])
def test_linear_backward_workspace_goes_by_the_sizes(L, rows, out, act):
    """dz where it is not dy, and a row of sums for every 32 rows begun."""
    dz = up(2 * rows * up(out, 8), 256) if act or out % 8 else 0
    assert L.pe_linear_backward_workspace(rows, out, act) == dz + up(4 * -(-rows // 32) * out, 256)


def test_linear_backward_workspace_of_nothing(L):
    assert L.pe_linear_backward_workspace(0, 64, 1) == L.pe_linear_backward_workspace(4, 0, 1) == 0
    assert L.pe_linear_backward_workspace(4, 64, 5) == 0
