"""Which request owns a packed row, run on the host: rows before the first window and after the last belong to none."""
import ctypes

import numpy as np
import pytest

from tests import host_library


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return host_library.load("packed_rows", tmp_path_factory.mktemp("host"))


def _owner(host, cu, rows, row):
    cu = np.ascontiguousarray(cu, np.int32)
    return host.request_of(cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), cu.size - 1, rows, row)


@pytest.mark.parametrize("first", [0, 1, 7])
@pytest.mark.parametrize("ns", [[1], [3, 0, 2], [0, 4], [0, 0], [2] * 70, [1] * 32])
def test_owner(host, first, ns):
    cu = first + np.concatenate([[0], np.cumsum(ns)])
    rows = int(cu[-1]) + 3
    owners = [len(ns)] * first + [r for r, n in enumerate(ns) for _ in range(n)] + [len(ns)] * 3
    assert [_owner(host, cu, rows, i) for i in range(rows)] == owners


@pytest.mark.parametrize("cu", [[-1, 2], [0, 3, 2], [0, 11], [3, 1], [0, 2, 2, 1]])
def test_no_list_of_windows(host, cu):
    assert all(_owner(host, cu, 10, i) == -1 for i in range(10))
