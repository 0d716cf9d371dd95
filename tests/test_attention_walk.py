"""The order in which the attention kernels load the KV tiles of a range, run on the host: every K and every V tile
once, none that the products do not wait for."""
import ctypes

import numpy as np
import pytest

from tests import host_library


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return host_library.load("attention_walk", tmp_path_factory.mktemp("host"))


def _ints(x):
    return np.ascontiguousarray(x, np.int32).ctypes.data_as(ctypes.POINTER(ctypes.c_int))


def _tiles(host, ns, ctxs, hkv, window, sinks, shift, unit):
    """All (request, KV head, first packed row, tile) of a call, and each one's Start (r, h, t, tile)."""
    out, row = [], 0
    for r, (n, c) in enumerate(zip(ns, ctxs)):
        for h in range(hkv):
            for t in range(-(-n // unit)):
                for i in range(host.tiles_of_unit(c, n, t, window, sinks, shift, unit)):
                    out.append(((r, h, row + t * unit, i), (r, h, t, i)))
        row += n
    return out


def _loads(host, ns, ctxs, hkv, window, sinks, shift, unit, start, count):
    cu, room = np.concatenate([[0], np.cumsum(ns)]), 2 * count + 64
    to = np.zeros((room, 5), np.int32)
    n = host.loads_of_range(_ints(cu), _ints(ctxs), len(ns), hkv, window, sinks, shift, unit, *start, ctypes.c_uint(count),
                            to.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), room)
    assert n <= room
    return [(x[0], tuple(x[1:])) for x in to[:n].tolist()]


CALLS = [
    # rows, cached tokens, KV heads, window, sinks, block shift, tokens of a unit
    ([1], [0], 1, 0, 0, 5, 1),
    ([1], [300], 1, 0, 0, 5, 1),             # a unit of three tiles
    ([1, 1, 1], [200, 10, 130], 2, 0, 0, 5, 1),
    ([8, 0, 3], [500, 7, 1000], 2, 300, 4, 4, 8),
    ([40, 5], [900, 0], 1, 0, 0, 3, 16),
    ([9], [100], 3, 64, 70, 5, 4),
]


@pytest.mark.parametrize("call", CALLS)
def test_loads_of_every_range(host, call):
    """Ranges of every length from every tile of the call: K 0, K 1, then V t, K t + 2, and nothing more."""
    every = _tiles(host, *call)
    assert every
    for at in range(len(every)):
        for count in range(1, min(len(every) - at, 9) + 1):
            tiles = [t for t, _ in every[at:at + count]]
            want = [(0, t) for t in tiles[:2]]
            for i, t in enumerate(tiles):
                want.append((1, t))
                want += [(0, x) for x in tiles[i + 2:i + 3]]
            assert _loads(host, *call, every[at][1], count) == want, (at, count)


def test_a_range_that_the_call_does_not_fill(host):
    """A range counted longer than what is there ends with it."""
    call = ([1], [300], 1, 0, 0, 5, 1)
    got = _loads(host, *call, (0, 0, 0, 0), 7)
    assert len(got) == 2 * len(_tiles(host, *call))


def test_an_empty_range_loads_nothing(host):
    assert _loads(host, *CALLS[1], (0, 0, 0, 0), 0) == []


@pytest.mark.parametrize("slots", [1, 2, 3, 5, 8])
def test_the_phase_that_a_drain_waits_for(host, slots):
    """The parity of a slot's last use, however far the ring has turned: not all slots used, whole turns, a part of one."""
    used = {}
    for n in range(1, 4 * slots + 3):
        slot = (n - 1) % slots
        used[slot] = used.get(slot, 0) + 1
        for s, times in used.items():
            assert host.last_use(n, slots, s) == (times - 1) % 2
