"""The paged cache's bookkeeping on the host (no GPU: the tensors lie in host memory and no call is made on them)."""
import random

import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import build as _build  # noqa: E402
from speculative_decoding_draft_markov_gb300 import serving as V  # noqa: E402

PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _cache(n_pages, bs, max_pages, window=0, n_sink=0):
    return V.PagedCache(1, n_pages, PAGE, 2, 1, 64, bs, max_pages, V.rotation_table(8, 64, device="cpu"), window, n_sink,
                        device="cpu")


@pytest.mark.parametrize("lag", [0, 1, 3])
def test_rejected_drafts_give_their_place_back(lag):
    """Windows of 8 rows of which 1 to 3 are kept, lengths known `lag` steps late: the pages are those of the tokens that
    are there and of the steps under way."""
    rng, rows, steps = random.Random(lag), 8, 200
    c = _cache(1 + (3 * steps + rows * (lag + 2)) // PAGE, 1, 200)
    length, known = 0, []
    for t in range(steps):
        c.reserve(0, rows)
        assert c.bound[0] >= length + rows  # room for this step whatever the ones before kept
        assert len(c.pages[0]) * PAGE >= c.bound[0]
        length += rng.randint(1, 3)
        known.append(length)
        if t >= lag:
            c.settle(0, known[t - lag], since=rows * lag)
        assert c.bound[0] <= length + rows * (lag + 1)
    assert len(c.pages[0]) <= 1 + (length + rows * (lag + 2)) // PAGE


def test_a_length_never_raises_the_bound():
    c = _cache(10, 1, 10)
    c.reserve(0, 20)
    c.settle(0, 100)
    assert c.bound[0] == 20
    c.settle(0, 7, since=5)
    assert c.bound[0] == 12 and len(c.pages[0]) == 2
    c.reserve(0, 20)  # 32 tokens: the two pages it has
    assert len(c.pages[0]) == 2
    for bad in ((-1, 0), (3, -1)):
        with pytest.raises(ValueError):
            c.settle(0, *bad)


@pytest.mark.parametrize("window,n_sink,lag", [(40, 0, 0), (33, 4, 2), (1, 17, 0), (64, 100, 1)])
def test_pages_behind_the_window_come_back(window, n_sink, lag):
    """Two long requests in a cache that holds their windows and sinks: every position that a row can see has a page of
    its request's own, and nothing else is kept."""
    rng, rows, steps = random.Random(window), 8, 400
    one = -(-n_sink // PAGE) + -(-(window + rows * (lag + 2)) // PAGE) + 2
    c = _cache(2 * one, 2, 300, window, n_sink)
    length, known, owner = [0, 0], [[0, 0]], {}
    for t in range(steps):
        for r in range(2):
            c.reserve(r, rows)
        table = c.page_table.tolist()
        held = [p for q in c.pages for p in q if p is not None] + c.free
        assert sorted(held) == list(range(2 * one))
        for r in range(2):
            last = length[r] + rows - 1  # the step's rows: length .. last
            for j in range(last + 1):
                page = table[r][j // PAGE]
                if j > length[r] - window or j < n_sink:
                    assert page >= 0 and c.pages[r][j // PAGE] == page
            length[r] += rng.randint(1, 4)
        known.append(list(length))
        if t >= lag:
            for r in range(2):
                c.settle(r, known[t + 1 - lag][r], since=rows * lag)
    assert min(length) > 2 * one * PAGE  # more than the whole cache holds
    for r in range(2):
        c.release(r)
    assert sorted(c.free) == list(range(2 * one)) and (c.page_table == -1).all()


def test_a_length_of_an_earlier_request_takes_no_pages():
    """A length that came late, after its request was released and the place taken by a shorter one."""
    c = _cache(40, 1, 40, window=32)
    c.reserve(0, 500)
    c.release(0)
    c.reserve(0, 60)
    before = list(c.pages[0])
    c.settle(0, 490)
    assert c.pages[0] == before and c.bound[0] == 60 and (c.page_table[0, :4] >= 0).all()
    c.settle(0, 60)
    assert c.pages[0] == [None] + before[1:] and c.page_table[0, 0] == -1
