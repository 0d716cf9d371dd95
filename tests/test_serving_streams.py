"""The served step and the paged cache do all their work on the stream they are given (no GPU: the library's calls are
stood in for, and every torch operation is asked which stream is the current one)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")
from torch.overrides import TorchFunctionMode  # noqa: E402

from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import serving as V  # noqa: E402
from speculative_decoding_draft_markov_gb300 import step as S  # noqa: E402


class FakeStream:
    cuda_stream = 4096


@pytest.fixture
def current(monkeypatch):
    """The streams that torch's stream contexts have made current, the innermost last."""
    stack = [None]

    @contextlib.contextmanager
    def use(stream):
        stack.append(stream)
        yield
        stack.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    return stack


class Asks(TorchFunctionMode):
    """Collects the stream that is current at each torch operation that writes or computes."""

    def __init__(self, current):
        self.current, self.seen = current, []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        name = getattr(func, "__name__", str(func))
        if name not in ("__get__", "__len__", "size", "dim"):
            self.seen.append((name, self.current[-1]))
        return func(*args, **(kwargs or {}))


def _cache():
    c = V.PagedCache.__new__(V.PagedCache)
    c.page_size, c.page_table = 16, torch.full((2, 4), -1, dtype=torch.int32)
    c.ctx_len, c.bound, c.pages, c.free = torch.zeros(2, dtype=torch.int32), [0, 0], [[], []], list(range(8))
    return c


def test_cache_updates_on_the_given_stream(current):
    c, s = _cache(), FakeStream()
    with Asks(current) as asks:
        c.reserve(0, 40, stream=s)
        c.advance(torch.ones(2, dtype=torch.int32), stream=s)
        c.release(0, stream=s)
    at = [x for x in asks.seen if x[0] in ("__setitem__", "__iadd__", "to", "add_")]
    assert len(at) >= 4 and all(stream is s for _, stream in at), asks.seen


def test_served_step_on_the_given_stream(current, monkeypatch):
    s, calls = FakeStream(), []
    buf = S.StepBuffers(2, 2, 8, 6)
    buf.out_tokens = torch.tensor([[3, 4, -1], [-1, -1, -1]], dtype=torch.int32)
    buf.acc_len = torch.tensor([1, 0], dtype=torch.int32)

    def note(name):
        def call(*a, **k):
            stream = k.get("stream", a[-1] if a and isinstance(a[-1], FakeStream) else None)
            calls.append((name, stream if stream is not None else current[-1]))
        return call

    def run_step(inp, b, sps, target, *a, **k):
        note("run_step")(*a, **k)
        target(b)

    monkeypatch.setattr(S, "run_step", run_step)
    monkeypatch.setattr(B, "dspark_process_logits", note("rules"))
    monkeypatch.setattr(B, "dspark_history_commit", note("commit"))
    cache, inp = _cache(), dict(anchor=torch.tensor([5, 6], dtype=torch.int32))
    rules = V.LogitRules(hist=torch.zeros(2, 8, dtype=torch.int16), mask=note("mask"))
    with Asks(current) as asks:
        V.run_served_step(inp, buf, None, lambda b, c: note("forward")(), cache, rules, 0.0, 1, 0, stream=s)
    assert [n for n, _ in calls] == ["run_step", "forward", "mask", "rules", "commit"]
    assert all(stream is s for _, stream in calls), calls
    assert asks.seen and all(stream is s for _, stream in asks.seen), asks.seen
    assert inp["anchor"].tolist() == [4, 6] and cache.ctx_len.tolist() == [2, 0]
