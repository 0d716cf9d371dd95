"""A report of log probabilities that could not be taken is refused before anything of the step has run (no GPU), and the step's
state stays as it was (GPU)."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import build as _build  # noqa: E402
from speculative_decoding_draft_markov_gb300 import serving as V  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture
def buf():
    _build.build()

    class Buf:
        packed, cu = torch.zeros(8, 64), torch.tensor([0, 4, 8], dtype=torch.int32)
        out_tokens = torch.zeros(2, 4, dtype=torch.int32)
    return Buf


def _step(buf, report):
    V.run_served_step({}, buf, None, None, None, None, 1.0, 0, 0, logprobs=report)  # with nothing to run on


@pytest.mark.parametrize("temperature", [0.0, -1.0, float("inf"), float("nan"), 1e-39, 1e39, 1e-46])
def test_a_temperature_that_was_changed(buf, temperature):
    report = V.Logprobs.allocate(2, 3, 64, 4, device="cpu")
    report.temperature = temperature
    with pytest.raises(ValueError, match="temperature"):
        _step(buf, report)
    with pytest.raises(ValueError, match="temperature"):
        V.Logprobs.allocate(2, 3, 64, 4, temperature, device="cpu")


def test_a_workspace_of_another_vocabulary(buf, monkeypatch):
    monkeypatch.setattr(B, "dspark_token_logprobs_workspace_bytes", lambda items, vocab, top_n: items * vocab * (1 + top_n))
    report = V.Logprobs.allocate(2, 3, 56, 4, device="cpu")
    with pytest.raises(ValueError, match="vocabulary"):
        _step(buf, report)
    report.check(type("Buf", (buf,), dict(packed=torch.zeros(8, 56))))
    report.check(type("Buf", (buf,), dict(packed=torch.zeros(8, 48))))  # a larger workspace does


def test_a_vocabulary_that_the_call_refuses(buf):
    with pytest.raises(ValueError, match="vocabulary"):
        _step(type("Buf", (buf,), dict(packed=torch.zeros(8, 60))), V.Logprobs.allocate(2, 3, 64, 4, device="cpu"))


def test_what_fits_passes(buf):
    for top in (0, 4):
        V.Logprobs.allocate(2, 3, 64, top, 0.7, device="cpu").check(buf)


@pytest.mark.gpu
def test_nothing_has_run_when_a_report_is_refused():
    """One request, so that the workspace goes by the vocabulary: the cache's lengths, the anchors and the history stay."""
    import served_step as E
    _, _, made = E.generate(steps=1, temperature=0.0, bs=1)
    model, _, cache, rules, inp, step, sps = made
    small = V.Logprobs.allocate(1, step.gamma, 64, 5)
    assert small.ws.numel() < B.dspark_token_logprobs_workspace_bytes(step.gamma + 1, 152064, 5)
    kept = [t.clone() for t in (cache.ctx_len, inp["anchor"], rules.hist, step.out_tokens)]
    cold = V.Logprobs.allocate(1, step.gamma, model.vocab, 5)
    cold.temperature = 0.0
    wide = type("Buf", (), dict(packed=torch.zeros(step.gamma + 1, 152064, device="cuda"), out_tokens=step.out_tokens))
    with pytest.raises(ValueError, match="vocabulary"):
        V.run_served_step(inp, wide, sps, model.forward, cache, rules, 0.0, 5, 1, logprobs=small)
    with pytest.raises(ValueError, match="temperature"):
        V.run_served_step(inp, step, sps, model.forward, cache, rules, 0.0, 5, 1, logprobs=cold)
    assert all(torch.equal(a, b) for a, b in zip(kept, (cache.ctx_len, inp["anchor"], rules.hist, step.out_tokens)))
