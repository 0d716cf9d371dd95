"""Served steps on a side stream give what they give on the current one, however far that stream lags behind."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_side_stream(raw):
    import served_step as E
    from speculative_decoding_draft_markov_gb300 import serving as V
    steps, got = 6, []
    for side in (None, torch.cuda.Stream()):
        model, prompts, cache, rules, inp, buf, sps = E.set_up()
        torch.cuda.synchronize()
        stream = side.cuda_stream if side is not None and raw else side
        said = []
        for t in range(steps):
            for r in range(len(prompts)):
                cache.reserve(r, buf.gamma + 1, stream=stream)
            if side is not None:
                with torch.cuda.stream(side):
                    torch.cuda._sleep(2_000_000)  # about a millisecond: what runs elsewhere would run before this step
            V.run_served_step(inp, buf, sps, model.forward, cache, rules, 1.0, 5, t, stream=stream)
            if side is not None:
                side.synchronize()
            said.append(buf.out_tokens.tolist())
        torch.cuda.synchronize()
        got.append((said, cache.ctx_len.tolist(), inp["anchor"].tolist(), cache.page_table.tolist()))
    assert got[0] == got[1]
