"""The served step with each scheduler and mode of the step, and with the recurrent drafter by hand: what is said follows
the mask and is what history, lengths and anchors say."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import serving as V  # noqa: E402
from speculative_decoding_draft_markov_gb300 import step as S  # noqa: E402

pytestmark = pytest.mark.gpu


def _rnn_step(model, cache, rules, inp, buf, temperature, t, head):
    """The recurrent head's draft, then the same way as run_served_step."""
    Wg, bg, states = head
    B.dspark_draft_block_rnn(inp["U"], inp["W1"], inp["W2t"], Wg, bg, inp["anchor"], temperature, 5, t, buf.tokens, buf.logit_x,
                             buf.lse, states, buf.ws)
    B.dspark_pack(None, inp["anchor"], buf.tokens, None, buf.cu, buf.ids, buf.req, buf.pos, buf.padded, buf.ws)
    model.forward(buf, cache)
    rules.apply(buf)
    S.verify(inp, buf, temperature, 5, t, B.DSPARK_STATIC, states=states)
    V.take_outcome(inp, buf, cache, rules)


@pytest.mark.parametrize("temperature", [0.0, 1.0])
@pytest.mark.parametrize("how", ["early_stop", "argmax", "zos", "zos_side", "static", "cap_accept", "tiers", "rnn"])
def test_schedulers(how, temperature):
    import served_step as E
    model, prompts, cache, rules, inp, buf, sps = E.set_up(max_tokens=200)
    side = torch.cuda.Stream() if how == "zos_side" else None
    more = dict(early_stop={}, argmax=dict(sched_mode=B.DSPARK_SCHED_GLOBAL_ARGMAX), static=dict(mode=B.DSPARK_STATIC),
                cap_accept=dict(mode=B.DSPARK_CAP_ACCEPT), tiers=dict(tiers=torch.tensor([4, 8, 16], dtype=torch.int32, device="cuda")),
                zos=dict(ring=S.zos_ring()), zos_side=dict(ring=S.zos_ring(), side_stream=side)).get(how)
    if how == "rnn":
        r = inp["W1"].shape[1]
        g = torch.Generator(device="cuda")
        g.manual_seed(54)
        head = ((torch.randn(2 * r, r, generator=g, device="cuda") * 0.05).to(torch.bfloat16),
                torch.zeros(r, device="cuda"), torch.zeros(len(prompts), buf.gamma, r, dtype=torch.bfloat16, device="cuda"))
    said = [[] for _ in prompts]
    for t in range(8):
        for i in range(len(prompts)):
            cache.reserve(i, buf.gamma + 1)
        if how == "rnn":
            _rnn_step(model, cache, rules, inp, buf, temperature, t, head)
        else:
            V.run_served_step(inp, buf, sps, model.forward, cache, rules, temperature, 5, t, **more)
        for i, row in enumerate(buf.out_tokens.tolist()):
            said[i] += [x for x in row if x >= 0]
    assert B.dspark_read_device_status(buf.ws) == B.DSPARK_OK and B.dspark_read_device_status(cache.ws) == B.DSPARK_OK
    hist, lens, anchors = rules.hist.cpu().numpy().astype(np.int64), cache.ctx_len.tolist(), inp["anchor"].tolist()
    for i, (p, s) in enumerate(zip(prompts, said)):
        assert len(s) >= 8 and all(x % 7 for x in s)
        assert lens[i] == len(p) - 1 + len(s) and anchors[i] == s[-1]
        assert np.array_equal(hist[i] & 0x7FFF, np.bincount(s, minlength=model.vocab))
