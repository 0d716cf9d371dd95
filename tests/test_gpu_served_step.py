"""The target-side operators together, as examples/served_step.py uses them: speculative decoding over the paged
cache gives the tokens that the target model alone gives, one at a time, without a cache."""
import math
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _plain_logits(model, tokens, window, n_sink):
    """The model over a whole sequence with elementary operations in 32 bits: the last row's logits."""
    from tests.serving_reference import rotate
    n = len(tokens)
    x = model.embed[torch.tensor(tokens, device="cuda")].float()
    inv = 10000.0 ** (-np.arange(model.D // 2) / (model.D // 2))
    ang = np.arange(n)[:, None] * inv
    cos, sin = np.cos(ang)[:, None], np.sin(ang)[:, None]
    p = torch.arange(n, device="cuda")
    seen = (p[None] <= p[:, None]) & ((p[None] > p[:, None] - window) | (p[None] < n_sink))
    g = model.Hq // model.Hkv
    for i in range(model.layers):
        nx = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        qkv = (nx @ model.qkv[i].float().T).view(n, -1, model.D)
        q, k, v = qkv.split([model.Hq, model.Hkv, model.Hkv], 1)
        q, k = (torch.from_numpy(rotate(t.cpu().numpy(), cos, sin, False)).float().cuda() for t in (q, k))
        s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(g, 1)) / math.sqrt(model.D)
        w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        o = torch.einsum("hij,jhd->ihd", w, v.repeat_interleave(g, 1))
        x = x + o.reshape(n, -1) @ model.o[i].float().T
    x = x[-1:]
    nx = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return (nx @ model.head.float().T)[0].cpu().numpy().astype(np.float64)


def _rules(l, prompt, said):
    """Penalties, biases and mask of the example on one row, plainly."""
    V = l.size
    count = np.bincount(said, minlength=V) if said else np.zeros(V, int)
    seen = (count > 0) | np.isin(np.arange(V), prompt)
    l = np.where(seen, np.where(l > 0, l / 1.2, l * 1.2), l) - 0.3 * count - 0.2 * (count > 0)
    l[3] += 2.0
    l[70] -= 5.0
    l[::7] = -np.inf
    return l


def test_greedy_served_steps_equal_the_target_alone():
    import served_step as E
    steps = 12
    prompts, said, made = E.generate(steps=steps, temperature=0.0)
    model, _, cache, rules, _, buf, _ = made
    lens = cache.ctx_len.tolist()
    hist = rules.hist.cpu().numpy().astype(np.int64)
    total = 0
    for r, prompt in enumerate(prompts):
        assert len(said[r]) >= steps and lens[r] == len(prompt) - 1 + len(said[r])
        # the history holds the prompt and every token that was given out
        assert np.array_equal(hist[r] & 0x7FFF, np.bincount(said[r], minlength=model.vocab))
        assert np.array_equal(np.nonzero(hist[r] < 0)[0], np.unique(prompt))
        for i in range(len(said[r])):
            l = _rules(_plain_logits(model, prompt + said[r][:i], 48, 4), prompt, said[r][:i])
            # the served logits are bf16 (values up to about 16: steps of 1/16) after bf16 layers: the token
            # given out is the best one up to that
            assert l[said[r][i]] >= l.max() - 0.35, (r, i, l[said[r][i]], l.max())
            total += 1
    assert total > steps * len(prompts)  # some drafts were accepted
    assert len(set(sum(said, []))) > 10   # and what was said is no loop of a token


def test_sampled_served_steps_keep_to_the_mask():
    import served_step as E
    prompts, said, made = E.generate(steps=10, temperature=1.0, window=20, n_sink=0)
    for s in said:
        assert len(s) >= 10 and all(x % 7 for x in s)
    # the example's run is reproducible: same seeds, same tokens
    _, again, _ = E.generate(steps=10, temperature=1.0, window=20, n_sink=0)
    assert again == said


def test_a_mask_that_allows_nothing_keeps_the_request_where_it_is():
    import served_step as E
    from speculative_decoding_draft_markov_gb300 import serving as V
    model, prompts, cache, rules, inp, buf, sps = E.set_up()
    keep = rules.mask
    dead = torch.zeros(buf.packed.shape[0], (model.vocab + 31) // 32, dtype=torch.int32, device="cuda")
    for r in range(len(prompts)):
        cache.reserve(r, 2 * (buf.gamma + 1))
    before, anchor = cache.ctx_len.clone(), inp["anchor"].clone()
    hist = rules.hist.clone()
    rules.mask = lambda b: dead
    for temperature in (0.0, 1.0):
        V.run_served_step(inp, buf, sps, model.forward, cache, rules, temperature, 5, 0)
        assert (buf.out_tokens == -1).all() and torch.equal(cache.ctx_len, before)
        assert torch.equal(inp["anchor"], anchor) and torch.equal(rules.hist, hist)
    rules.mask = keep
    V.run_served_step(inp, buf, sps, model.forward, cache, rules, 0.0, 5, 1)
    assert (cache.ctx_len > before).all() and (inp["anchor"] >= 0).all()


def test_cache_pages():
    from speculative_decoding_draft_markov_gb300 import serving as V
    c = V.PagedCache(1, 5, 16, 2, 1, 64, 2, 4, V.rotation_table(64, 64))
    c.reserve(0, 17)
    c.reserve(1, 16)
    c.reserve(0, 15)
    assert len(c.pages[0]) == 2 and len(c.pages[1]) == 1 and len(c.free) == 2
    assert sorted(c.pages[0] + c.pages[1] + c.free) == list(range(5))
    with pytest.raises(RuntimeError):
        c.reserve(1, 49)  # beyond the table
    with pytest.raises(RuntimeError):
        c.reserve(0, 33)  # beyond the pages
    c.release(0)
    assert len(c.free) == 4 and (c.page_table[0] == -1).all()
