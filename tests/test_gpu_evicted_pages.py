"""Long generation in a paged cache that holds only the windows: pages that were given back and taken again by other
requests change nothing."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_small_cache_says_what_a_large_one_says():
    import served_step as E
    from speculative_decoding_draft_markov_gb300 import serving as V
    steps, got = 90, []
    for small in (False, True):
        model, prompts, cache, rules, inp, buf, sps = E.set_up(window=48, n_sink=4)
        if small:  # four windows of 48 with their sinks, pages at their ends and room for a step
            keep = 4 * 7
            held = {p for q in cache.pages for p in q}
            cache.free = [p for p in cache.free if p not in held][:keep - len(held)]
        said = [[] for _ in prompts]
        for t in range(steps):
            for r in range(len(prompts)):
                cache.reserve(r, buf.gamma + 1)
            V.run_served_step(inp, buf, sps, model.forward, cache, rules, 1.0, 5, t)
            lens = cache.ctx_len.tolist()
            for r, row in enumerate(buf.out_tokens.tolist()):
                said[r] += [x for x in row if x >= 0]
                if small:
                    cache.settle(r, lens[r])
                else:
                    cache.bound[r] = lens[r]
        got.append((said, lens))
        if small:
            assert sum(lens) > 28 * cache.page_size  # more than those pages hold
    assert got[0] == got[1]
