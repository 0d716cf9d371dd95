"""The served step over an 8-bit cache, with its report: greedy tokens are the target's own over a cache of that kind, and the
reported log probabilities are those of the logits that were verified."""
import math
import os
import sys

import numpy as np
import pytest

from tests import kv8_reference as K

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _plain_logits(model, tokens, window, n_sink):
    """The model over a whole sequence with elementary operations, K and V quantised: the last row's logits."""
    from tests.serving_reference import rotate
    n = len(tokens)
    x = model.embed[torch.tensor(tokens, device="cuda")].float()
    inv = 10000.0 ** (-np.arange(model.D // 2) / (model.D // 2))
    ang = np.arange(n)[:, None] * inv
    cos, sin = np.cos(ang)[:, None], np.sin(ang)[:, None]
    p = torch.arange(n, device="cuda")
    seen = (p[None] <= p[:, None]) & ((p[None] > p[:, None] - window) | (p[None] < n_sink))
    g = model.Hq // model.Hkv

    def quantised(t):
        byte = K.exponent_byte(t)
        return K.values(K.codes(t, byte), byte)

    for i in range(model.layers):
        nx = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        qkv = (nx.to(torch.bfloat16) @ model.qkv[i].T).view(n, -1, model.D)
        q, k, v = (t.float().cpu().numpy().astype(np.float64) for t in qkv.split([model.Hq, model.Hkv, model.Hkv], 1))
        q, k = rotate(q, cos, sin, False), rotate(k, cos, sin, False)
        q, k, v = (torch.from_numpy(t).float().cuda() for t in (q, quantised(k), quantised(v)))
        s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(g, 1)) / math.sqrt(model.D)
        w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        o = torch.einsum("hij,jhd->ihd", w, v.repeat_interleave(g, 1))
        x = x + o.reshape(n, -1) @ model.o[i].float().T
    x = x[-1:]
    nx = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return (nx @ model.head.float().T)[0].cpu().numpy().astype(np.float64)


def test_greedy_served_steps_equal_the_target_alone():
    import served_step as E
    from tests.test_gpu_served_step import _rules
    steps = 8
    prompts, said, made = E.generate(steps=steps, temperature=0.0, eight_bit=True)
    model, _, cache, _, _, _, _ = made
    assert cache.k[0].dtype == torch.float8_e4m3fn
    lens = cache.ctx_len.tolist()
    total = 0
    for r, prompt in enumerate(prompts):
        assert len(said[r]) >= steps and lens[r] == len(prompt) - 1 + len(said[r])
        for i in range(len(said[r])):
            l = _rules(_plain_logits(model, prompt + said[r][:i], 48, 4), prompt, said[r][:i])
            # bf16 logits (steps of 1/16) after bf16 layers, and values that lie at a border of two codes may take the other:
            # the token given out is the best one up to that
            assert l[said[r][i]] >= l.max() - 0.5, (r, i, l[said[r][i]], l.max())
            total += 1
    assert total > steps * len(prompts)  # some drafts were accepted


@pytest.mark.parametrize("eight_bit", [False, True])
@pytest.mark.parametrize("temperature,top", [(0.0, 5), (1.0, 0)])
def test_the_report_is_of_the_logits_that_were_verified(eight_bit, temperature, top):
    import served_step as E
    seen = []

    def look(buf, report):
        x, cu, out = buf.packed.float().cpu().numpy().astype(np.float64), buf.cu.tolist(), buf.out_tokens.tolist()
        lp, ent, rank = report.logprob.tolist(), report.entropy.tolist(), report.rank.tolist()
        for r, row in enumerate(out):
            for j, t in enumerate(row):
                if t < 0:
                    assert lp[r][j] == 0 and rank[r][j] == 0
                    continue
                want = K.token_logprobs(x[cu[r] + j], t, 1.0, top)
                np.testing.assert_allclose([lp[r][j], ent[r][j]], want[:2], rtol=1e-5, atol=5e-5)
                assert rank[r][j] == want[2] and (temperature > 0 or rank[r][j] == 1)
                if top:
                    assert report.top_ids[r, j].tolist() == want[3].tolist()
                seen.append(t)

    _, said, _ = E.generate(steps=5, temperature=temperature, logprobs=top, on_step=look, eight_bit=eight_bit)
    assert len(seen) == sum(map(len, said)) > 20


def test_reading_a_layer_back():
    """What read_back leaves is what the rows see, as 64 bits of the codes give it; a 16-bit cache gives its own pages."""
    import served_step as E
    from speculative_decoding_draft_markov_gb300 import binding as B
    prompts, said, made = E.generate(steps=3, temperature=0.0, window=0, n_sink=0, eight_bit=True)
    _, _, cache, _, _, _, _ = made
    lens = cache.ctx_len.tolist()
    cu = torch.arange(len(prompts) + 1, dtype=torch.int32, device="cuda")
    keep = cache.ctx_len.clone()
    cache.ctx_len -= 1  # the last position's row
    for layer in range(len(cache.k)):
        k, v = cache.read_back(layer, cu, len(prompts))
        assert B.dspark_read_device_status(cache.ws) == B.DSPARK_OK
        for r, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            pages = cache.page_table[r].long()[pos // cache.page_size]
            for got, codes, which in ((k, cache.k[layer], 0), (v, cache.v[layer], 1)):
                at = pages.cpu().numpy(), slice(None), (pos % cache.page_size).cpu().numpy()
                want = K.values(codes.view(torch.uint8).cpu().numpy()[at], cache.scale[layer].cpu().numpy()[at + (which,)])
                assert np.array_equal(got.float().cpu().numpy()[at], want)
    cache.ctx_len.copy_(keep)
    _, _, made = E.generate(steps=1, temperature=0.0)
    assert made[2].read_back(1, cu, 4) == (made[2].k[1], made[2].v[1])


def test_the_example_runs():
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, os.path.join(root, "examples", "served_step.py"), "--steps", "2", "--eight-bit", "--top", "3"],
                         capture_output=True, text=True)
    assert out.returncode == 0 and "likeliest" in out.stdout, out.stderr[-500:]
