"""Speculative decoding over a paged cache: a small target model with random weights, its attention on the
paged cache with a sliding window and sinks, penalties, a bias and a mask on its logits, and the verification.

    python examples/served_step.py [--steps N] [--temperature T] [--eight-bit] [--top N]

With --eight-bit the cache's pages are of 8 bits; with --top the log probability, rank and N likeliest alternatives
of each token are reported.  The target is a stack of attention layers (no feed-forward parts: the cache and the attention are what is
shown).  The drafter sees no context: its base logits U are 0 and its Markov term is the target's head on the
previous token's embedding, in low rank; some drafts are accepted, some are not."""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import serving as V  # noqa: E402
from speculative_decoding_draft_markov_gb300 import step as S  # noqa: E402


class SmallTarget:
    """Embedding, layers of norm -> attention -> residual, head; bf16 weights."""

    def __init__(self, vocab=2048, width=256, layers=2, Hq=4, Hkv=2, D=64, seed=1, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def w(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).to(torch.bfloat16)

        self.vocab, self.layers, self.Hq, self.Hkv, self.D = vocab, layers, Hq, Hkv, D
        self.embed, self.head = w(vocab, width, std=1.0), w(vocab, width, std=3.0 * width ** -0.5)
        self.qkv = [w((Hq + 2 * Hkv) * D, width, std=width ** -0.5) for _ in range(layers)]
        self.o = [w(width, Hq * D, std=(Hq * D) ** -0.5) for _ in range(layers)]

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def logits(self, ids, attend):
        """ids [rows]; attend(layer, q, k, v) -> [rows, Hq, D]: logits [rows, vocab] in bf16 (std about 3)."""
        x = self.embed[ids.clamp(min=0).long()]
        for i in range(self.layers):
            qkv = (self.norm(x) @ self.qkv[i].T).view(-1, self.Hq + 2 * self.Hkv, self.D)
            q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], 1)
            x = x + attend(i, q, k, v).reshape(-1, self.Hq * self.D) @ self.o[i].T
        return self.norm(x) @ self.head.T

    def forward(self, buf, cache):
        """The packed batch of a step (serving.run_served_step's forward)."""
        rows = buf.ids.shape[0]
        out = torch.zeros(rows, self.Hq, self.D, dtype=torch.bfloat16, device=buf.ids.device)

        def attend(i, q, k, v):
            cache.attend(i, q, k, v, buf.cu, buf.gamma + 1, self.D ** -0.5, out)
            return out

        buf.packed.copy_(self.logits(buf.ids, attend))

    def prefill(self, cache, prompts, ws):
        """All of each prompt but its last token (the first anchor) into the cache."""
        n = [len(p) - 1 for p in prompts]
        i32 = dict(dtype=torch.int32, device=cache.ctx_len.device)
        ids = torch.tensor([t for p in prompts for t in p[:-1]], **i32)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), **i32)
        out = torch.zeros(len(ids), self.Hq, self.D, dtype=torch.bfloat16, device=ids.device)

        def attend(i, q, k, v):
            cache.attend(i, q, k, v, cu, max(max(n), 1), self.D ** -0.5, out)
            return out

        if len(ids):
            self.logits(ids, attend)
        cache.advance(torch.tensor(n, **i32))


def set_up(bs=4, gamma=3, seed=3, window=48, n_sink=4, max_tokens=400, device="cuda", eight_bit=False):
    """A target, a cache with the prompts in it, rules, and the step's inputs and buffers."""
    rng = np.random.default_rng(seed)
    model = SmallTarget(device=device)
    prompts = [list(map(int, rng.integers(0, model.vocab, 5 + 23 * r))) for r in range(bs)]
    page = 16
    max_pages = -(-(max_tokens + 2 * gamma) // page)
    cache = V.PagedCache(model.layers, bs * max_pages, page, model.Hq, model.Hkv, model.D, bs, max_pages,
                         V.rotation_table(max_tokens + 2 * gamma, model.D, device=device), window, n_sink, device=device,
                         eight_bit=eight_bit)
    buf = S.StepBuffers.allocate(bs, gamma, model.vocab, bs * (gamma + 1), torch.bfloat16, device)
    f32 = dict(dtype=torch.float32, device=device)
    i32 = dict(dtype=torch.int32, device=device)
    rules = V.LogitRules(
        repetition=torch.full((bs,), 1.2, **f32), frequency=torch.full((bs,), 0.3, **f32),
        presence=torch.full((bs,), 0.2, **f32), bias_start=torch.arange(bs + 1, **i32) * 2,
        bias_ids=torch.tensor([3, 70], **i32).repeat(bs), bias_vals=torch.tensor([2.0, -5.0], **f32).repeat(bs))
    # ids divisible by 7 are forbidden to everyone
    allowed = torch.arange((model.vocab + 31) // 32 * 32, device=device) % 7 != 0
    words = (allowed.view(-1, 32).long() << torch.arange(32, device=device)).sum(1)
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    rules.mask = lambda b: mask.expand(b.packed.shape[0], -1).contiguous()
    V.build_history(rules, prompts, model.vocab, buf.ws, device)
    for r, p in enumerate(prompts):
        cache.reserve(r, len(p) - 1)
    model.prefill(cache, prompts, buf.ws)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r, d = model.embed.shape[1], 64
    # l = W1[x] . W2: the target without its attention
    w1, w2t = model.norm(model.embed), model.head
    inp = dict(U=torch.zeros(bs, gamma, model.vocab, dtype=torch.bfloat16, device=device), W1=w1, W2t=w2t,
               anchor=torch.tensor([p[-1] for p in prompts], **i32),
               h=torch.randn(bs, gamma, d, generator=g, device=device).to(torch.bfloat16),
               w=torch.randn(d + r, generator=g, device=device) * 0.05, b=1.0, sts_T=torch.ones(gamma, **f32))
    T_raw = 1.0 + 0.01 * np.arange(bs * (gamma + 1) + 1)
    return model, prompts, cache, rules, inp, buf, S.sps_table(T_raw, np.zeros(0, np.int32), device)


def generate(steps=20, temperature=0.0, seed=5, logprobs=None, on_step=None, **kw):
    """`steps` served steps; returns the prompts, what was generated for each and the set-up.  on_step(buf, logprobs) is
    called after each step; logprobs: how many alternatives to report, or None."""
    made = set_up(**kw)
    model, prompts, cache, rules, inp, buf, sps = made
    report = None if logprobs is None else V.Logprobs.allocate(len(prompts), buf.gamma, model.vocab, logprobs,
                                                               device=buf.packed.device)
    said = [[] for _ in prompts]
    for t in range(steps):
        for r in range(len(prompts)):
            cache.reserve(r, buf.gamma + 1)
        V.run_served_step(inp, buf, sps, model.forward, cache, rules, temperature, seed, t, logprobs=report)
        if on_step:
            on_step(buf, report)
        out, lens = buf.out_tokens.tolist(), cache.ctx_len.tolist()
        for r, row in enumerate(out):
            said[r] += [x for x in row if x >= 0]
            cache.settle(r, lens[r])  # the exact length is known here: fewer pages are needed next
    status = B.dspark_read_device_status(buf.ws) or B.dspark_read_device_status(cache.ws)
    if report is not None:
        status = status or B.dspark_read_device_status(report.ws)
    if status != B.DSPARK_OK:
        raise B.DSparkError(status, "served step")
    return prompts, said, made


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--eight-bit", action="store_true")
    ap.add_argument("--top", type=int, default=None)
    a = ap.parse_args()
    reported = []

    def note(buf, report):
        if report is not None:
            reported.append([x.tolist() for x in (buf.out_tokens, report.logprob, report.rank)])

    prompts, said, made = generate(a.steps, a.temperature, logprobs=a.top, on_step=note, eight_bit=a.eight_bit)
    for r, s in enumerate(said):
        print(f"request {r}: prompt of {len(prompts[r])} tokens, {len(s)} tokens in {a.steps} steps "
              f"({len(s) / a.steps:.2f} a step): {s[:12]} ...")
        if reported:
            tokens, lp, rank = ([x for step in reported for x in step[k][r]] for k in range(3))
            kept = [i for i, t in enumerate(tokens) if t >= 0]
            print(f"  mean log probability {sum(lp[i] for i in kept) / len(kept):.3f}, "
                  f"{sum(rank[i] == 1 for i in kept)} of {len(kept)} the likeliest")
