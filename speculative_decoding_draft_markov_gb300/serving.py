"""The target model's side of a step: the paged cache that takes the packed windows, the rules on the packed
logits, the token history they read and the log probabilities that are reported, around step.run_step.

    cache = PagedCache(...); rules = LogitRules(...)
    run_served_step(inp, buf, sps, forward, cache, rules, ...)

`forward(buf, cache)` is the caller's model: it fills buf.packed from the packed ids, calling cache.attend for
each layer's attention.  Everything runs on one stream, torch's current one or the `stream` that is given (a torch
stream or a raw handle); forward and the rules' mask are called with it as the current one.  A cache's `reserve`,
`release` and `advance` are enqueued like the rest: they take the stream of the steps around them.  Nothing is
read back; pages are handed out on the host, from upper bounds of the lengths."""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import Callable, List, Optional

from . import binding as B
from . import step as S


def _on(stream):
    """What torch does in this context it does on `stream`."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def rotation_table(max_pos: int, rot: int, base: float = 10000.0, device="cuda"):
    """cos_sin [max_pos, rot] fp32 of dspark_append_kv: angle of (p, t) = p base^(-2 t / rot)."""
    import torch
    half = rot // 2
    inv = base ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


class PagedCache:
    """K and V of every layer in pages [n_pages, Hkv, page_size, D], one page table for all layers.

    ctx_len (device) counts each request's cached tokens; a step's windows are appended behind them and
    `advance` keeps what the verification accepted.  `bound` (host) is an upper bound of ctx_len: `reserve` raises it by a
    whole window each step, and only `settle` lowers it, by a length that has been read back.  Without it every
    rejected draft keeps its place and the cache fills too early; how late the length comes does not matter.  With a
    window, `settle` also gives back the pages that the window has left behind.

    eight_bit: pages of e4m3 with an exponent byte for each position's K and V of each KV head: half of the pages' memory.
    One pair of bf16 pages, `wide`, of one layer's size serves all layers: prompts are read back into it, and read_back
    leaves there what the packed rows see.  So L layers take 1/2 + 1/L of a 16-bit cache (and 1/(2 D) for the exponents).  A step
    reads half as much, which windows over 128-lane heads gain by (GB300: a third less time); over 64-lane heads, where the reads
    are not what bounds it, a step's attention can take longer than over 16 bits (64 windows of 64 rows to a KV head: 97 us, 84)."""

    def __init__(self, n_layers: int, n_pages: int, page_size: int, Hq: int, Hkv: int, D: int, bs: int, max_pages: int,
                 cos_sin, window: int = 0, n_sink: int = 0, interleaved: bool = False, device="cuda", eight_bit: bool = False):
        import torch
        shape = (n_pages, Hkv, page_size, D)

        def pages(dtype, n, last=D):
            bits = {torch.float8_e4m3fn: torch.uint8}.get(dtype, dtype)  # zeros of eight bits are zeros of e4m3
            return [torch.zeros(shape[:3] + (last,), dtype=bits, device=device).view(dtype) for _ in range(n)]

        dtype = torch.float8_e4m3fn if eight_bit else torch.bfloat16
        self.k, self.v = pages(dtype, n_layers), pages(dtype, n_layers)
        self.eight_bit = eight_bit
        if eight_bit:
            self.scale, self.wide = pages(torch.uint8, n_layers, 2), pages(torch.bfloat16, 2)
        self.page_size, self.Hq, self.window, self.n_sink = page_size, Hq, window, n_sink
        self.interleaved, self.cos_sin = interleaved, cos_sin
        self.page_table = torch.full((bs, max_pages), -1, dtype=torch.int32, device=device)
        self.ctx_len = torch.zeros(bs, dtype=torch.int32, device=device)
        self.bound: List[int] = [0] * bs
        self.pages: List[List[Optional[int]]] = [[] for _ in range(bs)]  # None: given back from behind the window
        self.free = list(range(n_pages - 1, -1, -1))
        self.ws = B.alloc_attention_workspace(Hq, Hkv, D, device)

    def reserve(self, r: int, tokens: int, stream=None) -> None:
        """Pages for `tokens` more of request r (host; raises when none are left)."""
        import torch
        first = len(self.pages[r])
        need = -(-(self.bound[r] + tokens) // self.page_size) - first
        if need > len(self.free) or first + max(need, 0) > self.page_table.shape[1]:
            raise RuntimeError("the paged cache is full")
        new = [self.free.pop() for _ in range(need)]
        if new:
            self.pages[r] += new
            with _on(stream):
                self.page_table[r, first:first + need] = torch.tensor(new, dtype=torch.int32).to(self.page_table.device)
        self.bound[r] += tokens

    def settle(self, r: int, length: int, since: int = 0, stream=None) -> None:
        """Request r had `length` tokens in the cache after some step (ctx_len, read back at any later time); `since`
        tokens were reserved for its steps after that one.  Lowers the bound to what that allows, and gives back the
        pages that lie between the sinks and the window of the next position, which no later row sees.  A length of a
        request that has been released since must not be passed; one beyond the bound is seen to be such and changes
        nothing."""
        if length < 0 or since < 0:
            raise ValueError("length and since must not be negative")
        if length > self.bound[r]:
            return
        self.bound[r] = min(self.bound[r], length + since)
        if not self.window:
            return
        # rows from position `length` on see j > length - window and j < n_sink
        pages, first = self.pages[r], -(-self.n_sink // self.page_size)
        gone = [i for i in range(first, min(max(0, length - self.window + 1) // self.page_size, len(pages)))
                if pages[i] is not None]
        if gone:
            self.free += [pages[i] for i in gone]
            for i in gone:
                pages[i] = None
            with _on(stream):
                self.page_table[r, gone[0]:gone[-1] + 1] = -1

    def release(self, r: int, stream=None) -> None:
        """Request r is done: its pages go back."""
        self.free += [p for p in self.pages[r] if p is not None]
        self.pages[r], self.bound[r] = [], 0
        with _on(stream):
            self.page_table[r] = -1
            self.ctx_len[r] = 0

    def attend(self, layer: int, q, k, v, cu_seqlens, max_rows: int, scale: float, out, stream=None,
               widen: bool = True) -> None:
        """Rotate and append the packed rows' q, k, v, then attend: out [rows, Hq, D].  `out` is the rotated
        queries' place as well.  widen (8 bits): whether what the rows see may be read back to `wide` first where max_rows is a
        prompt's; False for a prompt's chunk among many short windows, whose whole caches would be read back with it."""
        if self.eight_bit:
            pages = self.k[layer], self.v[layer], self.scale[layer]
            B.dspark_append_kv8(q, k, v, cu_seqlens, self.ctx_len, self.cos_sin, self.page_table, out, *pages, self.ws,
                                self.interleaved, stream)
            B.dspark_window_attention_kv8(out, *pages, self.page_table, cu_seqlens, self.ctx_len, max_rows, scale,
                                          self.window, self.n_sink, out, None, *(self.wide if widen else (None, None)), self.ws, stream)
            return
        B.dspark_append_kv(q, k, v, cu_seqlens, self.ctx_len, self.cos_sin, self.page_table, out, self.k[layer],
                           self.v[layer], self.ws, self.interleaved, stream)
        B.dspark_window_attention(out, self.k[layer], self.v[layer], self.page_table, cu_seqlens, self.ctx_len, max_rows,
                                  scale, self.window, self.n_sink, out, None, self.ws, stream)

    def read_back(self, layer: int, cu_seqlens, rows: int, stream=None):
        """bf16 pages k, v, numbered as the cache's, that hold what the packed rows (of `rows` in all) see of a layer: an
        8-bit cache's are `wide`, until the next layer that is read back or attends to a prompt."""
        if not self.eight_bit:
            return self.k[layer], self.v[layer]
        B.dspark_read_kv8(self.k[layer], self.v[layer], self.scale[layer], self.page_table, cu_seqlens, self.ctx_len, rows,
                          self.window, self.n_sink, self.page_table, *self.wide, self.ws, stream)
        return tuple(self.wide)

    def advance(self, tokens, stream=None) -> None:
        """Keep `tokens` [bs] (device int32) more of each request."""
        with _on(stream):
            self.ctx_len += tokens


@dataclasses.dataclass
class LogitRules:
    """What dspark_process_logits applies to the packed rows; None: that rule is off."""
    hist: "object" = None         # [bs, V] int16: build_history
    repetition: "object" = None   # [bs] fp32
    frequency: "object" = None
    presence: "object" = None
    bias_start: "object" = None   # [bs + 1], bias_ids, bias_vals: sorted ids per request
    bias_ids: "object" = None
    bias_vals: "object" = None
    mask: Optional[Callable] = None  # buf -> [rows, ceil(V / 32)] int32 words for the packed rows, or None

    def apply(self, buf, stream=None) -> None:
        """The rules on buf.packed, in place."""
        with _on(stream):
            B.dspark_process_logits(buf.packed, buf.cu, buf.ids, self.hist, self.repetition, self.frequency, self.presence,
                                    self.bias_start, self.bias_ids, self.bias_vals, self.mask(buf) if self.mask else None,
                                    buf.packed, buf.ws)


def _check_temperature(temperature: float) -> None:
    t = ctypes.c_float(temperature).value  # as dspark_token_logprobs takes it
    if not 0 < t < float("inf") or ctypes.c_float(2 / t).value == float("inf"):
        raise ValueError("temperature of the report must be positive (1 for the logits as they are)")


@dataclasses.dataclass
class Logprobs:
    """What a step reports of the tokens that it commits, by the target's logits under the rules at `temperature`: for
    out_tokens[r, j] its log probability, the entropy of its row, its rank, and the top_n likeliest ids.  Where
    out_tokens is -1: 0, 0, 0, and ids -1 with -infinity."""
    logprob: "object"        # [bs, gamma + 1] fp32
    entropy: "object"        # [bs, gamma + 1] fp32
    rank: "object"           # [bs, gamma + 1] int32, from 1
    top_ids: "object"        # [bs, gamma + 1, top_n] int32, or None
    top_logprobs: "object"   # [bs, gamma + 1, top_n] fp32, or None
    ws: "object"
    temperature: float = 1.0

    @staticmethod
    def allocate(bs: int, gamma: int, V: int, top_n: int = 0, temperature: float = 1.0, device="cuda") -> "Logprobs":
        import torch
        _check_temperature(temperature)
        f32, i32 = dict(dtype=torch.float32, device=device), dict(dtype=torch.int32, device=device)
        n = gamma + 1
        return Logprobs(torch.zeros((bs, n), **f32), torch.zeros((bs, n), **f32), torch.zeros((bs, n), **i32),
                        torch.full((bs, n, top_n), -1, **i32) if top_n else None,
                        torch.full((bs, n, top_n), float("-inf"), **f32) if top_n else None,
                        B.alloc_logprobs_workspace(bs * n, V, top_n, device), temperature)

    def check(self, buf) -> None:
        """Raises where `take` could not report of buf's steps."""
        if self.logprob.shape != buf.out_tokens.shape:
            raise ValueError("logprobs must be of the step's requests and gamma")
        _check_temperature(self.temperature)
        top_n = 0 if self.top_ids is None else self.top_ids.shape[2]
        n = B.dspark_token_logprobs_workspace_bytes(self.logprob.numel(), buf.packed.shape[1], top_n)
        if n == 0 or self.ws.numel() < n:
            raise ValueError("logprobs must be of the step's vocabulary")

    def take(self, buf, stream=None) -> None:
        """Of buf.out_tokens, after a verification and before buf.packed is written anew."""
        with _on(stream):
            B.dspark_token_logprobs(buf.packed, buf.cu, buf.out_tokens, self.temperature, self.logprob, self.entropy,
                                    self.rank, self.top_ids, self.top_logprobs, self.ws)


def build_history(rules: LogitRules, prompts, V: int, ws, device="cuda", stream=None) -> None:
    """rules.hist from the prompts (host lists of ids); the last id of a prompt, the first step's anchor, is in it."""
    import torch
    start = [0]
    for p in prompts:
        start.append(start[-1] + len(p))
    i32 = dict(dtype=torch.int32, device=device)
    with _on(stream):
        rules.hist = torch.empty((len(prompts), V), dtype=torch.int16, device=device)
        B.dspark_history_build(torch.tensor([t for p in prompts for t in p], **i32), torch.tensor(start, **i32),
                               torch.tensor([len(p) for p in prompts], **i32), rules.hist, ws)


def take_outcome(inp: dict, buf: S.StepBuffers, cache: PagedCache, rules: LogitRules, stream=None) -> None:
    """After a verification: history, cache lengths and anchors (inp["anchor"]) take its outcome.
    A request whose deciding row allows nothing keeps its anchor and adds no token."""
    import torch
    with _on(stream):
        if rules.hist is not None:
            B.dspark_history_commit(buf.out_tokens, rules.hist, buf.ws)
        last = buf.out_tokens.gather(1, buf.acc_len.long()[:, None])[:, 0]
        dead = last < 0  # the anchor stays the last token: only the accepted ones before it are cached for good
        before = torch.where(buf.acc_len > 0, buf.out_tokens.gather(1, (buf.acc_len.long() - 1).clamp(min=0)[:, None])[:, 0],
                             inp["anchor"])
        inp["anchor"].copy_(torch.where(dead, before, last))
        cache.advance(buf.acc_len + (~dead).to(torch.int32))


def run_served_step(inp: dict, buf: S.StepBuffers, sps, forward: Callable, cache: PagedCache, rules: LogitRules,
                    temperature: float, seed: int, step: int, mode: int = B.DSPARK_COMPACT, tiers=None,
                    stream=None, sched_mode: int = B.DSPARK_SCHED_EARLY_STOP, ring=None, side_stream=None,
                    logprobs: Optional[Logprobs] = None) -> None:
    """One step: draft, schedule and pack; the target forward over the packed windows, its logits under the
    rules; the verification; with `logprobs` its report; then take_outcome.  mode, tiers, sched_mode, ring and side_stream as in step.run_step.
    A drafter that step.run_step does not run (the RNN head) takes the same way by hand: its draft and the pack,
    forward, rules.apply, step.verify with its states, take_outcome."""
    if logprobs is not None:
        logprobs.check(buf)

    def target(b: S.StepBuffers) -> None:
        forward(b, cache)
        rules.apply(b)

    with _on(stream):
        S.run_step(inp, buf, sps, target, temperature, seed, step, mode, sched_mode, tiers, ring=ring, side_stream=side_stream)
        if logprobs is not None:
            logprobs.take(buf)
        take_outcome(inp, buf, cache, rules)
