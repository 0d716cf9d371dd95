"""Cases of the 8-bit paged cache and of the log probabilities that a server reports: the append that
quantises what it writes, the windows' attention over that cache, reading it back to 16 bits, and the
log probabilities, entropies and top alternatives of the tokens that a step committed.

A cache slot holds one position's K and V of one KV head: D values of e4m3 each, and for each of the two one
power of two (an exponent byte, biased by 127; 255: the whole vector is NaN).

Every case gives sizes only.  Lengths are drawn from the case itself (so that its work is fixed),
values from the seed.  Rows are packed as the step packs them: request r owns rows
cu[r] .. cu[r+1]-1, its row i sits at position ctx[r] + i of its sequence."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one chat: the smallest call of a decoding loop, all latency
        dict(name="append8_one_token", op="append", bs=1, rows_lo=1, rows_hi=1, ctx_lo=777, ctx_hi=777, hq=32, hkv=8,
             d=128, page=16, rot=128, interleaved=False),
        # three prompts taken in at once, about 8000 tokens together, half of each head rotated
        dict(name="append8_prompts", op="append", bs=3, rows_lo=2400, rows_hi=3000, ctx_lo=1, ctx_hi=999, hq=32, hkv=8,
             d=128, page=64, rot=64, interleaved=True),
        # one token of one chat over its whole short context
        dict(name="attn8_one_token", op="attention", bs=1, rows_lo=1, rows_hi=1, ctx_lo=1500, ctx_hi=1500, hq=32,
             hkv=8, d=128, page=16, window=0, sinks=0),
        # a served batch with contexts from short to long; pruned windows of 1 to 8 rows
        dict(name="attn8_verify_64", op="attention", bs=64, rows_lo=1, rows_hi=8, ctx_lo=1000, ctx_hi=32000, hq=64,
             hkv=8, d=64, page=32, window=4096, sinks=4),
        # the benchmark's batch: 256 requests, the whole block of gamma = 7 verified
        dict(name="attn8_verify_256", op="attention", bs=256, rows_lo=8, rows_hi=8, ctx_lo=500, ctx_hi=6000, hq=32,
             hkv=8, d=128, page=64, window=1024, sinks=4),
        # two long documents, a block of gamma = 15, every position visible: what an 8-bit cache is for
        dict(name="attn8_long_2", op="attention", bs=2, rows_lo=16, rows_hi=16, ctx_lo=120001, ctx_hi=131000, hq=32,
             hkv=8, d=128, page=128, window=0, sinks=0),
        # two chunks of prompts, about 8000 tokens, over what is cached already
        dict(name="attn8_prompts", op="attention", bs=2, rows_lo=3700, rows_hi=4300, ctx_lo=1000, ctx_hi=5000, hq=32,
             hkv=8, d=128, page=64, window=4096, sinks=4),
        # one request's cache handed to a reader of 16-bit pages
        dict(name="read8_one", op="read", bs=1, rows_lo=1, rows_hi=1, ctx_lo=1200, ctx_hi=1200, hq=32, hkv=8, d=128,
             page=16, window=0, sinks=0),
        # what the windows of a served batch see
        dict(name="read8_64", op="read", bs=64, rows_lo=1, rows_hi=8, ctx_lo=1000, ctx_hi=32000, hq=64, hkv=8, d=64,
             page=32, window=4096, sinks=4),
        # one committed token of one chat, five alternatives
        dict(name="logprobs_one", op="logprobs", bs=1, rows_lo=1, rows_hi=1, vocab=151936, dtype="bf16", top=5, mask=False),
        # the benchmark's batch with pruned windows, under a grammar, twenty alternatives
        dict(name="logprobs_verify_256", op="logprobs", bs=256, rows_lo=1, rows_hi=8, vocab=151936, dtype="bf16", top=20,
             mask=True),
        # a few long windows whose logits are kept in 32 bits, no alternatives asked for
        dict(name="logprobs_f32_8", op="logprobs", bs=8, rows_lo=16, rows_hi=16, vocab=129280, dtype="f32", top=0, mask=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "read", "logprobs"])
    bs = _log(rng, 1, 256)
    prompts = rng.random() < 0.25
    if op == "logprobs":
        gamma = rng.randint(1, 15)
        vocab = 8 * _log(rng, 500, 18992)
        bs = max(1, min(bs, 160_000_000 // (vocab * (gamma + 1))))
        return dict(op=op, bs=bs, rows_lo=1, rows_hi=gamma + 1, vocab=vocab, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    top=rng.choice([0, 1, 5, 20, 32]), mask=rng.random() < 0.4)
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 3, 4, 5, 8])
    d = rng.choice([64, 128, 128])
    case = dict(op=op, bs=bs, rows_lo=1, rows_hi=rng.randint(1, 16), ctx_lo=0, ctx_hi=1, hq=hq, hkv=hkv, d=d,
                page=rng.choice([16, 32, 64, 128]))
    if prompts:
        case["bs"] = rng.randint(1, 4)
        case["rows_hi"] = _log(rng, 17, 4000 // case["bs"])
        case["rows_lo"] = 1 + case["rows_hi"] // 2
    if op == "append":
        case["ctx_hi"] = _log(rng, 1, 4000)
        case["rot"] = rng.choice([d, d, d // 2])
        case["interleaved"] = rng.random() < 0.4
        return case
    window = rng.choice([0, _log(rng, 16, 4096), _log(rng, 256, 4096)])
    # the cached tokens of the batch together: at most what the long listed case holds
    case["ctx_hi"] = max(1, min(_log(rng, 30, 100000), 250000 // case["bs"], 6000 if prompts else 100000))
    case["ctx_lo"] = case["ctx_hi"] // 3
    case["window"] = window
    case["sinks"] = rng.choice([0, 1, 4, 19]) if window else 0
    return case


def _lengths(case):
    """(rows of each request, tokens that each has in the cache): fixed by the case."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["bs"])]
    if "ctx_hi" not in case:
        return n, None
    lo, hi = math.log(case["ctx_lo"] + 1), math.log(case["ctx_hi"] + 1)
    return n, [int(round(math.exp(r.uniform(lo, hi)))) - 1 for _ in range(case["bs"])]


def _committed(case, n):
    """Tokens that each request commits: fixed by the case."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + "c")
    return [r.randint(1, x) for x in n]


def _starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return out


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    n, ctx = _lengths(case)
    cu = _starts(n)
    s = dict(case, cu=_i32(cu), rows=cu[-1], max_rows=max(n), max_ctx=max(ctx) if ctx else 0)
    if case["op"] == "logprobs":
        _prepare_logits(s, case, g, n)
    else:
        _prepare_cache(s, case, g, n, ctx)
    if own:
        from speculative_decoding_draft_markov_gb300 import binding as B
        if case["op"] == "attention":
            s["ws"] = B.alloc_attention_workspace(case["hq"], case["hkv"], case["d"])
            # one layer's worth of 16-bit pages, which all layers of a model share
            s["scratch"] = [torch.empty(s["k_cache"].shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        elif case["op"] == "logprobs":
            s["ws"] = B.alloc_logprobs_workspace(case["bs"] * s["max_rows"], case["vocab"], case["top"])
        else:
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)


def _prepare_cache(s, case, g, n, ctx):
    bs, page, hq, hkv, d, rows = case["bs"], case["page"], case["hq"], case["hkv"], case["d"], s["rows"]
    need = [-(-(c + x) // page) for c, x in zip(ctx, n)]
    n_pages = sum(need) + 3
    # pages are handed out as requests come and go: in no order
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor(_starts(need)[:-1], device="cuda")
    col = torch.arange(max(need), device="cuda")
    table = order[(first[:, None] + col).clamp(max=n_pages - 1)]
    s["page_table"] = torch.where(col < torch.tensor(need, device="cuda")[:, None], table, -1).contiguous()
    s["ctx"] = _i32(ctx)
    # what an append leaves: values whose largest lies between 224 and 448 of their slot's power of two
    shape = (n_pages, hkv, page, d)
    s["k_cache"], s["v_cache"] = ((_randn(g, *shape) * 100).clamp_(-448, 448).to(F8) for _ in range(2))
    s["kv_scale"] = torch.randint(117, 121, (n_pages, hkv, page, 2), generator=g, device="cuda", dtype=torch.uint8)
    if case["op"] == "attention":
        s["q"] = _randn(g, rows, hq, d)
        s["scale"] = d ** -0.5
        s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device="cuda")
        return
    if case["op"] == "read":
        # the reader's own pages, of other numbers
        s["out_table"] = torch.where(s["page_table"] >= 0, n_pages - 1 - s["page_table"], -1).contiguous()
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return
    # q, k and v as one projection leaves them: side by side in each row
    qkv = _randn(g, rows, hq + 2 * hkv, d)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(s["max_ctx"] + s["max_rows"], device="cuda", dtype=torch.float64)[:, None] * inv
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    s["q_out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")


def _prepare_logits(s, case, g, n):
    bs, vocab, rows, m = case["bs"], case["vocab"], s["rows"], s["max_rows"]
    x = _randn(g, rows, vocab, dtype=torch.float32) * 3
    if case["mask"]:
        # a grammar allows a few ids in one state and nearly all of them in another
        share = torch.where(torch.rand(rows, 1, generator=g, device="cuda") < 0.5, 0.02, 0.9)
        x.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") > share, float("-inf"))
    s["logits"] = x.to(DTYPES[case["dtype"]])
    # what was committed is likely, if not always the likeliest
    noise = _randn(g, rows, vocab, dtype=torch.float32)
    said = (x + 2 * noise).argmax(1).to(torch.int32)
    at = (s["cu"][:-1, None] + torch.arange(m, device="cuda")).clamp(max=rows - 1)
    kept = torch.arange(m, device="cuda") < _i32(_committed(case, n))[:, None]
    s["tokens"] = torch.where(kept, said[at], -1).contiguous()
    f32 = dict(dtype=torch.float32, device="cuda")
    s["logprob"], s["entropy"] = torch.empty(bs, m, **f32), torch.empty(bs, m, **f32)
    s["rank"] = torch.empty(bs, m, dtype=torch.int32, device="cuda")
    s["top_ids"] = torch.empty(bs, m, case["top"], dtype=torch.int32, device="cuda") if case["top"] else None
    s["top_logprobs"] = torch.empty(bs, m, case["top"], **f32) if case["top"] else None


# ------------------------------------------------------------------------------------- passes

def run(s):
    if own:
        from speculative_decoding_draft_markov_gb300 import binding as B
        if s["op"] == "append":
            B.dspark_append_kv8(s["q"], s["k"], s["v"], s["cu"], s["ctx"], s["cos_sin"], s["page_table"], s["q_out"],
                                s["k_cache"], s["v_cache"], s["kv_scale"], s["ws"], interleaved=s["interleaved"])
            return s["q_out"], s["k_cache"], s["v_cache"], s["kv_scale"]
        if s["op"] == "attention":
            B.dspark_window_attention_kv8(s["q"], s["k_cache"], s["v_cache"], s["kv_scale"], s["page_table"], s["cu"],
                                          s["ctx"], s["max_rows"], s["scale"], s["window"], s["sinks"], s["out"],
                                          s["lse"], *s["scratch"], s["ws"])
            return s["out"], s["lse"]
        if s["op"] == "read":
            B.dspark_read_kv8(s["k_cache"], s["v_cache"], s["kv_scale"], s["page_table"], s["cu"], s["ctx"], s["rows"],
                              s["window"], s["sinks"], s["out_table"], s["k_out"], s["v_out"], s["ws"])
            return s["k_out"], s["v_out"]
        B.dspark_token_logprobs(s["logits"], s["cu"], s["tokens"], 1.0, s["logprob"], s["entropy"], s["rank"],
                                s["top_ids"], s["top_logprobs"], s["ws"])
        return _reported(s)
    return {"append": _plain_append, "attention": _plain_attention, "read": _plain_read,
            "logprobs": _plain_logprobs}[s["op"]](s)


def _reported(s):
    top = (s["top_ids"], s["top_logprobs"]) if s["top"] else ()
    return (s["logprob"], s["entropy"], s["rank"], *top)


def _rows_of(s):
    """(request, place in its window) of each packed row."""
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["cu"], row, right=True) - 1
    return req, row - s["cu"][req]


def _power(e):
    """2^e of whole numbers from -126 to 127, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _value_of(codes, scale):
    """The values of cache slots [.., D] with their exponent bytes [..]."""
    e = scale.to(torch.int32)
    return codes.float() * torch.where(e == 255, float("nan"), _power(e.clamp(1, 254) - 127))[..., None]


def _quantise(x):
    """Codes and exponent bytes of fp32 vectors [.., D]: the smallest power of two under which all fit."""
    top = x.abs().amax(-1)
    part, e = torch.frexp(top)  # top = part 2^e, 1/2 <= part < 1; 448 = 0.875 2^9
    e = torch.where(part > 0.875, e - 8, e - 9)
    e = torch.where(top == 0, -126, e).clamp(min=-126)
    good = torch.isfinite(top)
    codes = torch.where(good[..., None], x * _power(torch.where(good, -e, 0))[..., None], 0.0).to(F8)
    return codes.view(torch.uint8), torch.where(good, e + 127, 255).to(torch.uint8)


def _rotate(x, cos, sin, rot, interleaved):
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_append(s):
    req, i = _rows_of(s)
    pos = (s["ctx"][req] + i).long()
    rot, page = s["rot"], s["page"]
    cos, sin = (t[:, None] for t in s["cos_sin"][pos].chunk(2, 1))
    at, slot = s["page_table"][req, pos // page].long(), pos % page
    k, ke = _quantise(_rotate(s["k"], cos, sin, rot, s["interleaved"]))
    v, ve = _quantise(s["v"].float())
    s["k_cache"].view(torch.uint8)[at, :, slot] = k
    s["v_cache"].view(torch.uint8)[at, :, slot] = v
    s["kv_scale"][at, :, slot] = torch.stack([ke, ve], -1)
    q = _rotate(s["q"], cos, sin, rot, s["interleaved"]).to(s["q"].dtype)
    return q, s["k_cache"], s["v_cache"], s["kv_scale"]


def _seen(s):
    """The places that any row of a request may see, its first tokens, then its window: positions [bs, places], whether
    each counts once, and the pages that hold them."""
    window, sinks, m, page = s["window"], s["sinks"], s["max_rows"], s["page"]
    ctx = s["ctx"].long()
    lo = (ctx - window + 1).clamp(min=0) if window else torch.zeros_like(ctx)
    span = min(window + m - 1, s["max_ctx"] + m) if window else s["max_ctx"] + m
    j = torch.arange(sinks + span, device="cuda")
    pos = torch.where(j < sinks, j, lo[:, None] + j - sinks)
    fresh = (j < sinks) | (pos >= sinks)
    return pos, fresh, (pos // page).clamp(max=s["page_table"].shape[1] - 1)


def _plain_attention(s):
    bs, page, hq, hkv, d = s["bs"], s["page"], s["hq"], s["hkv"], s["d"]
    window, sinks, m = s["window"], s["sinks"], s["max_rows"]
    ctx = s["ctx"].long()
    pos, fresh, col = _seen(s)
    at = s["page_table"].gather(1, col).clamp(min=0).long()
    scale = s["kv_scale"][at, :, pos % page]
    k = _value_of(s["k_cache"].view(torch.uint8)[at, :, pos % page].view(F8), scale[..., 0]).transpose(1, 2)
    v = _value_of(s["v_cache"].view(torch.uint8)[at, :, pos % page].view(F8), scale[..., 1]).transpose(1, 2)
    # the rows, padded to the longest window
    i = torch.arange(m, device="cuda")
    q = s["q"][(s["cu"][:-1, None] + i).clamp(max=s["rows"] - 1)].float()
    q = q.view(bs, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(bs, hkv, -1, d)
    p = (ctx[:, None] + i)[:, :, None]
    seen = fresh[:, None] & (pos[:, None] <= p)
    if window:
        seen = seen & ((pos[:, None] > p - window) | (pos[:, None] < sinks))
    x = (q @ k.transpose(2, 3)).view(bs, hkv, hq // hkv, m, -1) * s["scale"]
    x = x.masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(bs, hkv, -1, x.shape[-1]) @ v).view(bs, hkv, hq // hkv, m, d) / total
    req, row = _rows_of(s)
    o = o.permute(0, 3, 1, 2, 4)[req, row].reshape(s["rows"], hq, d)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2)[req, row].reshape(s["rows"], hq)
    return o.to(torch.bfloat16), lse


def _plain_read(s):
    page = s["page"]
    pos, fresh, col = _seen(s)
    last = s["ctx"] + s["cu"][1:] - s["cu"][:-1] - 1
    r, j = (fresh & (pos <= last[:, None])).nonzero(as_tuple=True)
    pos, col = pos[r, j], col[r, j]
    at, to, slot = s["page_table"][r, col].long(), s["out_table"][r, col].long(), pos % page
    scale = s["kv_scale"][at, :, slot]
    for k, (codes, out) in enumerate(((s["k_cache"], s["k_out"]), (s["v_cache"], s["v_out"]))):
        out[to, :, slot] = _value_of(codes.view(torch.uint8)[at, :, slot].view(F8), scale[..., k]).to(out.dtype)
    return s["k_out"], s["v_out"]


def _plain_logprobs(s):
    bs, m, vocab, top = s["bs"], s["max_rows"], s["vocab"], s["top"]
    token = s["tokens"].reshape(-1)
    row = (s["cu"][:-1, None] + torch.arange(m, device="cuda")).reshape(-1)
    item = (token >= 0).nonzero()[:, 0]  # the others report nothing
    x = s["logits"][row[item].long()].float()
    t = token[item].long()[:, None]
    high = x.amax(1, keepdim=True)
    w = (x - high).exp()
    total = w.sum(1, keepdim=True)
    lse = high + total.log()
    mean = torch.where(w > 0, w * (x - high), 0.0).sum(1, keepdim=True) / total
    chosen = x.gather(1, t)
    ids = torch.arange(vocab, device="cuda")
    ahead = (x > chosen) | ((x == chosen) & (ids < t))
    s["logprob"].zero_().view(-1)[item] = ((chosen - high) - total.log())[:, 0]
    s["entropy"].zero_().view(-1)[item] = (total.log() - mean)[:, 0]
    s["rank"].zero_().view(-1)[item] = 1 + ahead.sum(1, dtype=torch.int32)
    if top:
        # by value, then by the lower id: a whole number for each that orders them so
        bits = (x + 0.0).view(torch.int32).long()  # one zero
        key = torch.where(bits < 0, (bits ^ 0x7FFFFFFF), bits) * 2 ** 24 - ids
        at = key.topk(top, 1).indices
        value = x.gather(1, at)
        s["top_ids"].fill_(-1).view(-1, top)[item] = torch.where(value > float("-inf"), at, -1).to(torch.int32)
        s["top_logprobs"].fill_(float("-inf")).view(-1, top)[item] = value - lse
    return _reported(s)


# --------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    return {"append": _exact_append, "attention": _exact_attention, "read": _exact_read,
            "logprobs": _exact_logprobs}[case["op"]](prepare(case, seed), case)


def _exact_values(s, which, at, slot):
    """[places, hkv, d] in 64 bits: a number times a power of two."""
    codes = (s["k_cache"], s["v_cache"])[which].view(torch.uint8)[at, :, slot].view(F8).double()
    return codes * torch.pow(2.0, s["kv_scale"][at, :, slot, which].double() - 127)[..., None]


def _exact_codes(x):
    """The e4m3 values and exponent bytes of [n, d] vectors: 3 bits behind the first, steps of 2^-9 at the least."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448)).clamp(min=-126)
    e = torch.where(top <= 448 * torch.pow(2.0, e - 1), e - 1, e)  # where the logarithm was rounded up
    y = x * torch.pow(2.0, -e)
    step = torch.pow(2.0, torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round() * step, e[..., 0] + 127


def _exact_append(s, case):
    n, ctx = _lengths(case)
    rot, page = case["rot"], case["page"]
    half = rot // 2
    # complex numbers: a pair turned by its angle is a product
    turn = torch.complex(s["cos_sin"][:, :half].double(), s["cos_sin"][:, half:].double())

    def turned(x, pos):
        x = x.double()
        part = x[..., :rot]
        pair = part.reshape(*part.shape[:-1], half, 2) if case["interleaved"] else \
            part.reshape(*part.shape[:-1], 2, half).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[pos][:, None])
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.reshape(part.shape), x[..., rot:]], -1)

    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    sc = s["kv_scale"].double()
    first = 0
    for r in range(case["bs"]):
        rows = slice(first, first + n[r])
        first += n[r]
        pos = torch.arange(ctx[r], ctx[r] + n[r], device="cuda")
        pages, slot = s["page_table"][r].long()[pos // page], pos % page
        q[rows] = turned(s["q"][rows], pos)
        kc[pages, :, slot], sc[pages, :, slot, 0] = _exact_codes(turned(s["k"][rows], pos))
        vc[pages, :, slot], sc[pages, :, slot, 1] = _exact_codes(s["v"][rows].double())
    return q, kc, vc, sc.to(torch.uint8)


def _exact_attention(s, case):
    n, ctx = _lengths(case)
    page, hq, hkv, d, window, sinks = (case[k] for k in ("page", "hq", "hkv", "d", "window", "sinks"))
    g = hq // hkv
    out = torch.empty(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["rows"], hq, dtype=torch.float64, device="cuda")
    first = 0
    for r in range(case["bs"]):
        length = ctx[r] + n[r]
        pages = s["page_table"][r].long()[:-(-length // page)]
        at = torch.arange(length, device="cuda")
        if window:  # what no row of the request sees is left out
            at = at[(at < sinks) | (at > ctx[r] - window)]
        keys, vals = (_exact_values(s, k, pages[at // page], at % page) for k in range(2))
        for a in range(0, n[r], 512):
            b = min(n[r], a + 512)
            p = torch.arange(ctx[r] + a, ctx[r] + b, device="cuda")[:, None, None]
            hidden = at > p
            if window:
                hidden |= (at <= p - window) & (at >= sinks)
            for h in range(hkv):
                x = s["q"][first + a:first + b, h * g:h * g + g].double() @ keys[:, h].T / math.sqrt(d)
                x.masked_fill_(hidden, -math.inf)
                lse[first + a:first + b, h * g:h * g + g] = torch.logsumexp(x, 2)
                out[first + a:first + b, h * g:h * g + g] = torch.softmax(x, 2) @ vals[:, h]
        first += n[r]
    return out, lse


def _exact_read(s, case):
    n, ctx = _lengths(case)
    page, window, sinks = case["page"], case["window"], case["sinks"]
    outs = [s["k_out"].double(), s["v_out"].double()]
    for r in range(case["bs"]):
        at = torch.arange(ctx[r] + n[r], device="cuda")
        if window:
            at = at[(at < sinks) | (at > ctx[r] - window)]
        src, dst = (s[k][r].long()[at // page] for k in ("page_table", "out_table"))
        for k in range(2):
            outs[k][dst, :, at % page] = _exact_values(s, k, src, at % page)
    return outs


def _exact_logprobs(s, case):
    n, _ = _lengths(case)
    m, top = s["max_rows"], case["top"]
    logprob, entropy = (torch.zeros(case["bs"], m, dtype=torch.float64, device="cuda") for _ in range(2))
    best = torch.full((case["bs"], m, top), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for r, kept in enumerate(_committed(case, n)):
        x = torch.log_softmax(s["logits"][first:first + kept].double(), 1)
        logprob[r, :kept] = x.gather(1, s["tokens"][r, :kept, None].long())[:, 0]
        entropy[r, :kept] = torch.special.entr(x.exp()).sum(1)
        if top:
            best[r, :kept] = x.sort(1, descending=True).values[:, :top]
        first += n[r]
    return (logprob, entropy, None, None, best) if top else (logprob, entropy, None)


# -------------------------------------------------------------------------------------- work

def work(case):
    n, ctx = _lengths(case)
    rows, bs = sum(n), case["bs"]
    if case["op"] == "append":
        q, kv = case["hq"] * case["d"], 2 * case["hkv"] * case["d"]
        return {"bytes": rows * (4 * q + 3 * kv + 2 * case["hkv"] + 4 * case["rot"]) + 8 * bs,
                "flops": 3 * rows * (case["hq"] + case["hkv"]) * case["rot"] + 3 * rows * kv}
    if case["op"] == "logprobs":
        size, items = (2 if case["dtype"] == "bf16" else 4), sum(_committed(case, n))
        return {"bytes": items * case["vocab"] * size + bs * max(n) * (16 + 8 * case["top"]), "flops": 6 * items * case["vocab"]}
    pairs = places = 0
    for x, c in zip(n, ctx):
        w, k = case["window"] or c + x, case["sinks"]
        lo = max(0, c - w + 1)
        places += c + x - lo + min(lo, k)
        for p in range(c, c + x):
            at = max(0, p - w + 1)
            pairs += p + 1 - at + min(at, k)
    cache = places * case["hkv"] * (2 * case["d"] + 2) + 4 * sum(-(-(c + x) // case["page"]) for x, c in zip(n, ctx))
    if case["op"] == "read":
        return {"bytes": cache + places * case["hkv"] * 4 * case["d"], "flops": 2 * places * case["hkv"] * case["d"]}
    return {"bytes": cache + rows * case["hq"] * (4 * case["d"] + 4), "flops": 4 * pairs * case["hq"] * case["d"]}
