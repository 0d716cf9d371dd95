"""Cases of the serving-side operators around the speculative step: the paged cache append with
rotation, the windows' attention over that cache, the logit rules before the verification, and
the token history that those rules read.

Every case gives sizes only.  Lengths are drawn from the case itself (so that its work is fixed),
values from the seed.  Rows are packed as the step packs them: request r owns rows
cu[r] .. cu[r+1]-1, its row i sits at position ctx[r] + i of its sequence."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one chat: the smallest call of a decoding loop, all latency
        dict(name="append_one_token", op="append", bs=1, rows_lo=1, rows_hi=1, ctx_lo=777, ctx_hi=777, hq=32, hkv=8,
             d=128, page=16, rot=128, interleaved=False),
        # three prompts taken in at once, 8191 tokens together, half of each head rotated
        dict(name="append_prompts", op="append", bs=3, rows_lo=2400, rows_hi=3000, ctx_lo=1, ctx_hi=999, hq=32, hkv=8,
             d=128, page=64, rot=64, interleaved=True),
        # one token of one chat over its whole short context
        dict(name="attn_one_token", op="attention", bs=1, rows_lo=1, rows_hi=1, ctx_lo=1500, ctx_hi=1500, hq=32,
             hkv=8, d=128, page=16, window=0, sinks=0),
        # a served batch with contexts from short to long; pruned windows of 1 to 8 rows
        dict(name="attn_verify_64", op="attention", bs=64, rows_lo=1, rows_hi=8, ctx_lo=1000, ctx_hi=32000, hq=64,
             hkv=8, d=64, page=32, window=4096, sinks=4),
        # the benchmark's batch: 256 requests, the whole block of gamma = 7 verified
        dict(name="attn_verify_256", op="attention", bs=256, rows_lo=8, rows_hi=8, ctx_lo=500, ctx_hi=6000, hq=32,
             hkv=8, d=128, page=64, window=1024, sinks=4),
        # two long documents, a block of gamma = 15, every position visible
        dict(name="attn_long_2", op="attention", bs=2, rows_lo=16, rows_hi=16, ctx_lo=120001, ctx_hi=131000, hq=32,
             hkv=8, d=128, page=128, window=0, sinks=0),
        # two chunks of prompts, about 8000 tokens, over what is cached already
        dict(name="attn_prompts", op="attention", bs=2, rows_lo=3700, rows_hi=4300, ctx_lo=1000, ctx_hi=5000, hq=32,
             hkv=8, d=128, page=64, window=4096, sinks=4),
        # one row of one chat
        dict(name="logits_one_row", op="logits", bs=1, rows_lo=1, rows_hi=1, vocab=151936, dtype="bf16", hist=3000,
             biases=40, mask=True),
        # the benchmark's batch with pruned windows, under a grammar
        dict(name="logits_verify_256", op="logits", bs=256, rows_lo=1, rows_hi=8, vocab=151936, dtype="bf16",
             hist=4000, biases=100, mask=True),
        # a few long windows whose logits are kept in 32 bits, no grammar
        dict(name="logits_f32_8", op="logits", bs=8, rows_lo=16, rows_hi=16, vocab=129280, dtype="f32", hist=500,
             biases=300, mask=False),
        # one request admitted with a prompt of some pages
        dict(name="history_one", op="history", bs=1, rows_lo=2500, rows_hi=2500, vocab=151936, gamma=7),
        # a batch admitted again after a restart: prompts and what was answered so far
        dict(name="history_64", op="history", bs=64, rows_lo=100, rows_hi=8000, vocab=129280, gamma=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "logits", "history"])
    bs = _log(rng, 1, 256)
    prompts = rng.random() < 0.25
    if op == "history":
        bs = min(bs, 64)
        return dict(op=op, bs=bs, rows_lo=1 + rng.randrange(60), rows_hi=_log(rng, 61, 8000),
                    vocab=8 * _log(rng, 2000, 16160), gamma=rng.randint(1, 16))
    if op == "logits":
        gamma = rng.randint(1, 15)
        vocab = 8 * _log(rng, 500, 18992)
        bs = max(1, min(bs, 160_000_000 // (vocab * (gamma + 1))))
        return dict(op=op, bs=bs, rows_lo=1, rows_hi=gamma + 1, vocab=vocab, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    hist=_log(rng, 10, 6000), biases=rng.choice([0, 7, 100, 300]), mask=rng.random() < 0.6)
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
    {"append": _prepare_cache, "attention": _prepare_cache, "logits": _prepare_logits,
     "history": _prepare_history}[case["op"]](s, case, g, n, ctx)
    if own:
        from speculative_decoding_draft_markov_gb300 import binding as B
        if case["op"] == "attention":
            s["ws"] = B.alloc_attention_workspace(case["hq"], case["hkv"], case["d"])
        else:
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)


def _randint(g, lo, hi, shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


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
    shape = (n_pages, hkv, page, d)
    s["k_cache"], s["v_cache"] = _randn(g, *shape), _randn(g, *shape)
    if case["op"] == "attention":
        s["q"] = _randn(g, rows, hq, d)
        s["scale"] = d ** -0.5
        s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device="cuda")
        return
    # q, k and v as one projection leaves them: side by side in each row
    qkv = _randn(g, rows, hq + 2 * hkv, d)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(s["max_ctx"] + s["max_rows"], device="cuda", dtype=torch.float64)[:, None] * inv
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    s["q_out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")


def _zipf(g, shape, vocab):
    """Token ids as text has them: few of them often."""
    u = torch.rand(shape, generator=g, device="cuda")
    return ((vocab ** u - 1) * (vocab / (vocab - 1))).long().clamp(max=vocab - 1) * 7919 % vocab


def _prepare_logits(s, case, g, n, ctx):
    bs, vocab, rows = case["bs"], case["vocab"], s["rows"]
    s["logits"] = (_randn(g, rows, vocab, dtype=torch.float32) * 3).to(DTYPES[case["dtype"]])
    s["out"] = torch.empty_like(s["logits"])
    s["ids"] = _zipf(g, (rows,), vocab).to(torch.int32)
    prompt = _zipf(g, (bs, case["hist"]), vocab)
    said = _zipf(g, (bs, case["hist"] // 2 + 1), vocab)
    count = torch.zeros(bs, vocab, dtype=torch.int32, device="cuda")
    count.scatter_add_(1, said, torch.ones_like(said, dtype=torch.int32))
    flag = torch.zeros(bs, vocab, dtype=torch.int32, device="cuda").scatter_(1, prompt, 32768)
    s["hist"] = (count - flag).to(torch.int16)  # the flag is the sign bit
    plain = torch.rand(bs, generator=g, device="cuda") < 0.3  # requests that ask for no penalty
    s["repetition"] = torch.where(plain, 1.0, 1.0 + torch.rand(bs, generator=g, device="cuda"))
    s["frequency"] = torch.where(plain, 0.0, torch.rand(bs, generator=g, device="cuda"))
    s["presence"] = torch.where(plain, 0.0, torch.rand(bs, generator=g, device="cuda"))
    s["bias_start"] = s["bias_ids"] = s["bias_vals"] = s["mask"] = None
    if case["biases"]:
        m = min(case["biases"], vocab)
        order = torch.rand(bs, vocab, generator=g, device="cuda").topk(m, 1).indices
        s["bias_ids"] = order.sort(1).values.to(torch.int32).reshape(-1).contiguous()
        s["bias_vals"] = _randn(g, bs * m, dtype=torch.float32) * 5
        s["bias_start"] = _i32([m * r for r in range(bs + 1)])
    if case["mask"]:
        # a grammar allows a few ids in one state and nearly all of them in another
        words = (vocab + 31) // 32
        x, y = (_randint(g, -2**31, 2**31 - 1, (rows, words), torch.int64) for _ in range(2))
        wide = torch.rand(rows, 1, generator=g, device="cuda") < 0.5
        s["mask"] = torch.where(wide, x | y, x & y).to(torch.int32)


def _prepare_history(s, case, g, n, ctx):
    bs, vocab = case["bs"], case["vocab"]
    s["tokens"] = _zipf(g, (s["rows"],), vocab).to(torch.int32)
    # two thirds of a list are its prompt
    s["n_prompt"] = _i32([2 * x // 3 for x in n])
    s["hist"] = torch.empty(bs, vocab, dtype=torch.int16, device="cuda")
    # the step after: accepted tokens, then -1
    acc = _randint(g, 1, case["gamma"] + 2, (bs, 1))
    out = _zipf(g, (bs, case["gamma"] + 1), vocab).to(torch.int32)
    s["out_tokens"] = torch.where(torch.arange(case["gamma"] + 1, device="cuda") < acc, out, -1).contiguous()


# ------------------------------------------------------------------------------------- passes

def run(s):
    if own:
        from speculative_decoding_draft_markov_gb300 import binding as B
        if s["op"] == "append":
            B.dspark_append_kv(s["q"], s["k"], s["v"], s["cu"], s["ctx"], s["cos_sin"], s["page_table"], s["q_out"],
                               s["k_cache"], s["v_cache"], s["ws"], interleaved=s["interleaved"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if s["op"] == "attention":
            B.dspark_window_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu"], s["ctx"],
                                      s["max_rows"], s["scale"], s["window"], s["sinks"], s["out"], s["lse"], s["ws"])
            return s["out"], s["lse"]
        if s["op"] == "logits":
            B.dspark_process_logits(s["logits"], s["cu"], s["ids"], s["hist"], s["repetition"], s["frequency"],
                                    s["presence"], s["bias_start"], s["bias_ids"], s["bias_vals"], s["mask"], s["out"],
                                    s["ws"])
            return s["out"]
        B.dspark_history_build(s["tokens"], s["cu"], s["n_prompt"], s["hist"], s["ws"])
        B.dspark_history_commit(s["out_tokens"], s["hist"], s["ws"])
        return s["hist"]
    return {"append": _plain_append, "attention": _plain_attention, "logits": _plain_logits,
            "history": _plain_history}[s["op"]](s)


def _rows_of(s):
    """(request, place in its window) of each packed row."""
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["cu"], row, right=True) - 1
    return req, row - s["cu"][req]


def _rotate(x, cos, sin, rot, interleaved):
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_append(s):
    req, i = _rows_of(s)
    pos = (s["ctx"][req] + i).long()
    rot, page = s["rot"], s["page"]
    cos, sin = (t[:, None] for t in s["cos_sin"][pos].chunk(2, 1))
    at = s["page_table"][req, pos // page].long()
    s["k_cache"][at, :, pos % page] = _rotate(s["k"], cos, sin, rot, s["interleaved"])
    s["v_cache"][at, :, pos % page] = s["v"]
    return _rotate(s["q"], cos, sin, rot, s["interleaved"]), s["k_cache"], s["v_cache"]


def _plain_attention(s):
    bs, page, hq, hkv, d = s["bs"], s["page"], s["hq"], s["hkv"], s["d"]
    window, sinks, m = s["window"], s["sinks"], s["max_rows"]
    ctx = s["ctx"].long()
    # the places that any row of a request may see: its first tokens, then its window
    lo = (ctx - window + 1).clamp(min=0) if window else torch.zeros_like(ctx)
    span = min(window + m - 1, s["max_ctx"] + m) if window else s["max_ctx"] + m
    j = torch.arange(sinks + span, device="cuda")
    pos = torch.where(j < sinks, j, lo[:, None] + j - sinks)
    fresh = (j < sinks) | (pos >= sinks)
    at = s["page_table"].gather(1, (pos // page).clamp(max=s["page_table"].shape[1] - 1)).clamp(min=0).long()
    k = s["k_cache"][at, :, pos % page].float().transpose(1, 2)  # [bs, hkv, places, d]
    v = s["v_cache"][at, :, pos % page].float().transpose(1, 2)
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


def _plain_logits(s):
    bs, vocab, rows = s["bs"], s["vocab"], s["rows"]
    req, i = _rows_of(s)
    hist = s["hist"].int()[req]
    count, prompt = hist & 32767, hist < 0
    # the window's own drafted tokens up to the row count as said
    k = torch.arange(1, s["max_rows"] + 1, device="cuda")
    drafted = s["ids"][(s["cu"][req][:, None] + k).clamp(max=rows - 1)].long()
    count.scatter_add_(1, drafted, (k <= i[:, None]).int())
    x = s["logits"].float()
    rho = s["repetition"][req][:, None]
    x = torch.where(prompt | (count > 0), torch.where(x > 0, x / rho, x * rho), x)
    x = x - s["frequency"][req][:, None] * count - s["presence"][req][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        entry = torch.arange(s["bias_ids"].numel(), device="cuda", dtype=torch.int32)
        of = torch.searchsorted(s["bias_start"], entry, right=True) - 1
        dense = torch.zeros(bs, vocab, device="cuda")
        dense[of, s["bias_ids"].long()] = s["bias_vals"]
        x = x + dense[req]
    if s["mask"] is not None:
        v = torch.arange(vocab, device="cuda", dtype=torch.int32)
        x = x.masked_fill(((s["mask"][:, v >> 5] >> (v & 31)) & 1) == 0, float("-inf"))
    return x.to(s["logits"].dtype)


def _plain_history(s):
    bs, vocab = s["bs"], s["vocab"]
    req, i = _rows_of(s)
    asked = i < s["n_prompt"][req]
    tokens = s["tokens"].long()
    flag = torch.zeros(bs * vocab, dtype=torch.int32, device="cuda")
    flag.scatter_reduce_(0, req * vocab + tokens, asked.int(), "amax")
    count = torch.zeros(bs * vocab, dtype=torch.int32, device="cuda")
    count.scatter_add_(0, req * vocab + tokens, (~asked).int())
    out = s["out_tokens"].long()
    at = torch.arange(bs, device="cuda")[:, None] * vocab + out.clamp(min=0)
    count.scatter_add_(0, at.reshape(-1), (out >= 0).int().reshape(-1))
    return (count.clamp(max=32767) - 32768 * flag).to(torch.int16).view(bs, vocab)


# --------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    return {"append": _exact_append, "attention": _exact_attention, "logits": _exact_logits,
            "history": _exact_history}[case["op"]](prepare(case, seed), case)


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
    first = 0
    for r in range(case["bs"]):
        rows = slice(first, first + n[r])
        first += n[r]
        pos = torch.arange(ctx[r], ctx[r] + n[r], device="cuda")
        pages = s["page_table"][r].long()[pos // page]
        q[rows] = turned(s["q"][rows], pos)
        kc[pages, :, pos % page] = turned(s["k"][rows], pos)
        vc[pages, :, pos % page] = s["v"][rows].double()
    return q, kc, vc


def _exact_attention(s, case):
    n, ctx = _lengths(case)
    page, hq, hkv, d, window, sinks = (case[k] for k in ("page", "hq", "hkv", "d", "window", "sinks"))
    out = torch.empty(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["rows"], hq, dtype=torch.float64, device="cuda")
    first = 0
    for r in range(case["bs"]):
        length = ctx[r] + n[r]
        pages = s["page_table"][r].long()[:-(-length // page)]
        at = torch.arange(length, device="cuda")
        if window:  # what no row of the request sees is left out
            at = at[(at < sinks) | (at > ctx[r] - window)]
        keys = s["k_cache"][pages[at // page], :, at % page].double()
        vals = s["v_cache"][pages[at // page], :, at % page].double()
        for a in range(0, n[r], 512):
            b = min(n[r], a + 512)
            p = torch.arange(ctx[r] + a, ctx[r] + b, device="cuda")[:, None]
            hidden = at > p
            if window:
                hidden |= (at <= p - window) & (at >= sinks)
            for h in range(hq):
                x = s["q"][first + a:first + b, h].double() @ keys[:, h // (hq // hkv)].T * case_scale(d)
                x.masked_fill_(hidden, -math.inf)
                lse[first + a:first + b, h] = torch.logsumexp(x, 1)
                out[first + a:first + b, h] = torch.softmax(x, 1) @ vals[:, h // (hq // hkv)]
        first += n[r]
    return out, lse


def case_scale(d):
    return 1.0 / math.sqrt(d)


def _exact_logits(s, case):
    n, _ = _lengths(case)
    vocab = case["vocab"]
    out = torch.empty(s["rows"], vocab, dtype=torch.float64, device="cuda")
    shift = torch.arange(32, device="cuda")
    first = 0
    for r in range(case["bs"]):
        word = s["hist"][r].long() & 0xFFFF
        count, prompt = (word & 0x7FFF).double(), word >= 0x8000
        rho, freq, pres = (s[k][r].double() for k in ("repetition", "frequency", "presence"))
        bias = torch.zeros(vocab, dtype=torch.float64, device="cuda")
        if case["biases"]:
            m = s["bias_ids"].numel() // case["bs"]
            bias[s["bias_ids"][r * m:(r + 1) * m].long()] = s["bias_vals"][r * m:(r + 1) * m].double()
        for i in range(n[r]):
            if i:
                count[s["ids"][first + i].long()] += 1
            said = count > 0
            x = s["logits"][first + i].double()
            factor = torch.where(x > 0, 1 / rho, rho)
            x = x * torch.where(said | prompt, factor, 1.0) - count * freq - said * pres + bias
            if case["mask"]:
                bits = (s["mask"][first + i].long()[:, None] >> shift & 1).flatten()[:vocab]
                x = torch.where(bits == 1, x, -math.inf)
            out[first + i] = x
        first += n[r]
    return out


def _exact_history(s, case):
    return None  # whole numbers: they are equal or they are not


# -------------------------------------------------------------------------------------- work

def work(case):
    n, ctx = _lengths(case)
    rows, bs = sum(n), case["bs"]
    if case["op"] == "append":
        row = (case["hq"] + 2 * case["hkv"]) * case["d"] * 2
        return {"bytes": rows * (2 * row + 4 * case["rot"]) + 8 * bs,
                "flops": 3 * rows * (case["hq"] + case["hkv"]) * case["rot"]}
    if case["op"] == "attention":
        pairs = places = 0
        for x, c in zip(n, ctx):
            w, k = case["window"] or c + x, case["sinks"]
            lo = max(0, c - w + 1)
            places += c + x - lo + min(lo, k)
            for p in range(c, c + x):
                at = max(0, p - w + 1)
                pairs += p + 1 - at + min(at, k)
        io = rows * case["hq"] * (4 * case["d"] + 4)
        return {"bytes": places * case["hkv"] * case["d"] * 4 + io + 4 * sum(-(-(c + x) // case["page"])
                                                                          for x, c in zip(n, ctx)),
                "flops": 4 * pairs * case["hq"] * case["d"]}
    if case["op"] == "logits":
        size = 2 if case["dtype"] == "bf16" else 4
        words = (case["vocab"] + 31) // 32
        return {"bytes": rows * case["vocab"] * 2 * size + bs * case["vocab"] * 2 + 8 * bs * case["biases"]
                + (4 * rows * words if case["mask"] else 0), "flops": 3 * rows * case["vocab"]}
    return {"bytes": bs * case["vocab"] * 2 + 4 * rows + 4 * bs * (case["gamma"] + 1), "flops": rows}
