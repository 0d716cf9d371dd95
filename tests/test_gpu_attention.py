"""The paged cache on the GPU: appending with rotation and the windows' attention, against plain
64-bit forms, at the sizes, masks and page layouts where they can go wrong."""
import numpy as np
import pytest

from tests import serving_reference as R

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _status_ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


class Cache:
    """A paged cache with pages in random order; what no request owns is NaN."""

    def __init__(self, ns, ctxs, hkv, d, page, seed, fill=float("nan"), extra_pages=2, evict=None):
        rng = np.random.default_rng(seed)
        self.ns, self.ctxs, self.page = ns, ctxs, page
        need = [-(-(c + n) // page) for c, n in zip(ctxs, ns)]
        self.n_pages = sum(need) + extra_pages
        order = rng.permutation(self.n_pages)
        table = np.full((len(ns), max(max(need), 1) + 1), -1, np.int32)
        at = 0
        for r, m in enumerate(need):
            table[r, :m] = order[at:at + m]
            at += m
        g = torch.Generator().manual_seed(seed)
        self.k = torch.full((self.n_pages, hkv, page, d), fill, dtype=torch.bfloat16)
        self.v = torch.full((self.n_pages, hkv, page, d), fill, dtype=torch.bfloat16)
        self.keys, self.vals = [], []
        for r, (n, c) in enumerate(zip(ns, ctxs)):
            kk = torch.randn(c + n, hkv, d, generator=g).to(torch.bfloat16)
            vv = torch.randn(c + n, hkv, d, generator=g).to(torch.bfloat16)
            for p0 in range(0, c + n, page):
                m = min(page, c + n - p0)
                pg = table[r, p0 // page]
                self.k[pg, :, :m] = kk[p0:p0 + m].transpose(0, 1)
                self.v[pg, :, :m] = vv[p0:p0 + m].transpose(0, 1)
            self.keys.append(_f64(kk))
            self.vals.append(_f64(vv))
        if evict:  # (window, sinks): what no row sees any more is NaN; its whole pages leave the table
            window, sinks = evict
            for r, c in enumerate(ctxs):
                for p in range(sinks, c - window + 1):
                    self.k[table[r, p // page], :, p % page] = float("nan")
                    self.v[table[r, p // page], :, p % page] = float("nan")
                first, last = -(-sinks // page), (max(0, c - window + 1)) // page
                table[r, first:max(first, last)] = -1
        self.table = torch.from_numpy(table).cuda()
        self.k, self.v = self.k.cuda(), self.v.cuda()
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device="cuda")
        self.ctx = torch.tensor(ctxs, dtype=torch.int32, device="cuda")


def _check_attention(c, hq, window, sinks, seed, max_rows=None, q_scale=1.0, pad=3, strided=False, scale=None):
    hkv, d = c.k.shape[1], c.k.shape[3]
    rows = sum(c.ns) + pad
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(rows, hq, d, generator=g) * q_scale).to(torch.bfloat16)
    if strided:
        wide = torch.full((rows, hq + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :hq] = q.cuda()
        qd = wide[:, :hq]
    else:
        qd = q.cuda()
    scale = d ** -0.5 if scale is None else scale
    out = torch.full((rows, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, hq), 7.0, dtype=torch.float32, device="cuda")
    ws = B.alloc_attention_workspace(hq, hkv, d)
    max_rows = max(max(c.ns), 1) if max_rows is None else max_rows
    for _ in range(2):  # the second call runs on a workspace that has been used
        B.dspark_window_attention(qd, c.k, c.v, c.table, c.cu, c.ctx, max_rows, scale, window, sinks, out, lse, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    got, got_lse, qn = _f64(out), _f64(lse), _f64(q)
    first = 0
    for r, n in enumerate(c.ns):
        ref, rl, mag = R.attention(qn[first:first + n], c.keys[r], c.vals[r], c.ctxs[r], scale, window, sinks)
        off = np.abs(got[first:first + n] - ref) - R.attention_bound(mag)
        assert not np.isnan(got[first:first + n]).any(), (r, n)
        assert off.max(initial=-1.0) <= 0, (r, n, off.max())
        size = 1.0 + np.abs(rl).max(initial=0.0)
        assert np.abs(got_lse[first:first + n] - rl).max(initial=0.0) <= 1e-4 * size
        first += n
    assert (got[first:] == 7.0).all() and (got_lse[first:] == 7.0).all()  # pad rows are left alone
    return out, lse


CASES = {
    # name: (rows of each request, tokens cached before, hq, hkv, d, page, window, sinks)
    "one_token_first": ([1], [0], 4, 1, 128, 16, 0, 0),
    "one_token": ([1], [200], 8, 2, 128, 16, 0, 0),
    "one_token_mha": ([1, 1], [127, 128], 3, 3, 64, 32, 0, 0),
    "window_rows": ([8, 1, 3, 0, 5], [300, 17, 0, 90, 128], 8, 2, 128, 16, 0, 0),
    "group_5": ([4, 2], [130, 255], 10, 2, 128, 64, 0, 0),
    "group_3_d64": ([9, 2, 1], [64, 63, 65], 3, 1, 64, 16, 0, 0),
    "group_16": ([16, 3], [500, 1], 16, 1, 64, 128, 0, 0),
    "group_48": ([3, 2], [100, 31], 48, 1, 128, 8, 0, 0),
    "page_8": ([2, 4], [77, 200], 4, 2, 64, 8, 0, 0),
    "page_256": ([2, 4], [300, 700], 4, 2, 128, 256, 0, 0),
    "page_4096": ([2, 4], [4095, 5000], 2, 1, 64, 4096, 600, 3),
    "sinks_only": ([3, 1], [400, 50], 4, 1, 128, 16, 1, 4),
    "window_1": ([6], [333], 4, 1, 64, 32, 1, 0),
    "window_sinks": ([8, 8, 2], [900, 40, 129], 8, 2, 128, 32, 100, 4),
    "window_meets_sinks": ([8, 4], [140, 135], 4, 1, 128, 16, 128, 9),
    "many_sinks": ([8, 1], [700, 20], 4, 1, 64, 64, 50, 200),
    "wide_window": ([5, 2], [900, 10], 4, 2, 128, 64, 100000, 4),
    "long_split": ([2, 1], [6000, 9], 4, 1, 128, 64, 0, 0),
    "long_split_window": ([4, 4], [7000, 3000], 2, 1, 64, 16, 2500, 4),
    "prompt_first": ([300], [0], 4, 1, 128, 64, 0, 0),
    "prompts": ([257, 1, 130], [5, 600, 40], 4, 2, 128, 32, 0, 0),
    "prompt_window": ([400, 190], [100, 0], 6, 2, 64, 16, 90, 5),
    "prompt_group_5": ([150, 77], [300, 12], 5, 1, 128, 128, 64, 4),
    "rows_16": ([4, 1, 2], [300, 128, 1000], 8, 2, 64, 32, 200, 4),
    "rows_64": ([16, 5], [700, 77], 8, 2, 128, 32, 300, 4),
    "rows_64_d64": ([13, 16], [900, 130], 4, 1, 64, 64, 0, 0),
    "rows_128": ([16, 11], [700, 77], 16, 2, 128, 32, 300, 4),
    "rows_128_d64": ([16, 9, 3], [900, 130, 0], 8, 1, 64, 16, 500, 2),
    "rows_128_split": ([16], [5000], 8, 1, 128, 64, 0, 0),
    # enough work that one block takes many tiles of many units, at each tiling
    "busy_16": ([1, 3, 2] * 30, [1500, 700, 1111] * 30, 8, 2, 64, 64, 0, 0),
    "busy_32": ([8, 5, 3] * 25, [1500, 700, 90] * 25, 8, 2, 128, 32, 600, 4),
    "busy_64": ([16, 5, 9] * 12, [1500, 700, 2000] * 12, 16, 4, 64, 16, 900, 4),
    "busy_64_d128": ([16, 5, 9] * 12, [1500, 700, 2000] * 12, 8, 2, 128, 64, 0, 0),
    "busy_128": ([16, 5] * 12, [1500, 300] * 12, 16, 2, 128, 64, 800, 4),
    "busy_128_d64": ([16, 5] * 12, [1500, 300] * 12, 16, 2, 64, 64, 0, 0),
    "busy_prompts": ([90, 40] * 10, [1500, 300] * 10, 8, 2, 128, 64, 500, 4),
    "busy_prompts_d64": ([90, 40] * 10, [1500, 300] * 10, 8, 2, 64, 64, 0, 0),
    "many_requests": ([1 + r % 4 for r in range(150)], [(r * 37) % 300 for r in range(150)], 2, 1, 64, 16, 64, 2),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attention(name):
    ns, ctxs, hq, hkv, d, page, window, sinks = CASES[name]
    c = Cache(ns, ctxs, hkv, d, page, seed=len(name), evict=(window, sinks) if window else None)
    _check_attention(c, hq, window, sinks, seed=3)


@pytest.mark.parametrize("max_rows", [1, 5, 40, 100000])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_any_expected_rows(max_rows, d):
    """max_rows only picks the tiling: right where windows are longer or shorter than expected."""
    c = Cache([1, 70, 9, 0, 200], [500, 3, 130, 7, 64], 2, d, 32, seed=5, evict=(150, 4))
    _check_attention(c, 8, 150, 4, seed=6, max_rows=max_rows)


def test_attention_strided_queries():
    c = Cache([3, 4], [100, 260], 2, 128, 16, seed=7)
    _check_attention(c, 6, 0, 0, seed=8, strided=True)


@pytest.mark.parametrize("q_scale,scale", [(40.0, None), (1.0, 0.0), (1.0, -0.3)])
def test_attention_far_scores(q_scale, scale):
    """Peaked scores (one weight near 1, maxima that jump from tile to tile), equal ones (the mean of the
    values) and a negative scale."""
    c = Cache([3, 9], [1000, 390], 1, 128, 32, seed=9)
    # peaked scores: an error of the fp32 score moves the weights by as much
    hkv, d = 1, 128
    if q_scale > 1:
        c.keys = [np.round(k * 4) / 4 for k in c.keys]  # quarters: products and sums are exact in fp32
        for r, (n, x) in enumerate(zip(c.ns, c.ctxs)):
            for p in range(n + x):
                c.k[c.table[r, p // 32], :, p % 32] = torch.from_numpy(c.keys[r][p]).to(torch.bfloat16).cuda()
        q_scale = 1.0
        g = torch.Generator().manual_seed(10)
        q = (torch.randn(15, 4, d, generator=g) * 8).round()
        rows, hq = 15, 4
        out = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(rows, hq, dtype=torch.float32, device="cuda")
        ws = B.alloc_attention_workspace(hq, hkv, d)
        B.dspark_window_attention(q.to(torch.bfloat16).cuda(), c.k, c.v, c.table, c.cu, c.ctx, 9, 0.25, 0, 0, out, lse, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        first = 0
        for r, n in enumerate(c.ns):
            ref, rl, mag = R.attention(q[first:first + n].numpy().astype(np.float64), c.keys[r], c.vals[r], c.ctxs[r], 0.25, 0, 0)
            assert (np.abs(_f64(out)[first:first + n] - ref) <= R.attention_bound(mag)).all()
            assert np.abs(_f64(lse)[first:first + n] - rl).max() <= 1e-4 * (1 + np.abs(rl).max())
            first += n
        return
    _check_attention(c, 4, 0, 0, seed=10, scale=scale)


@pytest.mark.parametrize("n,hq", [(1, 4), (8, 4), (16, 4), (16, 8), (40, 8)])
def test_attention_scores_that_grow(n, hq):
    """Scores that jump by hundreds from tile to tile, up and down, at each tiling: the reference of the
    exponentials has to follow.  q = 1, key j = c_j in every lane and scale 1 / D: the scores are c_j exactly."""
    d, page, ctx = 64, 32, 900
    c = Cache([n], [ctx], 1, d, page, seed=18)
    step = np.array([0.0, 110.0, -40.0, 300.0, 290.0, 301.0, 1000.0, 990.0])
    level = step[np.minimum(np.arange(ctx + n) // 128, 7)] + (np.arange(ctx + n) % 4) * 0.5
    level = _f64(torch.from_numpy(level).to(torch.bfloat16))
    c.keys[0] = np.repeat(level[:, None, None], d, 2)
    table = c.table.cpu().numpy()
    for j in range(ctx + n):
        c.k[table[0, j // page], :, j % page] = float(level[j])
    # 160 requests over the same pages: enough work that a block takes whole units
    bs = 160
    q = torch.ones(bs * n, hq, d, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(0, bs * n + 1, n, dtype=torch.int32, device="cuda")
    many = c.ctx.repeat(bs), c.table.repeat(bs, 1)
    ws = B.alloc_attention_workspace(hq, 1, d)
    for window, sinks in ((0, 0), (200, 4), (600, 0)):
        out = torch.zeros_like(q)
        lse = torch.zeros(bs * n, hq, device="cuda")
        B.dspark_window_attention(q, c.k, c.v, many[1], cu, many[0], n, 1.0 / d, window, sinks, out, lse, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        ref, rl, mag = R.attention(_f64(q)[:n], c.keys[0], c.vals[0], ctx, 1.0 / d, window, sinks)
        assert (np.abs(_f64(out).reshape(bs, n, hq, d) - ref) <= R.attention_bound(mag)).all()
        assert np.abs(_f64(lse).reshape(bs, n, hq) - rl).max() <= 1e-4 * (1 + np.abs(rl).max())


def test_attention_offsets_beyond_32_bits():
    """Pages whose element offsets pass 2^31 (and byte offsets 2^32)."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 31) // (page * hkv * d) + 40
    c = Cache([2, 3], [200, 500], hkv, d, page, seed=11)
    k = torch.empty(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    shift = n_pages - c.n_pages
    k[shift:], v[shift:] = c.k, c.v
    c.k, c.v = k, v
    c.table = torch.where(c.table >= 0, c.table + shift, c.table)
    _check_attention(c, 16, 0, 0, seed=12)


def test_attention_on_another_stream_and_in_a_graph():
    ns, ctxs = [4, 2, 8], [700, 90, 1500]
    c = Cache(ns, ctxs, 2, 128, 64, seed=13)
    out0, lse0 = _check_attention(c, 8, 0, 0, seed=14, pad=0)
    q = torch.randn(sum(ns), 8, 128, generator=torch.Generator().manual_seed(15)).to(torch.bfloat16).cuda()
    out, lse = torch.zeros_like(out0), torch.zeros_like(lse0)
    ws = B.alloc_attention_workspace(8, 2, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def call(o, l):
        B.dspark_window_attention(q, c.k, c.v, c.table, c.cu, c.ctx, 8, 128 ** -0.5, 0, 0, o, l, ws)

    with torch.cuda.stream(s):
        call(out, lse)
    s.synchronize()
    want, want_lse = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(out, lse)
    out.zero_()
    lse.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)  # and the same bits each time


def test_attention_device_errors():
    """A page number that is no page reads as zeros, a bad length leaves its rows alone, both with EINVAL;
    the other requests' rows are right."""
    c = Cache([2, 2, 2], [100, 100, 100], 1, 64, 16, seed=16)
    q = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(17)).to(torch.bfloat16).cuda()
    out = torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = B.alloc_attention_workspace(2, 1, 64)

    def call():
        B.dspark_window_attention(q, c.k, c.v, c.table, c.cu, c.ctx, 2, 0.125, 0, 0, out, None, ws)
        return B.dspark_read_device_status(ws)

    assert call() == B.DSPARK_OK
    good = out.clone()
    keep = c.table.clone()
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        c.table = keep.clone()
        c.table[1, 2] = bad
        assert call() == B.DSPARK_EINVAL
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
        assert not torch.isnan(out).any()
    c.table = keep
    for bad in (-1, 16 * keep.shape[1] - 1, 2 ** 31 - 1):
        c.ctx = torch.tensor([100, bad, 100], dtype=torch.int32, device="cuda")
        out.fill_(7.0)
        assert call() == B.DSPARK_EINVAL
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:]) and (out[2:4] == 7.0).all()
    c.ctx = torch.tensor([100, 100, 100], dtype=torch.int32, device="cuda")
    cu = c.cu
    for bad in ([0, 2, 4, 7], [0, 4, 2, 6], [-1, 2, 4, 6]):
        c.cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out.fill_(7.0)
        assert call() == B.DSPARK_EINVAL
        assert (out == 7.0).all()
    c.cu = cu
    assert call() == B.DSPARK_OK and torch.equal(out, good)


@pytest.mark.parametrize("rows,hq", [(1, 4), (8, 4), (16, 8), (60, 4)])
def test_attention_wait_timeout_is_reported_and_recovers(rows, hq):
    """With a deadline of 1 ns the kernels' waits run out: they report it, drain their copies and MMAs and
    return; the next call with the normal deadline is right again, on the same workspace."""
    # enough tiles for each block that its ring of tiles goes round
    c = Cache([rows] * 20, [1500] * 20, 2, 64, 32, seed=19)
    many = 12
    c.table, c.ctx = c.table.repeat(many, 1), c.ctx.repeat(many)
    c.cu = torch.arange(0, 20 * many * rows + 1, rows, dtype=torch.int32, device="cuda")
    q = torch.randn(20 * many * rows, 2 * hq, 64, generator=torch.Generator().manual_seed(20)).to(torch.bfloat16).cuda()
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    ws = B.alloc_attention_workspace(2 * hq, 2, 64)

    def call(o):
        B.dspark_window_attention(q, c.k, c.v, c.table, c.cu, c.ctx, rows, 0.125, 1000, 4, o, None, ws)
        return B.dspark_read_device_status(ws)

    assert call(want) == B.DSPARK_OK
    old = B.dspark_set_wait_timeout_ns(1)
    try:
        st = call(out)
    finally:
        B.dspark_set_wait_timeout_ns(old)
    assert st == B.DSPARK_ETIMEOUT, B.dspark_status_string(st)
    assert call(out) == B.DSPARK_OK and torch.equal(out, want)


# ------------------------------------------------------------------------------- append

def _table(max_pos, rot, dtype=np.float32):
    t = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return np.concatenate([np.cos(t), np.sin(t)], 1).astype(dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("ns,ctxs,hq,hkv,d,page,rot", [
    ([1], [0], 4, 1, 128, 16, 128),
    ([3, 0, 1, 8], [14, 3, 63, 120], 8, 2, 128, 16, 64),
    ([2, 5], [31, 0], 3, 3, 64, 32, 64),
    ([1] * 70, list(range(70)), 2, 1, 64, 8, 16),
    ([2100, 2300], [0, 77], 2, 1, 64, 128, 32),
    ([40, 13], [250, 5], 10, 2, 128, 256, 112),
])
def test_append(ns, ctxs, hq, hkv, d, page, rot, interleaved):
    c = Cache(ns, ctxs, hkv, d, page, seed=21, fill=5.0)
    rows = sum(ns) + 2
    g = torch.Generator().manual_seed(22)
    qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cs = _table(max(x + n for x, n in zip(ctxs, ns)) + 1, rot)
    k0, v0 = c.k.clone(), c.v.clone()
    q_out = torch.full((rows, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = _status_ws()
    B.dspark_append_kv(q, k, v, c.cu, c.ctx, torch.from_numpy(cs).cuda(), c.table, q_out, c.k, c.v, ws,
                       interleaved=interleaved)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    first, table = 0, c.table.cpu().numpy()
    half = rot // 2
    kc, vc, qo = _f64(c.k), _f64(c.v), _f64(q_out)
    for r, (n, x) in enumerate(zip(ns, ctxs)):
        pos = np.arange(x, x + n)
        cos, sin = (cs[pos][:, None, s].astype(np.float64) for s in (slice(0, half), slice(half, rot)))
        pages = table[r, pos // page]
        for got, src in ((qo[first:first + n], q), (kc[pages, :, pos % page], k)):
            src = _f64(src)[first:first + n]
            ref = R.rotate(src, cos, sin, interleaved)
            # fp32 products and sums of the pair, then one rounding to bf16
            size = np.abs(R.rotate(np.abs(src), np.abs(cos), -np.abs(sin), interleaved)) + np.abs(src).max(initial=0.0)
            assert (np.abs(got - ref) <= R.BF16 * np.abs(ref) + 1e-6 * size).all()
        assert np.array_equal(vc[pages, :, pos % page], _f64(v)[first:first + n])
        first += n
    # nothing else was touched: undo the appended slots and compare whole caches
    for r, (n, x) in enumerate(zip(ns, ctxs)):
        pos = torch.arange(x, x + n, device="cuda")
        pages = c.table[r][pos // page].long()
        c.k[pages, :, pos % page] = k0[pages, :, pos % page]
        c.v[pages, :, pos % page] = v0[pages, :, pos % page]
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)
    assert (q_out[sum(ns):] == 7.0).all()


def test_append_in_place_and_keys_only():
    c = Cache([3, 2], [10, 40], 2, 128, 16, seed=23, fill=0.0)
    g = torch.Generator().manual_seed(24)
    q = torch.randn(5, 4, 128, generator=g).to(torch.bfloat16).cuda()
    k = torch.randn(5, 2, 128, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(5, 2, 128, generator=g).to(torch.bfloat16).cuda()
    cs = torch.from_numpy(_table(64, 128)).cuda()
    ws, q_out = _status_ws(), torch.empty_like(q)
    c.k.zero_(), c.v.zero_()
    B.dspark_append_kv(q, k, v, c.cu, c.ctx, cs, c.table, q_out, c.k, c.v, ws)
    k1, v1 = c.k.clone(), c.v.clone()
    c.k.zero_(), c.v.zero_()
    B.dspark_append_kv(None, k, v, c.cu, c.ctx, cs, c.table, None, c.k, c.v, ws)
    assert torch.equal(c.k, k1) and torch.equal(c.v, v1) and (k1 != 0).any()
    B.dspark_append_kv(q, k, v, c.cu, c.ctx, cs, c.table, q, c.k, c.v, ws)
    assert torch.equal(q, q_out) and B.dspark_read_device_status(ws) == B.DSPARK_OK


def test_append_device_errors():
    c = Cache([2, 2], [30, 30], 1, 64, 16, seed=25, fill=0.0)
    q = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    cs = torch.from_numpy(_table(40, 64)).cuda()
    ws, q_out = _status_ws(), torch.full_like(q, 7.0)
    keep = c.table.clone()

    def call():
        k0 = c.k.clone()
        q_out.fill_(7.0)
        B.dspark_append_kv(q, q, q, c.cu, c.ctx, cs, c.table, q_out, c.k, c.v, ws)
        st = B.dspark_read_device_status(ws)
        changed = (c.k != k0).any().item()
        c.k.copy_(k0)
        return st, changed

    for bad in (-1, c.n_pages, 2 ** 31 - 1):
        c.table = keep.clone()
        c.table[1, 1] = bad  # positions 30, 31 of request 1
        st, _ = call()
        assert st == B.DSPARK_EINVAL and (q_out[2:] == 7.0).all() and not (q_out[:2] == 7.0).any()
    c.table = keep
    for bad in (-1, 39, 2 ** 31 - 1):  # below 0; the second row beyond the table of angles; far beyond
        c.ctx = torch.tensor([30, bad], dtype=torch.int32, device="cuda")
        st, _ = call()
        assert st == B.DSPARK_EINVAL and (q_out[3] == 7.0).all() and not (q_out[:2] == 7.0).any()
    c.ctx = torch.tensor([30, 30], dtype=torch.int32, device="cuda")
    c.cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")  # more rows than there are
    st, changed = call()
    assert st == B.DSPARK_EINVAL and not changed and (q_out == 7.0).all()


def test_append_then_attend_matches_one_sequence():
    """Appending windows one after another and attending equals attention over the whole sequence."""
    hq, hkv, d, page, total = 4, 2, 64, 16, 90
    g = torch.Generator().manual_seed(26)
    q = torch.randn(total, hq, d, generator=g).to(torch.bfloat16).cuda()
    k = torch.randn(total, hkv, d, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(total, hkv, d, generator=g).to(torch.bfloat16).cuda()
    kc = torch.full((8, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    table = torch.tensor([[5, 2, 7, 0, 1, 6]], dtype=torch.int32, device="cuda")
    cs = torch.from_numpy(_table(total, d)).cuda()
    ws = B.alloc_attention_workspace(hq, hkv, d)
    got = []
    at = 0
    for n in (40, 1, 8, 3, 30, 8):
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ctx = torch.tensor([at], dtype=torch.int32, device="cuda")
        qr = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        o = torch.empty_like(qr)
        B.dspark_append_kv(q[at:at + n], k[at:at + n], v[at:at + n], cu, ctx, cs, table, qr, kc, vc, ws)
        B.dspark_window_attention(qr, kc, vc, table, cu, ctx, n, d ** -0.5, 25, 3, o, None, ws)
        got.append(o)
        at += n
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    c64 = _table(total, d).astype(np.float64)
    cos, sin = c64[:, None, :d // 2], c64[:, None, d // 2:]

    def bf(x):
        return _f64(torch.from_numpy(x).to(torch.bfloat16))

    qn, kn = bf(R.rotate(_f64(q), cos, sin, False)), bf(R.rotate(_f64(k), cos, sin, False))
    ref, _, mag = R.attention(qn, kn, _f64(v), 0, d ** -0.5, 25, 3)
    # a rotated value that lies at a tie may round either way: one bf16 step in a score's term at most
    slack = R.BF16 * mag
    assert (np.abs(_f64(torch.cat(got)) - ref) <= R.attention_bound(mag) + slack).all()
