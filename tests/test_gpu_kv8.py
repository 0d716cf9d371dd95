"""The 8-bit paged cache on the GPU: the quantising append, the attention over it and reading it back, against plain 64-bit
forms, at the sizes, masks and page layouts where they can go wrong."""
import numpy as np
import pytest

from tests import kv8_reference as K
from tests import serving_reference as R

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from tests.test_gpu_attention import CASES, _f64, _status_ws, _table  # noqa: E402

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


class Cache8:
    """An 8-bit paged cache with pages in random order; what no request owns is NaN, by its codes and by its exponents."""

    def __init__(self, ns, ctxs, hkv, d, page, seed, extra_pages=2, evict=None, spread=3):
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
        shape = (self.n_pages, hkv, page, d)
        k, v = (np.full(shape, 127, np.uint8) for _ in range(2))
        scale = np.full(shape[:3] + (2,), 255, np.uint8)
        self.keys, self.vals = [], []
        for r, (n, c) in enumerate(zip(ns, ctxs)):
            pos = np.arange(c + n)
            at = table[r, pos // page], slice(None), pos % page
            for which, (codes, kept) in enumerate(((k, self.keys), (v, self.vals))):
                x = rng.standard_normal((c + n, hkv, d)) * 2.0 ** rng.integers(-spread, spread + 1, (c + n, hkv, 1))
                if which == 0:  # scores of unit size whatever the vector's: an error of the score moves the weights by as much
                    x = x / np.abs(x).max(-1, keepdims=True) * 2.5
                byte = K.exponent_byte(x)
                code = K.codes(x, byte)
                codes[at], scale[at + (which,)] = code, byte
                kept.append(K.values(code, byte))
        if evict:  # (window, sinks): what no row sees any more is NaN; its whole pages leave the table
            window, sinks = evict
            for r, c in enumerate(ctxs):
                pos = np.arange(sinks, max(sinks, c - window + 1))
                k[table[r, pos // page], :, pos % page] = 255
                v[table[r, pos // page], :, pos % page] = 127
                scale[table[r, pos // page], :, pos % page] = 255
                first, last = -(-sinks // page), (max(0, c - window + 1)) // page
                table[r, first:max(first, last)] = -1
        self.table = torch.from_numpy(table).cuda()
        self.k, self.v = (torch.from_numpy(x).cuda().view(F8) for x in (k, v))
        self.scale = torch.from_numpy(scale).cuda()
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device="cuda")
        self.ctx = torch.tensor(ctxs, dtype=torch.int32, device="cuda")

    def scratch(self):
        return [torch.full(self.k.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]


def _check(c, hq, window, sinks, seed, max_rows=None, pad=3, strided=False, scale=None, scratch=False, q=None):
    hkv, d = c.k.shape[1], c.k.shape[3]
    rows = sum(c.ns) + pad
    if q is None:
        q = torch.randn(rows, hq, d, generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16)
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
    ks, vs = c.scratch() if scratch else (None, None)
    for _ in range(2):  # the second call runs on a workspace that has been used
        B.dspark_window_attention_kv8(qd, c.k, c.v, c.scale, c.table, c.cu, c.ctx, max_rows, scale, window, sinks, out, lse,
                                      ks, vs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    got, got_lse, qn = _f64(out), _f64(lse), _f64(q)
    first = 0
    for r, n in enumerate(c.ns):
        ref, rl, mag = R.attention(qn[first:first + n], c.keys[r], c.vals[r], c.ctxs[r], scale, window, sinks)
        assert not np.isnan(got[first:first + n]).any(), (r, n)
        off = np.abs(got[first:first + n] - ref) - R.attention_bound(mag)
        assert off.max(initial=-1.0) <= 0, (r, n, off.max())
        assert np.abs(got_lse[first:first + n] - rl).max(initial=0.0) <= 1e-4 * (1.0 + np.abs(rl).max(initial=0.0))
        first += n
    assert (got[first:] == 7.0).all() and (got_lse[first:] == 7.0).all()  # pad rows are left alone
    return out, lse


@pytest.mark.parametrize("name", list(CASES))
def test_attention(name):
    ns, ctxs, hq, hkv, d, page, window, sinks = CASES[name]
    c = Cache8(ns, ctxs, hkv, d, page, seed=len(name), evict=(window, sinks) if window else None)
    _check(c, hq, window, sinks, seed=3)


@pytest.mark.parametrize("name", ["one_token", "prompts", "prompt_window", "prompt_group_5", "busy_prompts", "rows_128_d64"])
def test_attention_with_pages_to_read_back_to(name):
    ns, ctxs, hq, hkv, d, page, window, sinks = CASES[name]
    c = Cache8(ns, ctxs, hkv, d, page, seed=len(name), evict=(window, sinks) if window else None)
    _check(c, hq, window, sinks, seed=3, scratch=True)


@pytest.mark.parametrize("scratch", [False, True])
@pytest.mark.parametrize("max_rows", [1, 5, 40, 100000])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_any_expected_rows(max_rows, d, scratch):
    c = Cache8([1, 70, 9, 0, 200], [500, 3, 130, 7, 64], 2, d, 32, seed=5, evict=(150, 4))
    _check(c, 8, 150, 4, seed=6, max_rows=max_rows, scratch=scratch)


def test_attention_strided_queries():
    c = Cache8([3, 4], [100, 260], 2, 128, 16, seed=7)
    _check(c, 6, 0, 0, seed=8, strided=True)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_attention_other_scales(scale):
    c = Cache8([3, 9], [1000, 390], 1, 128, 32, seed=9)
    _check(c, 4, 0, 0, seed=10, scale=scale)


@pytest.mark.parametrize("n,hq", [(1, 4), (8, 4), (16, 4), (16, 8)])
def test_queries_of_every_size(n, hq):
    """Rows whose queries are tiny, huge (beyond fp16), zero, or of one large lane among small ones, in one tile: each
    keeps its own precision.  Keys of the opposite size bring the scores back to unit size."""
    d = 64
    c = Cache8([n] * 3, [300, 140, 1], 1, d, 32, seed=11)
    g = torch.Generator().manual_seed(12)
    q = torch.randn(3 * n + 3, hq, d, generator=g)
    power = torch.tensor([0, -60, 20, 40, -100, 0, 7, -3])[torch.arange((3 * n + 3) * hq) % 8].view(-1, hq, 1)
    q = torch.where(power == 7, torch.where(torch.arange(d) == 5, 60.0 * q, q / 16), q * 2.0 ** power.clamp(max=0))
    q = torch.where(power == -3, torch.zeros_like(q), q).to(torch.bfloat16)
    _check(c, hq, 0, 0, seed=13, q=q)


@pytest.mark.parametrize("power", [-90, -20, 30, 90])
def test_caches_of_every_size(power):
    """K times 2^power under queries times 2^-power, and V times 2^power: the outputs are the same ones times 2^power."""
    c = Cache8([4, 2], [200, 31], 2, 128, 16, seed=14)
    q = torch.randn(9, 4, 128, generator=torch.Generator().manual_seed(15)).to(torch.bfloat16)
    out, lse = _check(c, 4, 0, 0, seed=15, q=q)
    owned = c.scale != 255
    c.scale = torch.where(owned, c.scale.int() + power, 255).to(torch.uint8)
    ws = B.alloc_attention_workspace(4, 2, 128)
    got, got_lse = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    B.dspark_window_attention_kv8((q.double() * 2.0 ** -power).to(torch.bfloat16).cuda(), c.k, c.v, c.scale, c.table, c.cu,
                                  c.ctx, 4, 128 ** -0.5, 0, 0, got, got_lse, None, None, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    assert torch.equal(got[:6], (out[:6].double() * 2.0 ** power).to(torch.bfloat16)) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("n,hq", [(1, 4), (8, 4), (16, 4), (16, 8), (40, 8)])
def test_attention_scores_that_grow(n, hq):
    """Scores that jump by hundreds from tile to tile, up and down, and values whose powers of two jump by ten: the references
    have to follow.  q = 1, key j = c_j in every lane and scale 1 / D: the scores are c_j exactly."""
    d, page, ctx = 64, 32, 900
    c = Cache8([n], [ctx], 1, d, page, seed=18)
    step = np.array([0.0, 112.0, -40.0, 288.0, 256.0, 320.0, 1024.0, 960.0])
    level = step[np.minimum(np.arange(ctx + n) // 128, 7)]
    up = np.array([0, 10, -10, 4, 12, -3, 0, 11])[np.minimum(np.arange(ctx + n) // 128, 7)]
    c.keys[0] = np.repeat(level[:, None, None], d, 2)
    c.vals[0] = c.vals[0] * 2.0 ** up[:, None, None]
    byte = K.exponent_byte(c.keys[0])
    code = K.codes(c.keys[0], byte)
    assert (K.values(code, byte) == c.keys[0]).all()
    table = c.table.cpu().numpy()[0]
    pos = np.arange(ctx + n)
    k, s = _codes(c.k).copy(), c.scale.cpu().numpy().copy()
    k[table[pos // page], :, pos % page] = code
    s[table[pos // page], :, pos % page, 0] = byte
    s[table[pos // page], :, pos % page, 1] += up[:, None].astype(np.uint8)
    c.k, c.scale = torch.from_numpy(k).cuda().view(F8), torch.from_numpy(s).cuda()
    # 160 requests over the same pages: enough work that a block takes whole units
    bs = 160
    q = torch.ones(bs * n, hq, d, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(0, bs * n + 1, n, dtype=torch.int32, device="cuda")
    many = c.ctx.repeat(bs), c.table.repeat(bs, 1)
    ws = B.alloc_attention_workspace(hq, 1, d)
    for window, sinks in ((0, 0), (200, 4), (600, 0)):
        out = torch.zeros_like(q)
        lse = torch.zeros(bs * n, hq, device="cuda")
        B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, many[1], cu, many[0], n, 1.0 / d, window, sinks, out, lse, None,
                                      None, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        ref, rl, mag = R.attention(_f64(q)[:n], c.keys[0], c.vals[0], ctx, 1.0 / d, window, sinks)
        assert (np.abs(_f64(out).reshape(bs, n, hq, d) - ref) <= R.attention_bound(mag)).all()
        assert np.abs(_f64(lse).reshape(bs, n, hq) - rl).max() <= 1e-4 * (1 + np.abs(rl).max())


def test_vectors_of_nan_reach_the_rows_that_see_them():
    """An exponent byte of 255 in K or V of a position: the rows from there on are NaN; rows of other requests are not."""
    for which in (0, 1):
        c = Cache8([4, 4], [150, 150], 1, 64, 16, seed=30)
        out, _ = _check(c, 2, 0, 0, seed=31)
        c.scale[c.table[0, 151 // 16], 0, 151 % 16, which] = 255  # row 1's own position
        ws, got = B.alloc_attention_workspace(2, 1, 64), torch.zeros_like(out)
        q = torch.randn(11, 2, 64, generator=torch.Generator().manual_seed(32)).to(torch.bfloat16).cuda()
        B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, c.cu, c.ctx, 4, 0.125, 0, 0, got, None, None, None, ws)
        assert torch.isnan(got[1:4]).all() and not torch.isnan(got[4:8]).any()
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK


def test_attention_offsets_beyond_32_bits():
    """Pages whose offsets pass 2^32 bytes, in the codes."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * hkv * d) + 40
    c = Cache8([2, 3], [200, 500], hkv, d, page, seed=11)
    shift = n_pages - c.n_pages
    for name in ("k", "v", "scale"):
        old = getattr(c, name)
        new = torch.empty((n_pages,) + old.shape[1:], dtype=old.dtype, device="cuda")
        new.view(torch.uint8)[shift:] = old.view(torch.uint8)
        setattr(c, name, new)
    c.table = torch.where(c.table >= 0, c.table + shift, c.table)
    _check(c, 16, 0, 0, seed=12)


def test_attention_on_another_stream_and_in_a_graph():
    ns, ctxs = [4, 2, 8], [700, 90, 1500]
    c = Cache8(ns, ctxs, 2, 128, 64, seed=13)
    out0, lse0 = _check(c, 8, 0, 0, seed=14, pad=0)
    q = torch.randn(sum(ns), 8, 128, generator=torch.Generator().manual_seed(15)).to(torch.bfloat16).cuda()
    out, lse = torch.zeros_like(out0), torch.zeros_like(lse0)
    ws = B.alloc_attention_workspace(8, 2, 128)
    scratch = c.scratch()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for max_rows in (8, 100):  # the windows' kernel, and reading back first
        def call():
            B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, c.cu, c.ctx, max_rows, 128 ** -0.5, 0, 0, out, lse,
                                          *scratch, ws)

        with torch.cuda.stream(s):
            call()
        s.synchronize()
        want, want_lse = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        out.zero_()
        lse.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)  # and the same bits each time


def test_attention_in_place():
    c = Cache8([3, 9], [1000, 390], 2, 128, 32, seed=9)
    q = torch.randn(12, 8, 128, generator=torch.Generator().manual_seed(15)).to(torch.bfloat16).cuda()
    ws, out = B.alloc_attention_workspace(8, 2, 128), torch.zeros_like(q)
    B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, c.cu, c.ctx, 9, 0.1, 0, 0, out, None, None, None, ws)
    B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, c.cu, c.ctx, 9, 0.1, 0, 0, q, None, None, None, ws)
    assert torch.equal(q, out)


@pytest.mark.parametrize("scratch", [False, True])
def test_attention_device_errors(scratch):
    """A page number that is no page reads as zeros, a bad length leaves its rows alone, both with EINVAL; the other
    requests' rows are right."""
    c = Cache8([2, 2, 2], [100, 100, 100], 1, 64, 16, seed=16)
    q = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(17)).to(torch.bfloat16).cuda()
    out = torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = B.alloc_attention_workspace(2, 1, 64)
    pages = [torch.zeros(c.k.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)] if scratch else (None, None)

    def call():
        B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, c.cu, c.ctx, 100 if scratch else 2, 0.125, 0, 0, out,
                                      None, *pages, ws)
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


# ------------------------------------------------------------------------------- append

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("ns,ctxs,hq,hkv,d,page,rot", [
    ([1], [0], 4, 1, 128, 16, 128),
    ([3, 0, 1, 8], [14, 3, 63, 120], 8, 2, 128, 16, 64),
    ([2, 5], [31, 0], 3, 3, 64, 32, 64),
    ([1] * 70, list(range(70)), 2, 1, 64, 8, 16),
    ([2100, 2300], [0, 77], 2, 1, 64, 128, 32),
    ([40, 13], [250, 5], 10, 2, 128, 256, 112),
    ([2], [5], 33, 3, 64, 16, 48),
])
def test_append(ns, ctxs, hq, hkv, d, page, rot, interleaved):
    c = Cache8(ns, ctxs, hkv, d, page, seed=21)
    rows = sum(ns) + 2
    g = torch.Generator().manual_seed(22)
    size = 2.0 ** torch.randint(-30, 30, (rows, hq + 2 * hkv, 1), generator=g)
    qkv = (torch.randn(rows, hq + 2 * hkv, d, generator=g) * size).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cs = _table(max(x + n for x, n in zip(ctxs, ns)) + 1, rot)
    before = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.scale)]
    q_out = torch.full((rows, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = _status_ws()
    B.dspark_append_kv8(q, k, v, c.cu, c.ctx, torch.from_numpy(cs).cuda(), c.table, q_out, c.k, c.v, c.scale, ws,
                        interleaved=interleaved)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    first, table, half = 0, c.table.cpu().numpy(), rot // 2
    kc, vc, sc, qo = _codes(c.k), _codes(c.v), c.scale.cpu().numpy(), _f64(q_out)
    for r, (n, x) in enumerate(zip(ns, ctxs)):
        pos = np.arange(x, x + n)
        cos, sin = (cs[pos][:, None, s].astype(np.float64) for s in (slice(0, half), slice(half, rot)))
        at = table[r, pos // page], slice(None), pos % page
        rows_r = slice(first, first + n)

        def turned(t):
            src = _f64(t)[rows_r]
            size = np.abs(R.rotate(np.abs(src), np.abs(cos), -np.abs(sin), interleaved)) + np.abs(src).max(-1, initial=0.0, keepdims=True)
            return R.rotate(src, cos, sin, interleaved), size

        ref, size = turned(q)
        assert (np.abs(qo[rows_r] - ref) <= R.BF16 * np.abs(ref) + 1e-6 * size).all()
        ref, size = turned(k)
        power = 2.0 ** (sc[at + (0,)].astype(float) - 127)[..., None]
        top = np.abs(ref).max(-1, initial=0.0, keepdims=True)
        assert (top <= 448 * power * (1 + 1e-6)).all() and (top * (1 + 1e-6) > 224 * power).all()
        got = K.values(kc[at], sc[at + (0,)])
        assert (np.abs(got - ref) <= np.maximum(K.E4M3 * np.abs(ref), 2.0 ** -10 * power) + 1e-6 * size).all()
        val = _f64(v)[rows_r]
        byte = K.exponent_byte(val)
        assert np.array_equal(sc[at + (1,)], byte) and np.array_equal(vc[at], K.codes(val, byte))
        first += n
    # nothing else was touched: undo the appended slots and compare whole caches
    after = [c.k.view(torch.uint8), c.v.view(torch.uint8), c.scale]
    for r, (n, x) in enumerate(zip(ns, ctxs)):
        pos = torch.arange(x, x + n, device="cuda")
        pages = c.table[r][pos // page].long()
        for a, b in zip(after, before):
            a[pages, :, pos % page] = b[pages, :, pos % page]
    assert all(torch.equal(a, b) for a, b in zip(after, before))
    assert (q_out[sum(ns):] == 7.0).all()


def test_append_special_vectors():
    """Zeros, one tiny value, values at the borders of the powers of two, the largest bf16, NaN and infinities."""
    d, page = 64, 16
    big = torch.finfo(torch.bfloat16).max
    rows = [torch.zeros(d), torch.full((d,), -0.0), torch.full((d,), 448.0), torch.full((d,), 450.0), torch.full((d,), 224.0),
            torch.full((d,), 1e-40), torch.full((d,), 2.0 ** -126), torch.full((d,), big), torch.full((d,), -big),
            torch.full((d,), float("nan")), torch.full((d,), float("inf")), torch.arange(d) * 7.0,
            torch.cat([torch.tensor([float("-inf")]), torch.ones(d - 1)]), torch.cat([torch.ones(d - 1), torch.tensor([float("nan")])]),
            torch.cat([torch.tensor([1000.0]), torch.full((d - 1,), 2.0 ** -9)])]
    x = torch.stack(rows)[:, None].to(torch.bfloat16)
    n = len(rows)
    k, v = (torch.full((2, 1, page, d), 1.0, device="cuda").to(F8) for _ in range(2))
    scale = torch.full((2, 1, page, 2), 3, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    cs = torch.from_numpy(_table(40, 16)).cuda()
    cs[:, :8], cs[:, 8:] = 1.0, 0.0  # turned by nothing
    ws = _status_ws()
    B.dspark_append_kv8(None, x.cuda(), x.cuda(), torch.tensor([0, n], **i32), torch.tensor([0], **i32), cs,
                        torch.tensor([[1]], **i32), None, k, v, scale, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    ref = _f64(x)
    byte = K.exponent_byte(ref)
    good = byte[:, 0] != 255
    codes = K.codes(np.where(np.isfinite(ref), ref, 0.0), byte)
    for c, which in ((v, 1), (k, 0)):
        assert np.array_equal(scale[1, 0, :n, which].cpu().numpy(), byte[:, 0])
        got = _codes(c)[1, 0, :n]
        same = got == codes[:, 0]
        if which == 0:  # a pair's difference or sum with a product of 0 loses the sign of a zero
            same |= (got & 127 == 0) & (codes[:, 0] & 127 == 0)
        assert same[good].all() and (got[~good] == 0).all()
    assert byte[:, 0].tolist()[:5] == [1, 1, 127, 128, 126] and (~good).sum() == 4


def test_append_in_place_and_keys_only():
    c = Cache8([3, 2], [10, 40], 2, 128, 16, seed=23)
    g = torch.Generator().manual_seed(24)
    q = torch.randn(5, 4, 128, generator=g).to(torch.bfloat16).cuda()
    k = torch.randn(5, 2, 128, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(5, 2, 128, generator=g).to(torch.bfloat16).cuda()
    cs = torch.from_numpy(_table(64, 128)).cuda()
    ws, q_out = _status_ws(), torch.empty_like(q)

    def cleared():
        for t in (c.k, c.v, c.scale):
            t.view(torch.uint8).zero_()

    cleared()
    B.dspark_append_kv8(q, k, v, c.cu, c.ctx, cs, c.table, q_out, c.k, c.v, c.scale, ws)
    first = [t.view(torch.uint8).clone() for t in (c.k, c.v, c.scale)]
    cleared()
    B.dspark_append_kv8(None, k, v, c.cu, c.ctx, cs, c.table, None, c.k, c.v, c.scale, ws)
    assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(first, (c.k, c.v, c.scale))) and (first[0] != 0).any()
    B.dspark_append_kv8(q, k, v, c.cu, c.ctx, cs, c.table, q, c.k, c.v, c.scale, ws)
    assert torch.equal(q, q_out) and B.dspark_read_device_status(ws) == B.DSPARK_OK


def test_append_device_errors():
    c = Cache8([2, 2], [30, 30], 1, 64, 16, seed=25)
    q = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    cs = torch.from_numpy(_table(40, 64)).cuda()
    ws, q_out = _status_ws(), torch.full_like(q, 7.0)
    keep = c.table.clone()

    def call():
        old = [t.view(torch.uint8).clone() for t in (c.k, c.v, c.scale)]
        q_out.fill_(7.0)
        B.dspark_append_kv8(q, q, q, c.cu, c.ctx, cs, c.table, q_out, c.k, c.v, c.scale, ws)
        st = B.dspark_read_device_status(ws)
        changed = any((t.view(torch.uint8) != o).any().item() for t, o in zip((c.k, c.v, c.scale), old))
        for t, o in zip((c.k, c.v, c.scale), old):
            t.view(torch.uint8).copy_(o)
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


# ------------------------------------------------------------------------------- reading back

@pytest.mark.parametrize("ns,ctxs,hkv,d,page,window,sinks", [
    ([1], [0], 1, 128, 16, 0, 0),
    ([1, 3], [200, 31], 2, 64, 8, 0, 0),
    ([2, 0, 5], [500, 60, 129], 2, 128, 32, 100, 4),
    ([4], [300], 1, 64, 16, 20, 40),
    ([300, 1], [50, 4100], 1, 64, 256, 1000, 3),
    ([8, 2], [140, 900], 3, 128, 64, 128, 130),
    ([1] * 256, [(37 * r) % 700 for r in range(256)], 1, 64, 128, 64, 2),
])
@pytest.mark.parametrize("own_pages", [False, True])
def test_read(ns, ctxs, hkv, d, page, window, sinks, own_pages):
    c = Cache8(ns, ctxs, hkv, d, page, seed=40, evict=(window, sinks) if window else None)
    # other pages, more of them
    to = c.table if own_pages else torch.where(c.table >= 0, c.n_pages + 2 - c.table, -1)
    shape = (c.n_pages + (0 if own_pages else 3), hkv, page, d)
    outs = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = _status_ws()
    B.dspark_read_kv8(c.k, c.v, c.scale, c.table, c.cu, c.ctx, sum(ns), window, sinks, to, *outs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    want = [np.full(shape, 7.0) for _ in range(2)]
    table = to.cpu().numpy()
    for r, (n, x) in enumerate(zip(ns, ctxs)):
        pos = np.arange(x + n) if n else np.arange(0)
        if window:
            pos = pos[(pos > x - window) | (pos < sinks)]
        for w, kept in zip(want, (c.keys, c.vals)):
            w[table[r, pos // page], :, pos % page] = kept[r][pos]
    for o, w in zip(outs, want):
        assert np.array_equal(_f64(o), w)


def test_read_extremes_and_errors():
    """Exponents from end to end, NaN vectors; pages that are none, on either side, are left out with EINVAL."""
    c = Cache8([1, 1], [40, 40], 1, 64, 16, seed=41, spread=0)
    rng = np.random.default_rng(42)
    table = c.table.cpu().numpy()
    s = c.scale.cpu().numpy()
    pos = np.arange(41)
    s[table[0, pos // 16], 0, pos % 16] = rng.integers(1, 246, (41, 2))
    s[table[0, 0], 0, 3] = 255
    c.scale = torch.from_numpy(s).cuda()
    outs = [torch.full(c.k.shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = _status_ws()

    def call():
        B.dspark_read_kv8(c.k, c.v, c.scale, c.table, c.cu, c.ctx, 2, 0, 0, to, *outs, ws)
        return B.dspark_read_device_status(ws)

    to = c.table
    assert call() == B.DSPARK_OK
    for which, (codes, out) in enumerate(((c.k, outs[0]), (c.v, outs[1]))):
        at = table[0, pos // 16], 0, pos % 16
        ref = K.values(_codes(codes)[at], s[at + (which,)])
        got = _f64(out)[at]
        # one rounding to bf16, whose least step is 2^-133
        fine = np.abs(got - ref) <= np.maximum(R.BF16 * np.abs(ref), 2.0 ** -134)
        assert (fine | (np.isnan(got) & np.isnan(ref))).all() and np.isnan(got[3]).all()
        normal = np.abs(ref) >= 2.0 ** -126
        assert (got[normal] == ref[normal]).all()
    good = [o.clone() for o in outs]
    keep = c.table.clone()
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        for source in (True, False):
            c.table, to = keep.clone(), keep.clone()
            (c.table if source else to)[1, 1] = bad
            for o in outs:
                o.fill_(7.0)
            assert call() == B.DSPARK_EINVAL
            for o, g in zip(outs, good):
                left = int(keep[1, 1])
                assert (o[left] == 7.0).all()
                rest = [p for p in range(c.n_pages) if p != left]
                assert torch.equal(o[rest].view(torch.int16), g[rest].view(torch.int16))
    c.table = to = keep
    c.cu = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    for o in outs:
        o.fill_(7.0)
    assert call() == B.DSPARK_EINVAL and all((o == 7.0).all() for o in outs)


def test_append_attend_and_read_agree():
    """Appending windows one after another, attending, and reading back: the attention is that of what is read back."""
    hq, hkv, d, page, total = 4, 2, 64, 16, 90
    g = torch.Generator().manual_seed(26)
    q = torch.randn(total, hq, d, generator=g).to(torch.bfloat16).cuda()
    k = torch.randn(total, hkv, d, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(total, hkv, d, generator=g).to(torch.bfloat16).cuda()
    c8 = [torch.full((8, hkv, page, d), 127, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
    sc = torch.full((8, hkv, page, 2), 255, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[5, 2, 7, 0, 1, 6]], dtype=torch.int32, device="cuda")
    cs = torch.from_numpy(_table(total, d)).cuda()
    ws = B.alloc_attention_workspace(hq, hkv, d)
    outs = [torch.zeros(8, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    at = 0
    i32 = dict(dtype=torch.int32, device="cuda")
    for n in (40, 1, 8, 3, 30, 8):
        cu, ctx = torch.tensor([0, n], **i32), torch.tensor([at], **i32)
        qr = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        got, want = torch.empty_like(qr), torch.empty_like(qr)
        B.dspark_append_kv8(q[at:at + n], k[at:at + n], v[at:at + n], cu, ctx, cs, table, qr, *c8, sc, ws)
        B.dspark_window_attention_kv8(qr, *c8, sc, table, cu, ctx, n, d ** -0.5, 25, 3, got, None, None, None, ws)
        B.dspark_read_kv8(*c8, sc, table, cu, ctx, n, 25, 3, table, *outs, ws)
        at += n
        # 64 bits on what was read back
        pages = table[0].long()
        pos = torch.arange(at, device="cuda")
        keys, vals = (_f64(o[pages[pos // page], :, pos % page]) for o in outs)
        ref, _, mag = R.attention(_f64(qr), keys, vals, at - n, d ** -0.5, 25, 3)
        assert (np.abs(_f64(got) - ref) <= R.attention_bound(mag)).all()
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    assert (np.abs(vals - _f64(v)) <= np.maximum(K.E4M3 * np.abs(_f64(v)), 2.0 ** -10 * np.abs(_f64(v)).max(-1, keepdims=True) / 224)).all()
