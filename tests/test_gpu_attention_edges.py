"""The target-side calls where memory, masks and waits can go wrong: work that fits the attention's rings when a wait
runs out, tensors at the least alignment that is allowed."""
import numpy as np
import pytest

from tests import serving_reference as R

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from tests.test_gpu_attention import Cache, _check_attention, _f64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,hq,ctx", [(1, 2, 10), (8, 4, 200), (16, 8, 300), (60, 4, 200), (200, 4, 60)])
def test_waits_that_run_out_over_little_work(rows, hq, ctx):
    """All loads of a block fit its ring, so the loading warp itself never waits: whichever role gives up, if one does,
    the call reports it, and the next call on the same workspace is right."""
    c = Cache([rows] * 3, [ctx] * 3, 1, 64, 32, seed=40)
    q = torch.randn(3 * rows, hq, 64, generator=torch.Generator().manual_seed(41)).to(torch.bfloat16).cuda()
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    ws = B.alloc_attention_workspace(hq, 1, 64)

    def call(o):
        B.dspark_window_attention(q, c.k, c.v, c.table, c.cu, c.ctx, rows, 0.125, 0, 0, o, None, ws)
        return B.dspark_read_device_status(ws)

    assert call(want) == B.DSPARK_OK
    for _ in range(20):
        old = B.dspark_set_wait_timeout_ns(1)
        try:
            st = call(out)
        finally:
            B.dspark_set_wait_timeout_ns(old)
        assert st == B.DSPARK_ETIMEOUT or (st == B.DSPARK_OK and torch.equal(out, want))
        assert call(out) == B.DSPARK_OK and torch.equal(out, want)


def _at_16(t):
    """A copy of t that begins 16 bytes after a multiple of 32."""
    room = torch.empty(t.numel() + 32 // t.element_size(), dtype=t.dtype, device="cuda")
    skip = (16 - room.data_ptr() % 32) % 32 // t.element_size()
    out = room[skip:skip + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 32 == 16 and out.is_contiguous()
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 8, 40, 150])
def test_tensors_that_begin_at_16_bytes(rows, d):
    """Every tensor begins at an odd multiple of 16 bytes, at each tiling, whole units and cut ones."""
    ns, ctxs = [rows, max(1, rows - 3)] * 3, [300, 20, 1000, 0, 64, 5]
    c = Cache(ns, ctxs, 2, d, 16, seed=42)
    q = torch.randn(sum(ns), 8, d, generator=torch.Generator().manual_seed(43)).to(torch.bfloat16).cuda()
    ws = B.alloc_attention_workspace(8, 2, d)
    got = []
    for at in (lambda t: t, _at_16):
        out = at(torch.full_like(q, 7.0))
        lse = at(torch.zeros(sum(ns), 8, device="cuda"))
        B.dspark_window_attention(at(q), at(c.k), at(c.v), at(c.table), at(c.cu), at(c.ctx), rows, d ** -0.5, 100, 2, out, lse, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        got.append((out.clone(), lse.clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_append_and_rules_on_tensors_that_begin_at_16_bytes():
    ns, ctxs = [3, 1, 20], [40, 0, 7]
    c = Cache(ns, ctxs, 2, 64, 16, seed=44, fill=0.0)
    g = torch.Generator().manual_seed(45)
    q, k, v = (torch.randn(sum(ns), h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    ang = torch.arange(64)[:, None] * 10000.0 ** (-torch.arange(32) / 32)
    cs = torch.cat([ang.cos(), ang.sin()], 1).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = []
    for at in (lambda t: t, _at_16):
        qo, kc, vc = at(torch.zeros_like(q)), at(c.k), at(c.v)
        B.dspark_append_kv(at(q), at(k), at(v), at(c.cu), at(c.ctx), at(cs), at(c.table), qo, kc, vc, ws)
        got.append((qo, kc.clone(), vc.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    V, bs = 4104, 3
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(sum(ns), V, generator=g).to(dtype).cuda()
        hist = torch.zeros(bs, V, dtype=torch.int16, device="cuda")
        ids = torch.arange(sum(ns), dtype=torch.int32, device="cuda")
        toks = torch.arange(0, 900, 7, dtype=torch.int32, device="cuda")
        start = torch.tensor([0, 50, 60, len(toks)], dtype=torch.int32, device="cuda")
        asked = torch.tensor([10, 0, 30], dtype=torch.int32, device="cuda")
        mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (sum(ns), (V + 31) // 32), generator=g).int().cuda()
        some = torch.tensor([1.3, 0.7, 1.1], device="cuda")
        bias = (torch.tensor([0, 2, 2, 3], dtype=torch.int32, device="cuda"), torch.tensor([5, 900, 11], dtype=torch.int32, device="cuda"),
                torch.tensor([1.0, -2.0, 3.0], device="cuda"))
        got = []
        for at in (lambda t: t, _at_16):
            h, out = at(hist), at(torch.zeros_like(x))
            B.dspark_history_build(at(toks), at(start), at(asked), h, ws)
            B.dspark_process_logits(at(x), at(c.cu), at(ids), h, at(some), at(some), at(some), *(at(t) for t in bias), at(mask), out, ws)
            out_tokens = at(torch.tensor([[1, 2], [3, -1], [-1, -1]], dtype=torch.int32, device="cuda"))
            B.dspark_history_commit(out_tokens, h, ws)
            got.append((h.clone(), out.clone()))
        assert all(torch.equal(a, b) for a, b in zip(*got))
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK


@pytest.mark.parametrize("ctx0", [40, 2, 0])
def test_lists_that_start_behind_row_0(ctx0):
    """The last requests of a batch, with the whole batch's rows: what lies before their windows belongs to nobody (and no
    length makes it a cached position)."""
    ns, ctxs, skip = [5, 2, 3, 1], [9, 30, ctx0, 17], 2
    whole = Cache(ns, ctxs, 2, 64, 16, seed=46, fill=0.0)
    rows, first = sum(ns) + 2, sum(ns[:skip])
    g = torch.Generator().manual_seed(47)
    q, k, v = (torch.randn(rows, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    ang = torch.arange(64)[:, None] * 10000.0 ** (-torch.arange(32) / 32)
    cs = torch.cat([ang.cos(), ang.sin()], 1).cuda()
    ws = B.alloc_attention_workspace(4, 2, 64)
    kc, vc, qo = whole.k.clone(), whole.v.clone(), torch.full_like(q, 7.0)
    B.dspark_append_kv(q, k, v, whole.cu, whole.ctx, cs, whole.table, qo, kc, vc, ws)
    out = torch.full_like(q, 7.0)
    B.dspark_window_attention(qo, kc, vc, whole.table, whole.cu, whole.ctx, 5, 0.125, 20, 2, out, None, ws)
    cu, ctx, table = whole.cu[skip:], whole.ctx[skip:], whole.table[skip:]
    k2, v2, q2 = whole.k.clone(), whole.v.clone(), torch.full_like(q, 7.0)
    B.dspark_append_kv(q, k, v, cu, ctx, cs, table, q2, k2, v2, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    assert (q2[:first] == 7.0).all() and torch.equal(q2[first:], qo[first:])
    for r, (n, x) in enumerate(zip(ns, ctxs)):  # the other requests' slots are as they were
        pos = torch.arange(x, x + n, device="cuda")
        pages = whole.table[r][pos // 16].long()
        for got, full, before in ((k2, kc, whole.k), (v2, vc, whole.v)):
            want = full if r >= skip else before
            assert torch.equal(got[pages, :, pos % 16], want[pages, :, pos % 16])
            got[pages, :, pos % 16] = full[pages, :, pos % 16]
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
    for max_rows in (5, 100):
        o2 = torch.full_like(q, 7.0)
        B.dspark_window_attention(qo, kc, vc, table, cu, ctx, max_rows, 0.125, 20, 2, o2, None, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        assert (o2[:first] == 7.0).all() and (o2[sum(ns):] == 7.0).all()
        if max_rows == 5:
            assert torch.equal(o2[first:], out[first:])
    V = 2056
    x = torch.randn(rows, V, generator=g).to(torch.bfloat16).cuda()
    ids = torch.randint(0, 40, (rows,), generator=g).int().cuda()
    hist = torch.zeros(len(ns), V, dtype=torch.int16, device="cuda")
    some = torch.full((len(ns),), 1.5, device="cuda")
    a, b = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    B.dspark_process_logits(x, whole.cu, ids, hist, some, some, some, None, None, None, None, a, ws)
    B.dspark_process_logits(x, cu, ids, hist[skip:], some[skip:], some[skip:], some[skip:], None, None, None, None, b, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    assert (b[:first] == 7.0).all() and torch.equal(b[first:], a[first:])


@pytest.mark.parametrize("max_rows", [1, 5, 1 << 20])
def test_more_tiles_than_are_counted(max_rows):
    """A window of 2^20 rows over 2^29 positions is more work than a call takes, at every tiling: it is refused as a
    whole, also where the count passes 2^32."""
    n, ctx, page = 1 << 20, 1 << 29, 4096
    k = torch.zeros(1, 1, page, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, (ctx + n) // page + 1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = B.alloc_attention_workspace(1, 1, 64)
    B.dspark_window_attention(q, k, k, table, torch.tensor([0, n], **i32), torch.tensor([ctx], **i32), max_rows, 0.125, 0, 0,
                              out, None, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_EINVAL and (out == 7.0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,ctx", [(1, 2, 40), (1, 2, 9000), (8, 4, 9000), (16, 16, 6000), (150, 4, 5000)])
def test_scores_that_are_no_numbers(n, hq, ctx, d):
    """A key that holds NaN makes the rows that see it NaN, output and log-sum-exp, also where the tile that it lies in is
    one part of a unit that is cut; a score of -inf is a weight of 0, one of +inf no number (inf - inf).  The other KV
    head is untouched."""
    page = 32
    c = Cache([n], [ctx], 2, d, page, seed=48)
    table = c.table.cpu().numpy()
    q = torch.randn(n, hq, d, generator=torch.Generator().manual_seed(49)).to(torch.bfloat16)
    q[..., 0] = torch.where(torch.arange(hq) % 2 == 0, 1.0, -1.0).to(torch.bfloat16)  # the sign of an infinite lane's score
    ws = B.alloc_attention_workspace(hq, 2, d)
    g = hq // 2
    for value in (float("nan"), float("inf")):
        for at in (3, ctx // 2, ctx):
            keys = [c.keys[0].copy()]
            keys[0][at, 0, 0] = value
            k = c.k.clone()
            k[table[0, at // page], 0, at % page, 0] = value
            out = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros(n, hq, device="cuda")
            B.dspark_window_attention(q.cuda(), k, c.v, c.table, c.cu, c.ctx, n, d ** -0.5, 0, 0, out, lse, ws)
            assert B.dspark_read_device_status(ws) == B.DSPARK_OK
            with np.errstate(invalid="ignore"):
                ref, rl, mag = R.attention(_f64(q), keys[0], c.vals[0], ctx, d ** -0.5, 0, 0)
            got, got_lse = _f64(out), _f64(lse)
            no_number = np.isnan(ref)
            assert no_number[:, :g].any() and not no_number[:, g:].any()
            assert np.array_equal(np.isnan(got), no_number) and np.array_equal(np.isnan(got_lse), no_number.any(2))
            assert (np.abs(got - ref)[~no_number] <= R.attention_bound(mag)[~no_number]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,ctx", [(1, 2, 40), (1, 2, 9000), (16, 4, 3000), (150, 2, 3000)])
def test_rows_whose_scores_are_all_minus_infinity(n, hq, ctx, d):
    """Every key of a KV head has an infinite lane: heads whose query has the other sign there are 0 with lse -inf."""
    c = Cache([n], [ctx], 2, d, 32, seed=50)
    k = torch.nan_to_num(c.k, nan=0.0)
    k[:, 0, :, 0] = float("inf")
    q = torch.randn(n, hq, d, generator=torch.Generator().manual_seed(51)).to(torch.bfloat16).cuda()
    q[..., 0] = -1.0
    out, lse = torch.full_like(q, 7.0), torch.zeros(n, hq, device="cuda")
    ws = B.alloc_attention_workspace(hq, 2, d)
    B.dspark_window_attention(q, k, c.v, c.table, c.cu, c.ctx, n, d ** -0.5, 0, 0, out, lse, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    g = hq // 2
    assert (out[:, :g] == 0).all() and torch.isneginf(lse[:, :g]).all()
    assert torch.isfinite(out[:, g:]).all() and torch.isfinite(lse[:, g:]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name,ns,ctxs,hq,max_rows", [
    ("one", [1], [2500], 4, 1), ("windows", [1, 8, 3, 0, 5] * 30, [300, 17, 900, 90, 128] * 30, 8, 8),
    ("wide windows", [16, 9] * 20, [3000, 130] * 20, 8, 16), ("longer than expected", [20, 3, 40], [700, 9, 2000], 8, 2),
    ("prompts", [150, 33, 260], [700, 0, 2000], 8, 260), ("one prompt", [70], [9000], 4, 70)])
def test_output_in_place_of_the_queries(name, ns, ctxs, hq, max_rows, d):
    """`out` may be `q`: the same bits as with an output of its own, whole units and cut ones, at each tiling."""
    c = Cache(ns, ctxs, 2, d, 32, seed=52)
    q = torch.randn(sum(ns) + 2, hq, d, generator=torch.Generator().manual_seed(53)).to(torch.bfloat16).cuda()
    ws = B.alloc_attention_workspace(hq, 2, d)
    for window, sinks in ((0, 0), (200, 4)):
        out, both = torch.empty_like(q), q.clone()
        out[sum(ns):] = q[sum(ns):]
        lse = [torch.zeros(sum(ns) + 2, hq, device="cuda") for _ in range(2)]
        for x, o, l in ((q, out, lse[0]), (both, both, lse[1])):
            B.dspark_window_attention(x, c.k, c.v, c.table, c.cu, c.ctx, max_rows, d ** -0.5, window, sinks, o, l, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        assert torch.equal(both, out) and torch.equal(lse[0], lse[1])


@pytest.mark.parametrize("n,hq", [(1, 2), (8, 4), (16, 8), (90, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_large_values_under_scores_that_grow(n, hq, d):
    """Values of 2^75 and weights that outgrow those of the first tile by 2^57: finite outputs stay finite.  q = 1, key j =
    c_j in every lane, scale 1 / D: the scores are c_j."""
    page, ctx = 32, 700
    c = Cache([n], [ctx], 1, d, page, seed=55)
    level = np.where(np.arange(ctx + n) < 200, 0.0, 40.0) + (np.arange(ctx + n) % 4) * 0.25
    level[-1] = 0.0
    c.keys[0] = np.repeat(level[:, None, None], d, 2)
    c.vals[0] = c.vals[0] * 2.0 ** 75
    table = c.table.cpu().numpy()
    for j in range(ctx + n):
        c.k[table[0, j // page], :, j % page] = float(level[j])
    c.v = c.v * 2.0 ** 75
    bs = 160  # enough work that a block takes whole units, too
    q = torch.ones(bs * n, hq, d, dtype=torch.bfloat16, device="cuda")
    ws = B.alloc_attention_workspace(hq, 1, d)
    ref, rl, mag = R.attention(_f64(q)[:n], c.keys[0], c.vals[0], ctx, 1.0 / d, 0, 0)
    for many in (1, bs):
        out, lse = torch.zeros_like(q[:many * n]), torch.zeros(many * n, hq, device="cuda")
        cu = torch.arange(0, many * n + 1, n, dtype=torch.int32, device="cuda")
        B.dspark_window_attention(q[:many * n], c.k, c.v, c.table.repeat(many, 1), cu, c.ctx.repeat(many), n, 1.0 / d, 0, 0, out,
                                  lse, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        assert (np.abs(_f64(out).reshape(many, n, hq, d) - ref) <= R.attention_bound(mag)).all()
        assert np.abs(_f64(lse).reshape(many, n, hq) - rl).max() <= 1e-4 * (1 + np.abs(rl).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [49, 64, 65, 100, 127, 128])
@pytest.mark.parametrize("ns,ctxs", [([1, 2], [130, 3000]), ([5, 0, 40], [64, 9, 300])])
def test_many_query_heads_to_a_kv_head(g, d, ns, ctxs):
    """Groups of up to 128 query heads, the most that is allowed, at each tiling that takes them."""
    for window, sinks in ((0, 0), (100, 3)):
        c = Cache(ns, ctxs, 1, d, 16, seed=g, evict=(window, sinks) if window else None)
        for max_rows in (1, max(ns)):
            _check_attention(c, g, window, sinks, seed=56, max_rows=max_rows)
