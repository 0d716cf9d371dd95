"""The 8-bit cache's calls where memory, masks and waits can go wrong: waits that run out, tensors at the least alignment, pages
that two requests share, many query heads, lists of windows that begin behind row 0, the guards around what is written."""
import numpy as np
import pytest

from tests import kv8_reference as K
from tests import serving_reference as R

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from tests.test_gpu_attention import _f64, _status_ws, _table  # noqa: E402
from tests.test_gpu_attention_edges import _at_16  # noqa: E402
from tests.test_gpu_kv8 import F8, Cache8, _check, _codes  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,hq,ctx,many", [(1, 2, 10, 1), (8, 4, 200, 1), (16, 8, 300, 1), (60, 4, 200, 1), (1, 4, 1500, 60),
                                             (8, 4, 1500, 60), (16, 8, 1500, 60), (16, 4, 1500, 60)])
def test_waits_that_run_out_are_reported_and_recover(rows, hq, ctx, many):
    """With a deadline of 1 ns the kernel's waits run out, over little work and over much: it reports it, drains its copies and
    MMAs and returns; the next call with the normal deadline is right again, on the same workspace."""
    c = Cache8([rows] * 4, [ctx] * 4, 2, 64, 32, seed=40)
    table, lens = c.table.repeat(many, 1), c.ctx.repeat(many)
    cu = torch.arange(0, 4 * many * rows + 1, rows, dtype=torch.int32, device="cuda")
    q = torch.randn(4 * many * rows, 2 * hq, 64, generator=torch.Generator().manual_seed(41)).to(torch.bfloat16).cuda()
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    ws = B.alloc_attention_workspace(2 * hq, 2, 64)

    def call(o):
        B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, table, cu, lens, rows, 0.125, 0, 0, o, None, None, None, ws)
        return B.dspark_read_device_status(ws)

    assert call(want) == B.DSPARK_OK
    for _ in range(5):
        old = B.dspark_set_wait_timeout_ns(1)
        try:
            st = call(out)
        finally:
            B.dspark_set_wait_timeout_ns(old)
        assert st == B.DSPARK_ETIMEOUT or (st == B.DSPARK_OK and many == 1 and torch.equal(out, want))
        assert call(out) == B.DSPARK_OK and torch.equal(out, want)


@pytest.mark.parametrize("max_rows", [9, 200])
def test_least_alignment(max_rows):
    """Every tensor begins 16 bytes after a multiple of 32."""
    c = Cache8([3, 9], [100, 39], 2, 64, 16, seed=42)
    out, lse = _check(c, 8, 0, 0, seed=43, pad=0, max_rows=max_rows, scratch=True)
    q = torch.randn(12, 8, 64, generator=torch.Generator().manual_seed(44)).to(torch.bfloat16)
    c.k, c.v = (_at_16(t.view(torch.uint8)).view(F8) for t in (c.k, c.v))
    c.scale = _at_16(c.scale)
    got = _at_16(torch.zeros_like(out))
    ws = B.alloc_attention_workspace(8, 2, 64)
    B.dspark_window_attention_kv8(_at_16(q.cuda()), c.k, c.v, c.scale, c.table, c.cu, c.ctx, max_rows, 0.125, 0, 0, got, None,
                                  *[_at_16(t) for t in c.scratch()], ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    assert torch.equal(got, out)


@pytest.mark.parametrize("hq,hkv,d", [(49, 1, 64), (64, 1, 64), (65, 1, 64), (128, 1, 64), (100, 1, 128), (256, 2, 128)])
@pytest.mark.parametrize("scratch", [False, True])
def test_many_query_heads_to_a_kv_head(hq, hkv, d, scratch):
    c = Cache8([1, 3, 2], [200, 0, 131], hkv, d, 32, seed=45, evict=(90, 2))
    _check(c, hq, 90, 2, seed=46, scratch=scratch)


def test_units_that_are_not_full():
    """Windows of every length below the tile's: rows behind a unit's weigh nothing and set no reference."""
    ns = [1, 2, 3, 5, 7, 8, 4, 6] * 6
    c = Cache8(ns, [(97 * i) % 900 for i in range(len(ns))], 2, 64, 32, seed=47, evict=(300, 4), spread=8)
    _check(c, 16, 300, 4, seed=48)
    c = Cache8(ns, [(97 * i) % 900 for i in range(len(ns))], 2, 128, 64, seed=47, spread=8)
    _check(c, 8, 0, 0, seed=48)


def test_pages_that_two_requests_share():
    """A common prefix in pages of both: attention, and reading back to the same pages and to pages of their own."""
    c = Cache8([4, 4], [100, 100], 2, 64, 16, seed=49)
    c.table[1, :5] = c.table[0, :5]  # positions 0 .. 79
    for kept in (c.keys, c.vals):
        kept[1][:80] = kept[0][:80]
    _check(c, 4, 0, 0, seed=50)
    _check(c, 4, 0, 0, seed=50, max_rows=200, scratch=True)
    outs = [torch.zeros(c.k.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = _status_ws()
    B.dspark_read_kv8(c.k, c.v, c.scale, c.table, c.cu, c.ctx, 8, 0, 0, c.table, *outs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    pos = np.arange(104)
    for r in range(2):
        pages = c.table[r].cpu().numpy()[pos // 16]
        for o, kept in zip(outs, (c.keys, c.vals)):
            assert np.array_equal(_f64(o)[pages, :, pos % 16], kept[r])


def test_lists_that_begin_behind_row_0():
    c = Cache8([2, 3], [70, 10], 1, 64, 16, seed=51)
    rows, hq = 9, 2
    q = torch.randn(rows, hq, 64, generator=torch.Generator().manual_seed(52)).to(torch.bfloat16).cuda()
    kv = torch.randn(rows, 1, 64, generator=torch.Generator().manual_seed(53)).to(torch.bfloat16).cuda()
    cu = c.cu + 3
    for max_rows, scratch in ((3, (None, None)), (300, c.scratch())):
        out = torch.full((rows, hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = B.alloc_attention_workspace(hq, 1, 64)
        B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, cu, c.ctx, max_rows, 0.125, 0, 0, out, None, *scratch, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        assert (out[:3] == 7.0).all() and (out[8:] == 7.0).all()
        for r, (a, b) in enumerate(((3, 5), (5, 8))):
            ref, _, mag = R.attention(_f64(q)[a:b], c.keys[r], c.vals[r], c.ctxs[r], 0.125, 0, 0)
            assert (np.abs(_f64(out)[a:b] - ref) <= R.attention_bound(mag)).all()
    before = [t.view(torch.uint8).clone() for t in (c.k, c.v, c.scale)]
    q_out = torch.full_like(q, 7.0)
    B.dspark_append_kv8(q, kv, kv, cu, c.ctx, torch.from_numpy(_table(100, 64)).cuda(), c.table, q_out, c.k, c.v, c.scale, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    assert (q_out[:3] == 7.0).all() and (q_out[8:] == 7.0).all() and not (q_out[3:8] == 7.0).any()
    touched = (c.scale.view(torch.uint8) != before[2]).any(-1).sum().item()
    assert touched <= 5
    byte = K.exponent_byte(_f64(kv)[3:8])
    got = c.scale[c.table[0, 70 // 16], 0, 70 % 16, 1].item()
    assert got == byte[0, 0]


def test_guards_around_what_is_written():
    """Every output inside a larger allocation: nothing is written beside it."""
    c = Cache8([3, 5], [40, 131], 2, 64, 8, seed=54)

    def guarded(shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        room = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        return room, room[256:256 + n].view(dtype).view(shape)

    rooms = {}
    for name in ("k", "v", "scale"):
        t = getattr(c, name)
        rooms[name], new = guarded(t.shape, t.dtype)
        new.view(torch.uint8).copy_(t.view(torch.uint8))
        setattr(c, name, new)
    rows, hq = 8, 6
    g = torch.Generator().manual_seed(55)
    q = torch.randn(rows, hq, 64, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(rows, 2, 64, generator=g).to(torch.bfloat16).cuda()
    for name, shape, dtype in (("q_out", q.shape, q.dtype), ("out", q.shape, q.dtype), ("lse", (rows, hq), torch.float32),
                               ("k_wide", c.k.shape, torch.bfloat16), ("v_wide", c.k.shape, torch.bfloat16)):
        rooms[name] = guarded(shape, dtype)
    n_ws = B.dspark_window_attention_workspace_bytes(hq, 2, 64)
    rooms["ws"] = guarded((n_ws,), torch.uint8)
    rooms["ws"][1].zero_()
    at = {k: v[1] for k, v in rooms.items() if isinstance(v, tuple)}
    cs = torch.from_numpy(_table(200, 64)).cuda()
    B.dspark_append_kv8(q, kv, kv, c.cu, c.ctx, cs, c.table, at["q_out"], c.k, c.v, c.scale, at["ws"])
    for max_rows in (1, 5, 40, 500):
        B.dspark_window_attention_kv8(at["q_out"], c.k, c.v, c.scale, c.table, c.cu, c.ctx, max_rows, 0.125, 60, 3, at["out"],
                                      at["lse"], at["k_wide"], at["v_wide"], at["ws"])
    B.dspark_read_kv8(c.k, c.v, c.scale, c.table, c.cu, c.ctx, rows, 60, 3, c.table, at["k_wide"], at["v_wide"], at["ws"])
    assert B.dspark_read_device_status(at["ws"]) == B.DSPARK_OK
    torch.cuda.synchronize()
    for name, v in rooms.items():
        room = v[0] if isinstance(v, tuple) else v
        assert (room[:256] == 0x5A).all() and (room[-256:] == 0x5A).all(), name
    x = torch.randn(5, 5000, device="cuda")
    for top in (0, 1, 32):
        n_ws = B.dspark_token_logprobs_workspace_bytes(5, 5000, top)
        made = [guarded((n_ws,), torch.uint8), guarded((5, 1), torch.float32), guarded((5, 1), torch.float32),
                guarded((5, 1), torch.int32)] + ([guarded((5, 1, top), torch.int32), guarded((5, 1, top), torch.float32)] if top else [])
        made[0][1].zero_()
        o = [m[1] for m in made]
        tokens = torch.tensor([[1], [-1], [4999], [0], [17]], dtype=torch.int32, device="cuda")
        B.dspark_token_logprobs(x, None, tokens, 0.7, o[1], o[2], o[3], *(o[4:] or (None, None)), o[0])
        torch.cuda.synchronize()
        for room, _ in made:
            assert (room[:256] == 0x5A).all() and (room[-256:] == 0x5A).all()


def test_two_streams_at_once():
    """Two calls that can overlap, each with a workspace and pages of its own."""
    c = Cache8([8] * 30, [700] * 30, 2, 128, 64, seed=56)
    q = torch.randn(240, 8, 128, generator=torch.Generator().manual_seed(57)).to(torch.bfloat16).cuda()
    want = torch.zeros_like(q)
    made = [(torch.cuda.Stream(), B.alloc_attention_workspace(8, 2, 128), c.scratch(), torch.zeros_like(q)) for _ in range(2)]

    def call(ws, scratch, out, max_rows, stream=None):
        B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, c.cu, c.ctx, max_rows, 0.1, 0, 0, out, None, *scratch, ws, stream)

    for max_rows in (8, 200):
        call(made[0][1], made[0][2], want, max_rows)
        torch.cuda.synchronize()
        for _ in range(10):
            for s, ws, scratch, out in made:
                call(ws, scratch, out, max_rows, s)
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, _, _, out in made)


@pytest.mark.parametrize("which", [0, 1])
def test_vectors_of_nan_among_pages_read_back(which):
    """By way of bf16 pages, too, a vector of NaN reaches the rows that see it and no other row, log-sum-exps included."""
    c = Cache8([4, 4], [150, 150], 1, 64, 16, seed=30)
    c.scale[c.table[0, 151 // 16], 0, 151 % 16, which] = 255  # row 1's own position
    ws, q = B.alloc_attention_workspace(2, 1, 64), torch.randn(11, 2, 64, generator=torch.Generator().manual_seed(32))
    for max_rows, scratch in ((4, (None, None)), (200, c.scratch())):
        out = torch.zeros(11, 2, 64, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(11, 2, device="cuda")
        B.dspark_window_attention_kv8(q.to(torch.bfloat16).cuda(), c.k, c.v, c.scale, c.table, c.cu, c.ctx, max_rows, 0.125, 0,
                                      0, out, lse, *scratch, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        for got in (out, lse):
            assert torch.isnan(got[1:4]).all() and not torch.isnan(got[0]).any() and not torch.isnan(got[4:]).any()


def test_values_that_fall_by_powers_of_two():
    """V's powers of two fall by 40 from tile to tile while one head's scores grow, so that the tiles' references are set anew
    each time: another head, whose scores do not change, keeps its output of the first tile's size."""
    d, page, n, ctx, bs = 64, 32, 1, 1023, 250
    c = Cache8([n], [ctx], 1, d, page, seed=60, spread=0)
    pos = np.arange(ctx + n)
    tile = pos // 128
    up = np.array([0, -40, -80, -110, -110, -110, -110, -110])[tile]
    c.keys[0] = np.repeat((8.0 * tile)[:, None, None], d, 2)
    c.vals[0] = c.vals[0] * 2.0 ** up[:, None, None]
    byte = K.exponent_byte(c.keys[0])
    table = c.table.cpu().numpy()[0]
    k, s = _codes(c.k).copy(), c.scale.cpu().numpy().copy()
    k[table[pos // page], :, pos % page] = K.codes(c.keys[0], byte)
    s[table[pos // page], :, pos % page, 0] = byte
    s[table[pos // page], :, pos % page, 1] += up[:, None].astype(np.uint8)
    c.k, c.scale = torch.from_numpy(k).cuda().view(F8), torch.from_numpy(s).cuda()
    q = torch.ones(bs * n, 2, d, dtype=torch.bfloat16, device="cuda")
    q[:, 1] = 0.0
    cu = torch.arange(0, bs * n + 1, n, dtype=torch.int32, device="cuda")
    ws, out = B.alloc_attention_workspace(2, 1, d), torch.zeros_like(q)
    B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table.repeat(bs, 1), cu, c.ctx.repeat(bs), n, 1.0 / d, 0, 0, out,
                                  None, None, None, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    ref, _, mag = R.attention(_f64(q)[:n], c.keys[0], c.vals[0], ctx, 1.0 / d, 0, 0)
    assert (np.abs(_f64(out).reshape(bs, n, 2, d) - ref) <= R.attention_bound(mag)).all()


@pytest.mark.parametrize("list_", [[2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, 4], [5, -2 ** 31 + 8], [2, 2 ** 31 - 1], [-2 ** 31, 1]])
def test_lists_at_the_ends_of_32_bits(list_):
    """A list of windows whose differences pass 32 bits is refused by each call, and nothing is written."""
    c = Cache8([4], [20], 1, 64, 16, seed=61)
    cu = torch.tensor(list_, dtype=torch.int32, device="cuda")
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    wide = c.scratch()
    ws = B.alloc_attention_workspace(2, 1, 64)

    def refused(call):
        out = torch.full_like(q, 7.0)
        call(out)
        assert B.dspark_read_device_status(ws) == B.DSPARK_EINVAL and (out == 7.0).all()

    refused(lambda out: B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, cu, c.ctx, 4, 0.125, 0, 0, out, None, None,
                                                      None, ws))
    refused(lambda out: B.dspark_window_attention_kv8(q, c.k, c.v, c.scale, c.table, cu, c.ctx, 400, 0.125, 0, 0, out, None,
                                                      *wide, ws))
    refused(lambda out: B.dspark_window_attention(q, *wide, c.table, cu, c.ctx, 4, 0.125, 0, 0, out, None, ws))
    refused(lambda out: B.dspark_window_attention(q, *wide, c.table, cu, c.ctx, 400, 0.125, 0, 0, out, None, ws))
    refused(lambda out: B.dspark_read_kv8(c.k, c.v, c.scale, c.table, cu, c.ctx, 4, 0, 0, c.table, *wide, ws))
    assert all(torch.isnan(w).all() for w in wide)
    refused(lambda out: B.dspark_append_kv8(q, q[:, :1], q[:, 1:], cu, c.ctx, torch.from_numpy(_table(100, 64)).cuda(), c.table,
                                            out, c.k, c.v, c.scale, ws))
