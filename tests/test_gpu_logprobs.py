"""Log probabilities of tokens on the GPU against a plain 64-bit form.

Bounds.  x = l / temperature, x - max x (two roundings, 2^-24 of |l| / temperature each, which counts in absolute terms), exp
(2 ulp) and sums of V terms kept in partial sums of at most some hundred: the log-sum-exp is off by less than 1e-5 + 1e-6 max|x|,
an entropy by that times the entropy's own size and more for its products."""
import numpy as np
import pytest

from tests import kv8_reference as K

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _outputs(n, per, top, fill=5):
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    return [torch.full((n, per), fill, **f32), torch.full((n, per), fill, **f32), torch.full((n, per), fill, **i32),
            torch.full((n, per, top), fill, **i32) if top else None, torch.full((n, per, top), fill, **f32) if top else None]


def _check(logits, cu, tokens, temperature, top, ws=None):
    """cu: a host list or None.  Returns what the call wrote."""
    tokens = np.asarray(tokens, np.int32)
    n, per = tokens.shape
    outs = _outputs(n, per, top)
    ws = B.alloc_logprobs_workspace(n * per, logits.shape[1], top) if ws is None else ws
    d_cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    for _ in range(2):  # the second call runs on a workspace that has been used
        B.dspark_token_logprobs(logits, d_cu, torch.from_numpy(tokens).cuda(), temperature, *outs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    x = _f64(logits)
    lp, ent, rank, ids, best = (None if o is None else o.cpu().numpy() for o in outs)
    for r in range(n):
        for j in range(per):
            t = tokens[r, j]
            if t < 0:
                assert lp[r, j] == 0 and ent[r, j] == 0 and rank[r, j] == 0
                if top:
                    assert (ids[r, j] == -1).all() and (best[r, j] == -np.inf).all()
                continue
            row = x[(r * per if cu is None else cu[r]) + j]
            wlp, went, wrank, wids, wbest = K.token_logprobs(row, t, temperature, top)
            live = row[np.isfinite(row)]
            tol = 1e-5 + 1e-6 * (np.abs(live).max() if live.size else 0.0) / temperature
            np.testing.assert_allclose(lp[r, j], wlp, rtol=2e-6, atol=tol)
            np.testing.assert_allclose(ent[r, j], went, rtol=1e-5, atol=2 * tol)
            assert rank[r, j] == wrank, (r, j)
            if top:
                assert np.array_equal(ids[r, j], wids), (r, j, ids[r, j], wids)
                np.testing.assert_allclose(best[r, j], wbest, rtol=2e-6, atol=tol)
    return outs


def _logits(rows, V, dtype, seed, std=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(rows, V, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,n,per,top", [
    (8, 1, 1, 5), (8, 3, 2, 32), (64, 2, 3, 0), (1000, 4, 1, 1), (4096, 5, 3, 20), (5000, 70, 2, 7), (32000, 1, 1, 5),
    (32008, 40, 4, 20), (129280, 2, 3, 32), (151936, 1, 1, 20), (151936, 300, 1, 3), (50264, 150, 6, 8)])
def test_rows(dtype, V, n, per, top):
    rng = np.random.default_rng(V + n)
    tokens = rng.integers(0, V, (n, per))
    tokens[rng.random((n, per)) < 0.2] = -1
    _check(_logits(n * per, V, dtype, V), None, tokens, 1.0, top)


@pytest.mark.parametrize("temperature", [0.1, 0.7, 3.0])
def test_windows_and_temperatures(temperature):
    """Tokens of packed windows as a verification leaves them: -1 behind the committed ones, a list that begins behind row 0."""
    rng = np.random.default_rng(1)
    ns = [3, 1, 0, 8, 5]
    cu = np.concatenate([[2], 2 + np.cumsum(ns)]).tolist()
    tokens = np.full((5, 8), -1)
    for r, m in enumerate(ns):
        tokens[r, :rng.integers(0, m + 1)] = 7
        tokens[r] = np.where(tokens[r] < 0, -1, rng.integers(0, 3000, 8))
    for dtype in (torch.bfloat16, torch.float32):
        _check(_logits(cu[-1] + 4, 3000, dtype, 2), cu, tokens, temperature, 6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_id(dtype):
    """Rows of one value, of two, of steps with many equal ids each, ascending and descending: whole vocabularies of ties."""
    V = 40000
    v = torch.arange(V, device="cuda")
    rows = [torch.zeros(V, device="cuda"), (v % 2).float(), (v // 1000).float(), -(v // 3).float() / 64, (v % 17).float(),
            torch.where(v == V - 1, 1.0, -0.0), torch.where(v % 2 == 0, 0.0, -0.0), (v >= V - 5).float(), -v.float(), v.float()]
    logits = torch.stack(rows).to(dtype)
    tokens = [[(7919 * (i + 1)) % V] for i in range(len(rows))]
    _check(logits, None, tokens, 1.0, 32)
    _check(logits, None, tokens, 1.0, 5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_rows(dtype):
    """Rows of which a mask leaves all but one id, a few, one, and none."""
    V, top = 30000, 20
    x = _logits(5, V, dtype, 5)
    g = np.random.default_rng(6)
    kept = [V - 1, 300, 7, 1, 0]
    tokens = []
    for r, m in enumerate(kept):
        live = np.sort(g.permutation(V)[:m])
        gone = torch.ones(V, dtype=torch.bool, device="cuda")
        gone[torch.from_numpy(live).cuda()] = False
        x[r, gone] = float("-inf")
        tokens.append([int(live[m // 2]) if m else 11])
    _check(x, None, tokens, 1.0, top)
    # a token that the mask forbids
    _check(x[1:4].contiguous(), None, [[int((x[r] == float("-inf")).nonzero()[0])] for r in (1, 2, 3)], 1.0, top)


def test_masks_of_the_lowest_value():
    """Ids masked by the type's lowest value weigh nothing, unless there is nothing else: then all are equal."""
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(3, 9000, dtype, 12)
        x[0, 100:8000] = torch.finfo(dtype).min
        x[1] = torch.finfo(dtype).min
        x[2, 1:] = torch.finfo(dtype).min
        outs = _outputs(3, 1, 3)
        ws = B.alloc_logprobs_workspace(3, 9000, 3)
        B.dspark_token_logprobs(x, None, torch.tensor([[50], [77], [0]], dtype=torch.int32, device="cuda"), 1.0, *outs, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_OK
        lp, ent, rank, ids, best = (o.cpu().numpy() for o in outs)
        want = K.token_logprobs(_f64(x)[0], 50, 1.0, 3)
        np.testing.assert_allclose([lp[0, 0], ent[0, 0]], want[:2], atol=3e-5)
        assert rank[0, 0] == want[2] and np.array_equal(ids[0, 0], want[3])
        np.testing.assert_allclose([lp[1, 0], ent[1, 0]], [-np.log(9000), np.log(9000)], atol=3e-5)
        assert rank[1, 0] == 78 and ids[1, 0].tolist() == [0, 1, 2] and ids[2, 0].tolist() == [0, 1, 2]
        assert lp[2, 0] == 0 and abs(ent[2, 0]) < 1e-6 and rank[2, 0] == 1


def test_rows_with_nan_and_infinity():
    """NaN wherever it stands in the row, and +inf: NaN results; alternatives and ranks are those of the numbers."""
    V = 20000
    x = _logits(4, V, torch.float32, 7)
    x[0, 3], x[1, V - 1], x[2, 12000], x[3, :] = float("nan"), float("nan"), float("inf"), float("nan")
    outs = _outputs(4, 1, 3)
    ws = B.alloc_logprobs_workspace(4, V, 3)
    tokens = torch.tensor([[5], [6], [7], [8]], dtype=torch.int32, device="cuda")
    B.dspark_token_logprobs(x, None, tokens, 1.0, *outs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    lp, ent, rank, ids, best = (o.cpu().numpy() for o in outs)
    assert np.isnan(lp).all() and np.isnan(ent).all() and np.isnan(best[:3]).all()
    assert ids[2, 0, 0] == 12000 and (ids[3] == -1).all() and (best[3] == -np.inf).all()
    h = x.cpu().numpy()
    for r, t in ((0, 5), (1, 6), (2, 7)):
        assert rank[r, 0] == 1 + (h[r] > h[r, t]).sum()
        want = np.argsort(-np.where(np.isnan(h[r]), -np.inf, h[r]), kind="stable")[:3]
        assert np.array_equal(ids[r, 0], want)


def test_clustered_top():
    """The likeliest ids side by side in one place of the row, wherever it lies: more of them than a warp holds."""
    V = 151936
    x = _logits(6, V, torch.bfloat16, 8, std=0.5)
    for r, at in enumerate((0, 1000, 4096 - 20, 70000, V - 700, V - 32)):
        x[r, at:at + 600] += torch.arange(x[r, at:at + 600].numel(), device="cuda").to(torch.bfloat16) * 0.25 + 5
    _check(x, None, [[3], [1500], [4100], [70011], [9], [V - 1]], 1.0, 32)


def test_optional_outputs_and_no_alternatives():
    x = _logits(3, 5000, torch.bfloat16, 9)
    full = _check(x, None, [[1], [2], [-1]], 1.0, 4)
    lp = torch.zeros(3, 1, device="cuda")
    ws = B.alloc_logprobs_workspace(3, 5000, 0)
    B.dspark_token_logprobs(x, None, torch.tensor([[1], [2], [-1]], dtype=torch.int32, device="cuda"), 1.0, lp, None, None,
                            None, None, ws)
    assert torch.equal(lp, full[0])


def test_device_errors():
    """Tokens outside the vocabulary, tokens beyond their window, windows beyond the rows: nothing is asked there, with
    EINVAL; the others are right."""
    x = _logits(6, 2000, torch.float32, 10)
    good = _check(x, [0, 3, 6], [[5, 6, 7], [8, 9, 10]], 1.0, 2)
    ws = B.alloc_logprobs_workspace(6, 2000, 2)

    def call(cu, tokens):
        outs = _outputs(2, 3, 2)
        B.dspark_token_logprobs(x, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                torch.tensor(tokens, dtype=torch.int32, device="cuda"), 1.0, *outs, ws)
        return B.dspark_read_device_status(ws), outs

    assert call([0, 3, 6], [[5, 6, 7], [8, 9, 10]])[0] == B.DSPARK_OK
    for bad in (2000, -2, 2 ** 31 - 1, -2 ** 31):
        st, outs = call([0, 3, 6], [[5, bad, 7], [8, 9, 10]])
        assert st == B.DSPARK_EINVAL
        for o, g in zip(outs, good):
            assert torch.equal(o[1], g[1]) and torch.equal(o[0, 0], g[0, 0]) and torch.equal(o[0, 2], g[0, 2])
        assert outs[0][0, 1] == 0 and outs[2][0, 1] == 0 and (outs[3][0, 1] == -1).all()
    for cu in ([0, 3, 7], [0, 3, 2 ** 31 - 1], [0, 3, 5], [0, 3, 2]):
        st, outs = call(cu, [[5, 6, 7], [8, 9, 10]])
        assert st == B.DSPARK_EINVAL and torch.equal(outs[0][0], good[0][0]) and outs[0][1, 2] == 0
    st, outs = call([-1, 3, 6], [[5, 6, 7], [8, 9, 10]])
    assert st == B.DSPARK_EINVAL and (outs[0][0] == 0).all() and torch.equal(outs[0][1], good[0][1])


@pytest.mark.parametrize("n,per,top", [(1, 1, 5), (40, 4, 20)])
def test_same_bits_on_another_stream_and_in_a_graph(n, per, top):
    V = 50000
    x = _logits(n * per, V, torch.bfloat16, 11)
    tokens = torch.randint(0, V, (n, per), dtype=torch.int32, device="cuda")
    ws = B.alloc_logprobs_workspace(n * per, V, top)
    outs = _outputs(n, per, top)
    B.dspark_token_logprobs(x, None, tokens, 1.0, *outs, ws)
    want = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.dspark_token_logprobs(x, None, tokens, 1.0, *outs, ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("cu", [[2 ** 31 - 1, 4], [2 ** 31 - 1, -2 ** 31], [2 ** 31 - 2, 2], [5, 3], [-2 ** 31, 1]])
def test_lists_at_the_ends_of_32_bits(cu):
    """A window whose rows' numbers pass 32 bits asks nothing, on whole rows and on segments."""
    x = _logits(4, 20000, torch.float32, 11)
    ws = B.alloc_logprobs_workspace(4, 20000, 2)
    outs = _outputs(1, 4, 2)
    B.dspark_token_logprobs(x, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            torch.tensor([[5, 6, 7, 8]], dtype=torch.int32, device="cuda"), 1.0, *outs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_EINVAL
    assert (outs[0] == 0).all() and (outs[2] == 0).all() and (outs[3] == -1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n", [(2000, 40), (30000, 3), (30000, 400)])
def test_ranks_among_ties_and_zeros_of_both_signs(dtype, V, n):
    """Tokens of any likelihood among few values, half of them zeros of either sign, some masked, some NaN and the least
    numbers around 0: the rank counts what is larger, and of what is equal the lower ids."""
    rng = np.random.default_rng(V + n)
    tiny = float(torch.finfo(dtype).tiny) * torch.finfo(dtype).eps  # the least number above 0
    values = np.array([0.0, -0.0, 0.0, -0.0, tiny, -tiny, 1.0, -2.5, 3.0, -np.inf, -1e30, np.nan])
    x = torch.from_numpy(values[rng.integers(0, values.size - (np.arange(n) % 3 != 0)[:, None], (n, V))]).to(dtype).cuda()
    tokens = rng.integers(0, V, (n, 1)).astype(np.int32)
    tokens[:2, 0] = 0, V - 1
    outs = _outputs(n, 1, 3)
    B.dspark_token_logprobs(x, None, torch.from_numpy(tokens).cuda(), 1.0, *outs, B.alloc_logprobs_workspace(n, V, 3))
    host, rank = x.double().cpu().numpy(), outs[2].cpu().numpy()[:, 0]
    assert (host[:, :] == tiny).any() and (np.signbit(host) & (host == 0)).any()
    for r in range(n):
        t = int(tokens[r, 0])
        with np.errstate(invalid="ignore"):
            want = 1 + int((host[r] > host[r, t]).sum() + (host[r, :t] == host[r, t]).sum())
        assert rank[r] == want, (r, t, host[r, t])
