"""Log probabilities of rows with logits of every size, against a plain 64-bit form.

Bounds.  A difference of two fp32 logits is rounded to 2^-24 of itself, and so are its product with log2(e) / T, that factor (two
roundings), ln 2 and the last product: 2^-21 of the result in all.  A row's sum passes at most 60000 / 256 / 2 additions of a thread
and some twenty more, each rounded to 2^-24, with exponentials that are off by 2^-22: less than 2^-16 of it, of which the logarithm
makes as much in absolute terms.  Nothing of it grows with the logits themselves."""
import numpy as np
import pytest

from tests import kv8_reference as K

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu
RTOL, ATOL = 2.0 ** -21, 2.0 ** -16


def _call(x, tokens, temperature=1.0, top=3):
    n = len(tokens)
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    outs = [torch.full((n, 1), 5.0, **f32), torch.full((n, 1), 5.0, **f32), torch.full((n, 1), 5, **i32),
            torch.full((n, 1, top), 5, **i32), torch.full((n, 1, top), 5.0, **f32)]
    ws = B.alloc_logprobs_workspace(n, x.shape[1], top)
    B.dspark_token_logprobs(x, None, torch.tensor(tokens, **i32)[:, None], temperature, *outs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    return [o.cpu().numpy()[:, 0] for o in outs]


def _check(x, tokens, temperature=1.0, top=3):
    lp, ent, rank, ids, best = _call(x, tokens, temperature, top)
    h = x.double().cpu().numpy()
    for r, t in enumerate(tokens):
        want = K.token_logprobs(h[r], t, temperature, top)
        np.testing.assert_allclose(lp[r], want[0], rtol=RTOL, atol=ATOL)
        np.testing.assert_allclose(best[r], want[4], rtol=RTOL, atol=ATOL)
        # W / S: terms d 2^d, |d| below 25, where they count
        np.testing.assert_allclose(ent[r], want[1], rtol=RTOL, atol=32 * ATOL)
        assert rank[r] == want[2] and np.array_equal(ids[r], want[3])
        assert lp[r] <= 0 and (best[r] <= 0).all()


SIZES = [1e3, 1e5, 1e6, 1e7, 1e8, 1e9, 3.3e9, 1e10, 1e12, 1e20, 9e29, 1e31]


@pytest.mark.parametrize("V,rows", [(9000, 1), (60000, 1), (60000, 700)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_forced_id_and_rows_of_one_value(dtype, V, rows):
    """One id at L over a row of zeros has log probability 0, and a row of one value -log V, whatever L is; cut in segments and
    whole."""
    for L in SIZES:
        x = torch.zeros(4, V, device="cuda")
        x[0, V - 11] = L
        x[1, 17] = L
        x[2] = -L
        x[3] = L
        tokens, x = [V - 11, 40, 77, V - 1], x.to(dtype)
        if rows > 4:
            x, tokens = x.repeat(rows // 4, 1), tokens * (rows // 4)
            lp, ent, rank, ids, best = (o.reshape((rows // 4,) + (4,) + o.shape[1:]) for o in _call(x, tokens))
            assert all((o == o[0]).all() for o in (lp, ent, rank, ids, best))
        else:
            lp, ent, rank, ids, best = (o[None] for o in _call(x, tokens))
        real = float(x[0, V - 11])
        assert lp[0, 0] == 0 and best[0, 0, 0] == 0 and abs(ent[0, 0]) < 1e-6, (L, lp[0, 0])
        np.testing.assert_allclose(lp[0, 1], -real, rtol=RTOL)
        np.testing.assert_allclose(lp[0, 2:], -np.log(V), atol=ATOL)
        np.testing.assert_allclose(ent[0, 2:], np.log(V), atol=ATOL)
        np.testing.assert_allclose(best[0, 2:], -np.log(V), atol=ATOL)
        assert rank[0].tolist() == [1, 41, 78, V] and ids[0, 2].tolist() == [0, 1, 2] and ids[0, 1].tolist() == [17, 0, 1]


@pytest.mark.parametrize("value", [-1e4, -1e9, -1e10, -3e11, -1e15, -1e20, -5e29, -1e30])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_of_finite_values(dtype, value):
    """Few allowed ids, in one place and scattered, the others at a finite value: before a thread's allowed ids, behind them, and
    all that some threads have."""
    for V, rows in ((30000, 3), (9000, 700)):
        rng = np.random.default_rng(7)
        x = torch.full((3, V), value, device="cuda")
        x[0, V - 300:] = torch.from_numpy(3 * rng.standard_normal(300)).float().cuda()
        x[1, :200] = torch.from_numpy(3 * rng.standard_normal(200)).float().cuda()
        some = torch.from_numpy(rng.permutation(V)[:500]).cuda()
        x[2, some] = torch.from_numpy(3 * rng.standard_normal(500)).float().cuda()
        x = x.to(dtype)
        tokens = [V - 7, 3, int(some[8])]
        if rows == 3:
            _check(x, tokens, top=20)
        else:
            got = _call(x.repeat(rows // 3, 1), tokens * (rows // 3), top=20)
            want = [K.token_logprobs(x[r].double().cpu().numpy(), t, 1.0, 20) for r, t in enumerate(tokens)]
            np.testing.assert_allclose(got[0].reshape(-1, 3), np.broadcast_to([w[0] for w in want], (rows // 3, 3)), rtol=RTOL, atol=ATOL)
            assert np.array_equal(got[3].reshape(-1, 3, 20), np.broadcast_to([w[3] for w in want], (rows // 3, 3, 20)))


@pytest.mark.parametrize("temperature", [1.0, 0.1, 0.01, 1e-4, 1e-8, 30.0, 1e29])
@pytest.mark.parametrize("base", [0.0, 35.0, -1e5, 1e7])
def test_log_probabilities_are_never_above_0(temperature, base):
    """The likeliest token before the others by any distance: 0 at the most, and right, at every temperature."""
    rng = np.random.default_rng(8)
    x = torch.from_numpy(base + rng.standard_normal((24, 20000))).float().cuda()
    tokens = rng.integers(0, 20000, 24)
    for r, t in enumerate(tokens):
        x[r, t] = base + 5.0 + r * (1.0 + abs(base) * 2.0 ** -20)
    _check(x, tokens.tolist(), temperature)


def test_prompts():
    """Few requests of many tokens each: the next tokens of whole prompts, -1 at their ends."""
    V, cu = 2000, [0, 3000, 3001, 7001]
    x = (3 * torch.randn(cu[-1], V, generator=torch.Generator().manual_seed(9))).to(torch.bfloat16).cuda()
    rng = np.random.default_rng(10)
    per = 4000
    tokens = np.full((3, per), -1, np.int32)
    for r in range(3):
        n = cu[r + 1] - cu[r]
        tokens[r, :n - 1] = rng.integers(0, V, n - 1)
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    outs = [torch.full((3, per), 5.0, **f32), torch.full((3, per), 5.0, **f32), torch.full((3, per), 5, **i32),
            torch.full((3, per, 4), 5, **i32), torch.full((3, per, 4), 5.0, **f32)]
    ws = B.alloc_logprobs_workspace(3 * per, V, 4)
    B.dspark_token_logprobs(x, torch.tensor(cu, **i32), torch.from_numpy(tokens).cuda(), 0.7, *outs, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    h = x.double()
    lse = torch.logsumexp(h / 0.7, 1)
    for r in range(3):
        n = cu[r + 1] - cu[r] - 1
        rows, t = torch.arange(cu[r], cu[r] + n, device="cuda"), torch.from_numpy(tokens[r, :n]).long().cuda()
        chosen = h[rows, t]
        np.testing.assert_allclose(outs[0][r, :n].cpu().numpy(), (chosen / 0.7 - lse[rows]).cpu().numpy(), rtol=RTOL, atol=ATOL)
        before = (h[rows] > chosen[:, None]) | ((h[rows] == chosen[:, None]) & (torch.arange(V, device="cuda") < t[:, None]))
        assert torch.equal(outs[2][r, :n].long(), 1 + before.sum(1))
        order = torch.sort(h[rows], dim=1, descending=True, stable=True).indices[:, :4]
        assert torch.equal(outs[3][r, :n].long(), order)
        assert (outs[0][r, n:] == 0).all() and (outs[2][r, n:] == 0).all() and (outs[3][r, n:] == -1).all()
