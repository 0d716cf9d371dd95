"""How far the two e4m3 parts of a query's lane are from the lane: exhaustively on the CPU, and by the log-sum-exp of a single
position, which is the score itself, on the GPU."""
import numpy as np
import pytest

from tests import kv8_reference as K

EXACT, OFF = 2.0 ** -9.8, 2.0 ** -17.8  # of the row's largest: lanes from there on are exact, others off by at most that


def _nearest(x):
    grid = K.VALUES[:127]
    a = np.abs(x)
    i = np.clip(np.searchsorted(grid, a), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    return np.sign(x) * np.where((a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0)), hi, lo)


def test_every_lane_beside_every_largest():
    lanes = (np.arange(128, 256)[None] * 2.0 ** np.arange(-25, 2)[:, None]).ravel()  # bf16, under the row's power of two
    lanes = lanes[lanes <= 448]
    first = _nearest(lanes)
    err = np.abs(lanes - first - _nearest(lanes - first))
    for top in lanes[lanes > 224]:
        assert err[(lanes >= EXACT * top) & (lanes <= top)].max() == 0 and err.max() <= OFF * top
    assert err.max() > 2.0 ** -19 * 448  # no smaller bound holds


@pytest.mark.gpu
@pytest.mark.parametrize("n,hq,d", [(1, 4, 64), (8, 4, 128), (16, 8, 64), (16, 8, 128)])
def test_scores(n, hq, d):
    """A large lane, which K does not have, beside small ones: the worst that both bounds allow, and everything between."""
    torch = pytest.importorskip("torch")
    from speculative_decoding_draft_markov_gb300 import binding as B
    rng = np.random.default_rng(80)
    q = np.zeros((n, hq, d))
    top = rng.choice([225.0, 448.0, 300.0], (n, hq, 1)) * 2.0 ** rng.integers(-20, 20, (n, hq, 1))
    q[..., 1:] = top / 225 * 0.2490234375 * rng.choice([1.0, 1.0, 0.37, 2.0 ** -5, 1.03, 4.0], (n, hq, d - 1))
    q[..., :1] = top
    q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    qn = q.double().cpu().numpy()
    k = torch.full((n, 1, 8, d), 0x38, dtype=torch.uint8)  # 1.0
    k[..., 0] = 0
    f8 = torch.float8_e4m3fn
    scale = torch.full((n, 1, 8, 2), 127, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(n, hq, device="cuda")
    ws = B.alloc_attention_workspace(hq, 1, d)
    # each row a request of its own, which sees its own position alone
    B.dspark_window_attention_kv8(q, k.cuda().view(f8), k.cuda().view(f8), scale, torch.arange(n, **i32)[:, None],
                                  torch.arange(n + 1, **i32), torch.zeros(n, **i32), n, 1.0, 0, 0, out, lse, None, None, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    want, largest = qn[..., 1:].sum(-1), np.abs(qn).max(-1)
    small = np.where(np.abs(qn) < EXACT * largest[..., None], 1, 0).sum(-1)
    # and the rounding of a sum of 2 d products in fp32, of the factor and of the logarithm
    bound = OFF * largest * small + 2.0 ** -22 * (d * np.abs(qn[..., 1:]).sum(-1) + np.abs(want)) + 1e-6
    off = np.abs(lse.cpu().numpy() - want)
    assert (off <= bound).all(), (off / bound).max()
    assert (out.float().cpu().numpy()[..., 1:] == 1.0).all()
