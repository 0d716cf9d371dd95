"""Attention over the 8-bit cache where V's powers of two change from tile to tile while the scores stay as they are.

Each tile's V is nonzero in a lane of its own, so that the bound, which goes by the lane, holds every tile to its own size: a
weight that is kept against an earlier tile's larger V shows at once.  The weights within a tile are alike up to 2^6."""
import numpy as np
import pytest

from tests import kv8_reference as K
from tests import serving_reference as R

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from tests.test_gpu_attention import _f64  # noqa: E402
from tests.test_gpu_kv8 import F8, Cache8, _codes  # noqa: E402

pytestmark = pytest.mark.gpu
PAGE, CTX, BS = 32, 1015, 250  # a pipeline's range has several of a request's eight tiles


def _outputs(n, hq, d, vals, keys=None, q=None, seed=70):
    """BS requests of the same pages: outputs [BS, n, hq, d] and the plain form's of one of them.  vals [CTX + n, 1, d]."""
    c = Cache8([n], [CTX], 1, d, PAGE, seed=seed)
    pos = np.arange(CTX + n)
    at = c.table.cpu().numpy()[0][pos // PAGE], slice(None), pos % PAGE
    scale = c.scale.cpu().numpy().copy()
    if keys is not None:
        byte, k = K.exponent_byte(keys), _codes(c.k).copy()
        k[at], scale[at + (0,)] = K.codes(keys, byte), byte
        c.k, c.keys[0] = torch.from_numpy(k).cuda().view(F8), K.values(k[at], byte)
    byte, v = K.exponent_byte(vals), _codes(c.v).copy()
    v[at], scale[at + (1,)] = K.codes(vals, byte), byte
    c.v, c.vals[0] = torch.from_numpy(v).cuda().view(F8), K.values(v[at], byte)
    c.scale = torch.from_numpy(scale).cuda()
    if q is None:
        q = 0.3 * torch.randn(n, hq, d, generator=torch.Generator().manual_seed(seed + 1))
        q[:, 0] = 0.0  # scores all alike
    q = q.to(torch.bfloat16).cuda()
    cu = torch.arange(0, BS * n + 1, n, dtype=torch.int32, device="cuda")
    ws, out = B.alloc_attention_workspace(hq, 1, d), torch.zeros(BS * n, hq, d, dtype=torch.bfloat16, device="cuda")
    B.dspark_window_attention_kv8(q.repeat(BS, 1, 1), c.k, c.v, c.scale, c.table.repeat(BS, 1), cu, c.ctx.repeat(BS), n, d ** -0.5,
                                  0, 0, out, None, None, None, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK
    ref, _, mag = R.attention(_f64(q), c.keys[0], c.vals[0], CTX, d ** -0.5, 0, 0)
    return _f64(out).reshape(BS, n, hq, d), ref, mag


@pytest.mark.parametrize("n,hq,d", [(1, 4, 128), (8, 4, 128), (16, 4, 64), (16, 8, 128), (16, 8, 64)])
@pytest.mark.parametrize("name,up", [
    ("one fall", [0] + 7 * [-24]), ("steps", [-3 * i for i in range(8)]), ("to and fro", 4 * [0, -30]),
    ("zeros between", [0, None, -12, None, 8, None, None, -40]), ("a rise", [-60, -60, 0, 0, -60, -60, -60, -60])])
def test_tiles_whose_values_change_by_powers_of_two(n, hq, d, name, up):
    tile = np.arange(CTX + n) // 128
    vals = np.zeros((CTX + n, 1, d))
    for t, e in enumerate(up):
        if e is not None:
            vals[tile == t, :, 7 * t + 1] = 2.0 ** e
    got, ref, mag = _outputs(n, hq, d, vals)
    assert (np.abs(got - ref) <= R.attention_bound(mag)).all(), np.abs(got - ref).max((0, 1, 2))


@pytest.mark.parametrize("d", [64, 128])
def test_a_large_value_of_no_weight(d):
    """A V 2^20 times the others' in the first tile, seen with a weight of 2^-40, and nothing beside it there: the tiles behind
    it keep their bits."""
    n, hq = 8, 4
    rng = np.random.default_rng(71)
    vals = rng.standard_normal((CTX + n, 1, d))
    vals[:128] = 0.0
    vals[5, 0, 0] = 2.0 ** 20
    keys = np.zeros((CTX + n, 1, d))
    keys[5] = -40.0 * np.log(2.0) * d ** -0.5
    got, ref, mag = _outputs(n, hq, d, vals, keys, torch.ones(n, hq, d))
    assert (np.abs(got - ref) <= R.attention_bound(mag)).all(), np.abs(got - ref).max()
