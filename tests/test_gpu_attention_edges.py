"""The windows' attention where its memory, its masks and its waits can go wrong: work that fits its rings when a wait
runs out."""
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
