"""A prompt's chunk among short windows over the 8-bit cache: by way of bf16 pages and without them, through the paged cache."""
import numpy as np
import pytest

from tests import serving_reference as R

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import serving as V  # noqa: E402
from tests.test_gpu_kv8 import Cache8, _check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hkv,window", [(128, 8, 2, 0), (64, 8, 2, 0), (64, 8, 1, 200)])
@pytest.mark.parametrize("scratch", [False, True])
def test_a_chunk_among_windows(d, hq, hkv, window, scratch):
    ns = [3, 1, 300, 8, 0, 5] + [8] * 20
    ctxs = [700, 12, 60, 1500, 9, 31] + [37 * i for i in range(20)]
    c = Cache8(ns, ctxs, hkv, d, 32, seed=90, evict=(window, 4) if window else None)
    _check(c, hq, window, 4 if window else 0, seed=91, scratch=scratch)


def test_the_paged_cache_need_not_read_back():
    bs, hq, hkv, d, page = 3, 8, 2, 64, 16
    ns = [2, 300, 4]
    rows = sum(ns)
    g = torch.Generator(device="cuda")
    g.manual_seed(92)
    q, k, v = (torch.randn(rows, h, d, device="cuda", generator=g).to(torch.bfloat16) for h in (hq, hkv, hkv))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device="cuda")
    outs = []
    for widen in (True, False):
        cache = V.PagedCache(1, 40, page, hq, hkv, d, bs, 30, V.rotation_table(400, d), eight_bit=True)
        for r, n in enumerate(ns):
            cache.reserve(r, n)
        for w in cache.wide:
            w.fill_(7.0)
        outs.append(torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda"))
        cache.attend(0, q, k, v, cu, max(ns), d ** -0.5, outs[-1], widen=widen)
        assert B.dspark_read_device_status(cache.ws) == B.DSPARK_OK
        assert all((w == 7.0).all().item() != widen for w in cache.wide)
    a, b = (o.double().cpu().numpy() for o in outs)
    # both are off from the same value by at most the bound of its size: a row's weights times |V|, V below 6
    assert np.abs(a - b).max() <= 2 * R.attention_bound(6.0)
    plain = V.PagedCache(1, 40, page, hq, hkv, d, bs, 30, V.rotation_table(400, d))
    for r, n in enumerate(ns):
        plain.reserve(r, n)
    out = torch.zeros_like(outs[0])
    plain.attend(0, q, k, v, cu, max(ns), d ** -0.5, out, widen=False)  # says nothing to a 16-bit cache
    assert torch.isfinite(out).all() and B.dspark_read_device_status(plain.ws) == B.DSPARK_OK
