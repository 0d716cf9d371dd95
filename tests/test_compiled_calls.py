"""The compiled Python calls: what they raise, and that they keep no references."""
import sys

import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import build as _build  # noqa: E402

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _append(**over):
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k=torch.zeros(3, 2, 64, dtype=torch.bfloat16),
             v=torch.zeros(3, 2, 64, dtype=torch.bfloat16), cu_seqlens=torch.zeros(3, dtype=I32),
             ctx_len=torch.zeros(2, dtype=I32), cos_sin=torch.zeros(9, 64), page_table=torch.zeros(2, 5, dtype=I32),
             q_out=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k_cache=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16),
             v_cache=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), ws=torch.zeros(64, dtype=torch.uint8), stream=0)
    return {**a, **over}


@pytest.mark.parametrize("key,val", [
    ("q", torch.zeros(3, 4, 64)), ("q", torch.zeros(2, 4, 64, dtype=torch.bfloat16)), ("q", torch.zeros(3, 256, dtype=torch.bfloat16)),
    ("k", torch.zeros(3, 2, 32, dtype=torch.bfloat16)), ("k", torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2)),
    ("v", torch.zeros(3, 3, 64, dtype=torch.bfloat16)), ("cu_seqlens", torch.zeros(3)), ("cu_seqlens", torch.zeros(3, 1, dtype=I32)),
    ("ctx_len", torch.zeros(3, dtype=I32)), ("ctx_len", torch.zeros(4, dtype=I32)[::2]), ("cos_sin", torch.zeros(9, 64, 1)),
    ("page_table", torch.zeros(3, 5, dtype=I32)), ("page_table", torch.zeros(2, 10, dtype=I32)[:, ::2]),
    ("q_out", torch.zeros(3, 2, 64, dtype=torch.bfloat16)), ("v_cache", torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16)),
    ("k_cache", torch.zeros(4, 2, 16, dtype=torch.bfloat16))])
def test_append_refuses(key, val):
    with pytest.raises(ValueError):
        B.dspark_append_kv(**_append(**{key: val}))


def test_library_status_is_raised():
    with pytest.raises(B.DSparkError) as e:  # the workspace is too small: refused by the library before any launch
        B.dspark_append_kv(**_append())
    assert e.value.args and "dspark_append_kv" in str(e.value)
    with pytest.raises(B.DSparkError):
        B.dspark_history_commit(torch.zeros(2, 8, dtype=I32), torch.zeros(2, 64, dtype=torch.int16),
                                torch.zeros(8, dtype=torch.uint8), stream=0)


def test_other_objects_are_refused():
    for over in (dict(q=3), dict(k=None), dict(ws=None), dict(stream="x"), dict(page_table=[1])):
        with pytest.raises((AttributeError, TypeError, ValueError)):
            B.dspark_append_kv(**_append(**over))


def test_no_references_are_kept():
    a = _append()
    before = {k: sys.getrefcount(t) for k, t in a.items()}
    none = sys.getrefcount(torch.bfloat16)
    for _ in range(50):
        with pytest.raises(B.DSparkError):
            B.dspark_append_kv(**a)
        with pytest.raises(ValueError):
            B.dspark_append_kv(**{**a, "cu_seqlens": torch.zeros(3)})
    assert {k: sys.getrefcount(t) for k, t in a.items()} == before
    assert abs(sys.getrefcount(torch.bfloat16) - none) <= 1
