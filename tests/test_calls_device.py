"""The compiled Python calls refuse tensors in host memory, with workspaces and shapes that are otherwise right: nothing is
launched (no GPU)."""
import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import build as _build  # noqa: E402

I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _ws(n=1 << 16):
    t = torch.zeros(n + 256, dtype=torch.uint8)
    skip = -t.data_ptr() % 256
    return t[skip:skip + n]


def _calls():
    i = lambda *s: torch.zeros(*s, dtype=I32)  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    hist = torch.zeros(2, 64, dtype=torch.int16)
    return {
        "dspark_append_kv": (b(3, 4, 64), b(3, 2, 64), b(3, 2, 64), i(3), i(2), torch.zeros(9, 64), i(2, 5), b(3, 4, 64),
                             b(4, 2, 16, 64), b(4, 2, 16, 64), _ws()),
        "dspark_window_attention": (b(3, 4, 64), b(4, 2, 16, 64), b(4, 2, 16, 64), i(2, 5), i(3), i(2), 3, 1.0, 0, 0, b(3, 4, 64),
                                    torch.zeros(3, 4), _ws(1 << 26)),
        "dspark_process_logits": (torch.zeros(3, 64), i(3), i(3), hist, torch.ones(2), torch.ones(2), torch.ones(2), i(3), i(1),
                                  torch.zeros(1), i(3, 2), torch.zeros(3, 64), _ws()),
        "dspark_history_build": (i(5), i(3), i(2), hist, _ws()),
        "dspark_history_commit": (i(2, 8), hist, _ws()),
    }


@pytest.mark.parametrize("stream", [0, None])
@pytest.mark.parametrize("name", list(_calls()))
def test_host_tensors_are_refused(name, stream):
    with pytest.raises(B.DSparkDeviceError, match=name + ": .* must be on the current CUDA device") as e:
        getattr(B, name)(*_calls()[name], stream=stream)
    assert e.value.status == B.DSPARK_EINVAL and isinstance(e.value, ValueError)


def test_shapes_are_looked_at_first():
    q, *rest = _calls()["dspark_append_kv"]
    with pytest.raises(ValueError, match="q must have shape") as e:
        B.dspark_append_kv(q[:2], *rest, stream=0)
    assert not isinstance(e.value, B.DSparkDeviceError)


@pytest.mark.parametrize("name", list(_calls()))
def test_a_workspace_that_is_no_block_of_bytes(name):
    """An expanded byte has as many entries as one likes, and no memory behind them."""
    args = _calls()[name][:-1]
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 26), _ws(1 << 10)[::2]):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            getattr(B, name)(*args, ws, stream=0)
