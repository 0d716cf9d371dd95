"""Pointers that no 4-byte load may use, and an output that lies over strided queries, are refused on the host before
anything is launched (no GPU; pointers are host buffers that no call may touch)."""
import pytest

pytest.importorskip("torch")
from tests.test_serving_abi import APPEND, ATTEND, BUILD, COMMIT, EINVAL, PTR, RULES, _try, lib  # noqa: E402,F401


@pytest.mark.parametrize("off", [1, 2])
@pytest.mark.parametrize("name,args,keys", [
    ("dspark_append_kv", APPEND, ["cu", "ctx", "table"]),
    ("dspark_window_attention", ATTEND, ["cu", "ctx", "table"]),
    ("dspark_process_logits", RULES, ["cu", "ids", "repetition", "frequency", "presence", "bias_start", "bias_ids", "bias_vals",
                                      "mask"]),
    ("dspark_history_build", BUILD, ["tokens", "start", "n_prompt"]),
    ("dspark_history_commit", COMMIT, ["out_tokens"])])
def test_misaligned_words_are_refused(lib, name, args, keys, off):  # noqa: F811
    if name == "dspark_window_attention":
        args = dict(args, q_stride=1024)
    for key in keys:
        assert _try(lib, name, args, {key: PTR + off}) == EINVAL, key


def test_attention_refuses_strided_in_place(lib):  # noqa: F811
    assert _try(lib, "dspark_window_attention", ATTEND, {"q": PTR, "out": PTR, "q_stride": 1536}) == EINVAL
