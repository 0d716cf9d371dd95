"""Building where Python's headers are missing: the library is there, and the calls that need the extension module say
that it is not."""
import os

import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import build as _build  # noqa: E402


def test_build_without_python_headers(monkeypatch, tmp_path, capsys):
    _build.build()
    calls = tmp_path / "_calls.so"
    calls.write_bytes(b"of older sources")
    os.utime(calls, (0, 0))
    monkeypatch.setattr(_build, "CALLS", str(calls))
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB)
    assert "no Python.h" in capsys.readouterr().err and not calls.exists()


def test_calls_without_their_module_say_so(monkeypatch, tmp_path):
    _build.build()
    B.lib()
    monkeypatch.setattr(B, "_CALLS", None)
    monkeypatch.setattr(B, "library_path", lambda: str(tmp_path / "libdspark.so"))
    with pytest.raises(RuntimeError, match="_calls.so is not built"):
        B.dspark_history_commit(torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 64, dtype=torch.int16),
                                torch.zeros(256, dtype=torch.uint8), stream=0)
