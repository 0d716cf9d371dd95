"""Device code that also runs on the host, built as a shared library for the tests."""
import ctypes
import os
import subprocess

from speculative_decoding_draft_markov_gb300 import build as _build

HERE = os.path.dirname(os.path.abspath(__file__))


def load(name: str, folder) -> ctypes.CDLL:
    """tests/host/<name>.cu compiled into `folder`."""
    out = os.path.join(str(folder), name + ".so")
    cmd = [_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-O1", "-I" + _build.CSRC, "-shared", "-o", out,
           os.path.join(HERE, "host", name + ".cu")]
    res = subprocess.run([c for c in cmd if c != "-O3"], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    return ctypes.CDLL(out)
