"""The 8-bit cache's bookkeeping on the host, and the order in which its attention's two loading warps fill the ring (no GPU)."""
import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import build as _build  # noqa: E402
from speculative_decoding_draft_markov_gb300 import serving as V  # noqa: E402
from tests import host_library, kv8_reference as K  # noqa: E402


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    _build.build()
    return host_library.load("kv8_ring", tmp_path_factory.mktemp("host"))


def test_pages_of_eight_bits(host):
    c = V.PagedCache(2, 5, 16, 2, 1, 64, 2, 4, V.rotation_table(64, 64, device="cpu"), device="cpu", eight_bit=True)
    assert [t.dtype for t in c.k + c.v] == [torch.float8_e4m3fn] * 4 and c.k[0].shape == (5, 1, 16, 64)
    assert [t.shape for t in c.scale] == [(5, 1, 16, 2)] * 2 and len(c.wide) == 2 and c.wide[0].dtype == torch.bfloat16
    c.reserve(0, 17)
    c.settle(0, 16)
    c.reserve(0, 16)
    assert len(c.pages[0]) == 2
    wide = V.PagedCache(1, 5, 16, 2, 1, 64, 2, 4, V.rotation_table(64, 64, device="cpu"), device="cpu")
    assert wide.k[0].dtype == torch.bfloat16 and not hasattr(wide, "scale")
    with pytest.raises(B.DSparkDeviceError):  # host memory
        c.read_back(0, torch.tensor([0, 1, 2], dtype=torch.int32), 2)


def test_a_report_without_a_gpu_is_refused(host):
    r = V.Logprobs.allocate(2, 3, 64, 4, device="cpu")
    assert r.top_ids.shape == (2, 4, 4) and r.logprob.shape == (2, 4)

    class Buf:
        packed, cu = torch.zeros(8, 64), torch.tensor([0, 4, 8], dtype=torch.int32)
        out_tokens = torch.zeros(2, 4, dtype=torch.int32)

    with pytest.raises(B.DSparkDeviceError):
        r.take(Buf)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 9, 50])
def test_the_rings_order(host, n):
    """K 0, K 1, V 0, K 2, V 1 and so on: every place of the ring is one load's, and none is left out."""
    want = []
    for i in range(n):
        if i < 2:
            want.append(("k", i))
    for i in range(n):
        want.append(("v", i))
        if i + 2 < n:
            want.append(("k", i + 2))
    for at, (what, i) in enumerate(want):
        assert host.ring_place(int(what == "v"), i, n) == at, (what, i)


def test_exponent_bytes(host):
    """The kernels' exponent bytes, at and beside every power of two and 448 of it, against 64 bits."""
    import ctypes
    import numpy as np
    host.exponent_byte.restype = ctypes.c_uint
    for e in list(range(-149, 128)):
        for m in (1.0, 1.75, float(np.nextafter(np.float32(1.75), np.float32(2))), 1.9999):
            x = np.float32(min(m * 2.0 ** e, 3.4028234e38))
            got = host.exponent_byte(int(x.view(np.uint32)))
            assert got == int(K.exponent_byte(np.array([[float(x)]]))[0]), (e, m)
    assert host.exponent_byte(0) == 1 and host.exponent_byte(0x7F800000) == 255 and host.exponent_byte(0x7FC00000) == 255


def test_a_step_refuses_a_report_of_other_sizes(host):
    """Before anything of the step has run."""
    class Buf:
        out_tokens = torch.zeros(2, 4, dtype=torch.int32)

    for bs, gamma in ((3, 3), (2, 2)):
        with pytest.raises(ValueError, match="logprobs"):
            V.run_served_step({}, Buf, None, None, None, None, 1.0, 0, 0,
                              logprobs=V.Logprobs.allocate(bs, gamma, 64, 0, device="cpu"))


@pytest.mark.parametrize("temperature", [0.0, -1.0, float("inf"), float("nan")])
def test_a_report_at_no_temperature_is_refused(host, temperature):
    with pytest.raises(ValueError, match="temperature"):
        V.Logprobs.allocate(2, 3, 64, 4, temperature, device="cpu")
