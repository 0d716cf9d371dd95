"""One tensor of a target-side call in host memory, the others on the GPU: refused by name before anything is launched."""
import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from tests.test_calls_device import _calls  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", list(_calls()))
def test_each_tensor_alone(name):
    args = _calls()[name]
    at = [i for i, x in enumerate(args) if torch.is_tensor(x)]
    dev = [x.cuda() if torch.is_tensor(x) else x for x in args]
    for i in at:
        mixed = list(dev)
        mixed[i] = args[i]
        with pytest.raises(B.DSparkDeviceError):
            getattr(B, name)(*mixed)
    getattr(B, name)(*dev)  # empty windows: nothing to do
    getattr(B, name)(*dev, stream=torch.cuda.current_stream())
    assert B.dspark_read_device_status(dev[-1]) == B.DSPARK_OK
