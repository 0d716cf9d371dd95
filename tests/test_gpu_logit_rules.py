"""Penalties, biases, masks and the token history on the GPU, against plain 64-bit forms."""
import numpy as np
import pytest

from tests import serving_reference as R

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu

BIG = 2 ** 30


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def _dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda") if dtype is None else torch.tensor(x, dtype=dtype, device="cuda")


class Batch:
    def __init__(self, ns, V, dtype, seed, pad=2, use_mask=True, n_bias=5, pen=True):
        rng = np.random.default_rng(seed)
        self.ns, self.V, bs = ns, V, len(ns)
        rows = sum(ns) + pad
        self.cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.logits = torch.from_numpy(rng.normal(0, 3, (rows, V)).astype(np.float32)).to(dtype)
        pool = rng.integers(0, V, 12)
        self.ids = pool[rng.integers(0, 12, rows)].astype(np.int32)  # tokens repeat inside a window
        self.hist = np.zeros((bs, V), np.int16)
        for r in range(bs):
            said = np.concatenate([rng.integers(0, V, 30), np.repeat(pool[:3], 4)])
            self.hist[r] = R.history_words(rng.integers(0, V, 40), said, V)
        self.rho = np.where(rng.random(bs) < 0.3, 1.0, rng.uniform(0.8, 2.0, bs)).astype(np.float32)
        self.freq = rng.uniform(-0.5, 1.0, bs).astype(np.float32)
        self.pres = rng.uniform(-0.5, 1.0, bs).astype(np.float32)
        if not pen:
            self.rho[:], self.freq[:], self.pres[:] = 1, 0, 0
        per = [0 if r % 3 == 2 else min(n_bias + r, V) for r in range(bs)]
        self.bias_start = np.concatenate([[0], np.cumsum(per)]).astype(np.int32)
        self.bias_ids = np.concatenate([np.sort(rng.permutation(V)[:m]) for m in per]).astype(np.int32)
        self.bias_vals = rng.normal(0, 5, self.bias_ids.size).astype(np.float32)
        self.allowed = rng.random((rows, V)) < np.where(rng.random(rows) < 0.5, 0.02, 0.98)[:, None]
        self.allowed[rows // 2] = False  # a mask that leaves nothing
        if not use_mask:
            self.allowed[:] = True
        words = np.zeros((rows, (V + 31) // 32 * 32), bool)
        words[:, :V] = self.allowed
        self.mask = np.packbits(words, axis=1, bitorder="little").view(np.int32) if use_mask else None

    def call(self, out=None, logits=None, ws=None, **over):
        logits = self.logits.cuda() if logits is None else logits
        out = torch.full_like(logits, 7.0) if out is None else out
        ws = _ws() if ws is None else ws
        a = dict(hist=_dev(self.hist), repetition=_dev(self.rho), frequency=_dev(self.freq), presence=_dev(self.pres),
                 bias_start=_dev(self.bias_start), bias_ids=_dev(self.bias_ids), bias_vals=_dev(self.bias_vals),
                 mask=None if self.mask is None else _dev(self.mask))
        a.update(over)
        B.dspark_process_logits(logits, _dev(self.cu), _dev(self.ids), out=out, ws=ws, **a)
        return out, B.dspark_read_device_status(ws)

    def check(self, out, hist=True, bias=True):
        x = self.logits.float().numpy()
        got = out.float().cpu().numpy().astype(np.float64)
        u = R.BF16 if self.logits.dtype == torch.bfloat16 else 2.0 ** -24
        for r, n in enumerate(self.ns):
            a, b = self.cu[r], self.cu[r + 1]
            w = self.hist[r].astype(np.int64) & 0xFFFF if hist else np.zeros(self.V, np.int64)
            full = np.zeros(self.V)
            if bias:
                e = slice(self.bias_start[r], self.bias_start[r + 1])
                full[self.bias_ids[e]] = self.bias_vals[e]
            ids = self.ids[a:b] if hist else np.full(n, -1)
            pen = [float(t[r]) if hist else d for t, d in ((self.rho, 1.0), (self.freq, 0.0), (self.pres, 0.0))]
            ref, mag = R.logit_rules(x[a:b], ids, w & 0x7FFF, w >> 15 > 0, *pen, full, self.allowed[a:b])
            assert np.array_equal(np.isinf(got[a:b]), np.isinf(ref))
            fin = np.isfinite(ref)
            # the product, the three sums: five fp32 roundings of terms of size mag; then the type's own
            bound = u * np.abs(ref[fin]) + 6 * 2.0 ** -24 * mag[fin]
            assert (np.abs(got[a:b][fin] - ref[fin]) <= bound).all()
        assert (got[self.cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ns,V", [([1], 8), ([1], 1000), ([3, 0, 8, 1, 17], 2056), ([5, 2], 4104), ([9, 4, 1], 32768 + 24)])
@pytest.mark.parametrize("use_mask", [False, True])
def test_rules(ns, V, dtype, use_mask):
    b = Batch(ns, V, dtype, seed=V + len(ns), use_mask=use_mask)
    out, st = b.call()
    assert st == B.DSPARK_OK
    b.check(out)
    # in place: the same bits
    x = b.logits.cuda()
    x[sum(ns):] = 7.0
    got, st = b.call(out=x, logits=x)
    assert st == B.DSPARK_OK and torch.equal(got, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rules_many_short_windows(dtype):
    """Windows of one row in the main, a longer one, empty ones."""
    ns = [1] * 100 + [6, 0, 0, 2] + [1] * 60
    b = Batch(ns, 8200, dtype, seed=36, n_bias=3)
    out, st = b.call()
    assert st == B.DSPARK_OK
    b.check(out)
    x = b.logits.cuda()
    x[sum(ns):] = 7.0
    got, st = b.call(out=x, logits=x)
    assert st == B.DSPARK_OK and torch.equal(got, out)


@pytest.mark.parametrize("bs,n,V,dtype", [(130, 4, 10248, torch.bfloat16), (128, 16, 8192, torch.float32)])
def test_rules_large_batches(bs, n, V, dtype):
    """More blocks than the SMs hold: a window's rows in one block, or shared by two."""
    rng = np.random.default_rng(bs)
    b = Batch([int(x) for x in rng.integers(n // 2, n + n // 2 + 1, bs)], V, dtype, seed=38, n_bias=2)
    out, st = b.call()
    assert st == B.DSPARK_OK
    b.check(out)


@pytest.mark.parametrize("n_bias", [60, 65, 700, 5000])
def test_rules_many_biases(n_bias):
    """Lists that a warp searches in one, two and more steps, as long as the vocabulary at last."""
    b = Batch([2, 5, 1, 3], 5000, torch.float32, seed=32, n_bias=n_bias)
    out, st = b.call()
    assert st == B.DSPARK_OK
    b.check(out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rules_one_by_one(dtype):
    b = Batch([4, 2, 3], 3000, dtype, seed=31)
    none = dict(hist=None, repetition=None, frequency=None, presence=None)
    no_bias = dict(bias_start=None, bias_ids=None, bias_vals=None)
    out, st = b.call(**none)
    assert st == B.DSPARK_OK
    b.check(out, hist=False)
    out, st = b.call(**no_bias)
    assert st == B.DSPARK_OK
    b.check(out, bias=False)
    mask = b.mask
    b.mask, b.allowed = None, np.ones_like(b.allowed)
    out, st = b.call(**none, **no_bias)  # nothing to do: a copy
    assert st == B.DSPARK_OK and torch.equal(out[:9], b.logits.cuda()[:9])
    b.rho[:], b.pres[:] = 1.0, 0.0
    out, st = b.call(repetition=None, presence=None)
    assert st == B.DSPARK_OK
    b.check(out)
    assert mask is not None


def test_rules_infinities_and_nan():
    """-inf stays; what a mask hides becomes -inf even if it was NaN or infinite; a NaN that is allowed stays one."""
    V = 64
    x = torch.zeros(2, V, dtype=torch.bfloat16)
    x[0, :4] = torch.tensor([float("nan"), float("inf"), float("-inf"), float(torch.finfo(torch.bfloat16).min)])
    x[1] = x[0]
    allowed = np.ones((2, V), bool)
    allowed[0, :3] = False
    mask = np.packbits(allowed, axis=1, bitorder="little").view(np.int32)
    hist = np.zeros((1, V), np.int16)
    hist[0, :8] = 2
    one = torch.ones(1, device="cuda")
    out = torch.empty_like(x, device="cuda")
    ws = _ws()
    B.dspark_process_logits(x.cuda(), _dev([0, 2], torch.int32), _dev([1, 9], torch.int32), _dev(hist), 2 * one, one, one,
                            None, None, None, _dev(mask), out, ws)
    got = out.float().cpu().numpy()
    assert np.isneginf(got[0, :3]).all() and np.isneginf(got[0, 3])  # the lowest value, doubled, is beyond bf16
    assert np.isnan(got[1, 0]) and np.isposinf(got[1, 1]) and np.isneginf(got[1, 2])
    assert (got[1, 4:8] == -3.0).all() and got[0, 9] == 0.0 and got[1, 9] == -2.0


def test_rules_device_errors():
    b = Batch([3, 2, 4], 512, torch.bfloat16, seed=33, n_bias=9)
    good, st = b.call()
    assert st == B.DSPARK_OK
    for bad in ([0, 3, 5, 12], [0, 5, 3, 9], [-1, 3, 5, 9]):
        keep, b.cu = b.cu, np.array(bad, np.int32)
        out, st = b.call()
        assert st == B.DSPARK_EINVAL
        b.cu = keep
    keep = b.bias_ids.copy()
    for at, val in ((1, keep[0]), (0, -1), (b.bias_start[1] - 1, 512)):
        b.bias_ids = keep.copy()
        b.bias_ids[at] = val
        assert b.call()[1] == B.DSPARK_EINVAL
    b.bias_ids = keep
    for val in (-1, 512, 2 ** 31 - 1):
        ids, b.ids = b.ids, b.ids.copy()
        b.ids[1] = val
        out, st = b.call()
        assert st == B.DSPARK_EINVAL and torch.equal(out[0], good[0]) and torch.equal(out[3:9], good[3:9])
        b.check(out)
        b.ids = ids


def test_rules_bias_entries_out_of_range():
    """Entries that are not inside the list: reported; the other requests are served."""
    b = Batch([3, 2, 4], 512, torch.bfloat16, seed=37, n_bias=9)
    n = b.bias_ids.size
    for bad in ([0, n + 1, n, n], [-1, 9, n, n], [0, 9, 4, n]):
        keep, b.bias_start = b.bias_start, np.array(bad, np.int32)
        out, st = b.call()
        assert st == B.DSPARK_EINVAL
        b.bias_start = keep
        good, st = b.call()
        assert st == B.DSPARK_OK
        for r in range(3):
            rows = slice(int(b.cu[r]), int(b.cu[r + 1]))
            if bad[r:r + 2] == keep[r:r + 2].tolist():
                assert torch.equal(out[rows], good[rows])


def test_rules_empty_bias_lists():
    """A batch whose requests have no biases right now: lists that are there and empty."""
    b = Batch([3, 2, 4], 512, torch.bfloat16, seed=39, n_bias=9)
    none, st = b.call(bias_start=None, bias_ids=None, bias_vals=None)
    assert st == B.DSPARK_OK
    out, st = b.call(bias_start=_dev([0, 0, 0, 0], torch.int32), bias_ids=torch.empty(0, dtype=torch.int32, device="cuda"),
                     bias_vals=torch.empty(0, device="cuda"))
    assert st == B.DSPARK_OK and torch.equal(out, none)


# ------------------------------------------------------------------------------ history

@pytest.mark.parametrize("V", [8, 2048, 5000, 16392])
def test_history(V):
    rng = np.random.default_rng(V)
    lists = [rng.integers(0, V, n) for n in (0, 1, 700, 9000, 33)]
    n_prompt = np.array([0, 1, 300, 5, 0], np.int32)
    start = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    hist = torch.full((5, V), 1234, dtype=torch.int16, device="cuda")
    ws = _ws()
    B.dspark_history_build(_dev(np.concatenate(lists).astype(np.int32)), _dev(start), _dev(n_prompt), hist, ws)
    want = np.stack([R.history_words(x[:m], x[m:], V) for x, m in zip(lists, n_prompt)])
    assert np.array_equal(hist.cpu().numpy(), want)
    out = np.full((5, 9), -1, np.int32)
    for r in range(5):
        out[r, :r * 2] = rng.integers(0, min(V, 5), r * 2)  # the same tokens again and again
    B.dspark_history_commit(_dev(out), hist, ws)
    both = np.stack([R.history_words(x[:m], np.concatenate([x[m:], o[o >= 0]]), V)
                     for x, m, o in zip(lists, n_prompt, out)])
    assert np.array_equal(hist.cpu().numpy(), both)
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK


def test_history_saturates():
    V = 16
    said = np.concatenate([np.full(70000, 3), np.full(32766, 4), [5]]).astype(np.int32)
    hist = torch.zeros(1, V, dtype=torch.int16, device="cuda")
    ws = _ws()
    B.dspark_history_build(_dev(said), _dev([0, said.size], torch.int32), _dev([0], torch.int32), hist, ws)
    assert hist[0, 3:6].tolist() == [32767, 32766, 1]
    B.dspark_history_commit(_dev([[3, 4, 4, 4, 5, 2, -1]], torch.int32), hist, ws)
    assert hist[0, :7].tolist() == [0, 0, 1, 32767, 32767, 2, 0]
    # a full count beside a prompt flag: neither spills into the other, nor into the word's other half
    hist[0, 2:4] = torch.tensor([-1, -1], dtype=torch.int16)
    B.dspark_history_commit(_dev([[2, 3]], torch.int32), hist, ws)
    assert hist[0, 1:5].tolist() == [0, -1, -1, 32767]
    assert B.dspark_read_device_status(ws) == B.DSPARK_OK


def test_history_device_errors():
    V = 24
    hist = torch.zeros(2, V, dtype=torch.int16, device="cuda")
    ws = _ws()
    B.dspark_history_build(_dev([1, V, -1, 2, 2], torch.int32), _dev([0, 3, 5], torch.int32), _dev([0, 0], torch.int32),
                           hist, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_EINVAL
    assert hist[0].tolist() == [0, 1] + [0] * 22 and hist[1].tolist() == [0, 0, 2] + [0] * 21
    for bad in ([0, 3, 6], [0, 4, 3], [-1, 3, 5]):
        B.dspark_history_build(_dev([1, 1, 1, 2, 2], torch.int32), _dev(bad, torch.int32), _dev([0, 0], torch.int32),
                               hist, ws)
        assert B.dspark_read_device_status(ws) == B.DSPARK_EINVAL
    hist.zero_()
    B.dspark_history_commit(_dev([[0, V, -1], [-2, 1, -1]], torch.int32), hist, ws)
    assert B.dspark_read_device_status(ws) == B.DSPARK_EINVAL
    assert hist[0].tolist() == [1] + [0] * 23 and hist[1].tolist() == [0, 1] + [0] * 22
