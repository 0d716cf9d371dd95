"""Verification of target rows that a grammar mask has emptied almost, or wholly: ids of -inf."""
import numpy as np
import pytest

from oracle import dspark_oracle as O
from speculative_decoding_draft_markov_gb300 import binding as B
from speculative_decoding_draft_markov_gb300 import inputs as I
from speculative_decoding_draft_markov_gb300 import step as S
from tests.parity import compare_verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _draft(wl):
    host = I.make_host_inputs(wl, with_hidden=False)
    inp = S.device_inputs_from_host(host)
    buf = S.StepBuffers.allocate(wl.bs, wl.gamma, wl.V, wl.bs * (wl.gamma + 1), inp["U"].dtype)
    B.dspark_draft_block(inp["U"], inp["W1"], inp["W2t"], inp["anchor"], 1.0, wl.seed, 0, buf.tokens, buf.logit_x,
                         buf.lse, buf.ws)
    B.dspark_pack(None, inp["anchor"], buf.tokens, None, buf.cu, buf.ids, buf.req, buf.pos, buf.padded, buf.ws)
    S.gather_target_forward(inp["target"])(buf)
    return host, inp, buf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share", [0.01, 0.4])
def test_verify_of_masked_rows(dtype, share):
    """Few ids allowed (whole threads of the row pass see nothing but -inf) and many; the drafted tokens are
    allowed in most rows, so that some windows go on and some end at a masked token."""
    base = I.WORKLOADS["qwen3_4b" if dtype == "bf16" else "tiny_fp32"]
    wl = base.with_(name="masked", bs=24, gamma=3, V=20000, d=64, seed=51, sigmas=(0.5,))
    host, inp, buf = _draft(wl)
    bs, gamma, V = wl.bs, wl.gamma, wl.V
    rng = np.random.default_rng(52)
    rows = bs * (gamma + 1)
    allowed = rng.random((rows, V)) < share
    tok = buf.tokens.cpu().numpy()
    for r in range(bs):
        for k in range(gamma):
            allowed[r * (gamma + 1) + k, tok[r, k]] = rng.random() < 0.8
    words = np.zeros((rows, (V + 31) // 32 * 32), bool)
    words[:, :V] = allowed
    mask = torch.from_numpy(np.packbits(words, axis=1, bitorder="little").view(np.int32)).cuda()
    B.dspark_process_logits(buf.packed, buf.cu, buf.ids, None, None, None, None, None, None, None, mask, buf.packed, buf.ws)
    S.verify(inp, buf, 1.0, wl.seed, 0, B.DSPARK_STATIC)
    assert B.dspark_read_device_status(buf.ws) == B.DSPARK_OK
    cu, ids, req, pos, padded = O.pack(None, host["anchor"], tok, [], rows)
    packed = buf.packed.cpu()
    packed = packed.view(torch.int16).numpy().view(np.uint16) if dtype == "bf16" else packed.numpy()
    out_o, acc_o, _, mv_o = O.verify(packed, cu, None, O.STATIC, host["anchor"], tok, buf.logit_x.cpu().numpy(),
                                     buf.lse.cpu().numpy(), host["U"], host["W1"], host["W2t"], 1.0, wl.seed, 0,
                                     dtype=dtype)
    out, acc = buf.out_tokens.cpu().numpy(), buf.acc_len.cpu().numpy()
    checked, near = compare_verify(out, acc, out_o, acc_o, mv_o)
    assert near <= 1 and checked >= bs - 1
    for r in range(bs):  # nothing that the mask hides is ever given out
        for k in range(acc[r] + 1):
            assert allowed[r * (gamma + 1) + k, out[r, k]]
    S.verify(inp, buf, 0.0, wl.seed, 0, B.DSPARK_STATIC)
    out, acc = buf.out_tokens.cpu().numpy(), buf.acc_len.cpu().numpy()
    best = buf.packed.float().argmax(1).cpu().numpy().reshape(bs, gamma + 1)
    for r in range(bs):
        assert out[r, acc[r]] == best[r, acc[r]] and np.array_equal(out[r, :acc[r]], best[r, :acc[r]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_verify_of_a_row_that_allows_nothing(dtype, temperature):
    base = I.WORKLOADS["qwen3_4b" if dtype == "bf16" else "tiny_fp32"]
    wl = base.with_(name="nothing", bs=3, gamma=2, V=3000, d=64, seed=53, sigmas=(0.5,))
    _, inp, buf = _draft(wl)
    g1 = wl.gamma + 1
    buf.packed[g1:2 * g1] = float("-inf")  # request 1: nothing is allowed anywhere
    S.verify(inp, buf, temperature, wl.seed, 0, B.DSPARK_STATIC)
    assert B.dspark_read_device_status(buf.ws) == B.DSPARK_OK
    out, acc = buf.out_tokens.cpu().numpy(), buf.acc_len.cpu().numpy()
    assert acc[1] == 0 and (out[1] == -1).all()
    for r in (0, 2):
        assert 0 <= out[r, acc[r]] < wl.V
