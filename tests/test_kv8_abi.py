"""Refusals of the 8-bit cache's entry points and of the log probabilities: every bad argument is caught on the host, nothing
is launched (these run without a GPU; pointers are host buffers that no call may touch)."""
import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from tests.test_serving_abi import CACHE, EINVAL, EUNSUP, EWS, OTHER, PTR, _try, lib  # noqa: E402,F401

F8 = torch.float8_e4m3fn
APPEND = dict(q=PTR, q_stride=1024, k=PTR, k_stride=256, v=PTR, v_stride=256, dtype=B.DSPARK_BF16, cu=PTR, ctx=PTR, bs=2,
              rows=5, cos_sin=PTR, max_pos=100, rot=128, interleaved=0, table=PTR, max_pages=4, n_pages=9, page_size=16,
              Hq=8, Hkv=2, D=128, q_out=OTHER, k_cache=PTR, v_cache=PTR, kv_scale=PTR, ws=PTR, ws_bytes=256, stream=None)
READ = dict(k_cache=PTR, v_cache=PTR, kv_scale=PTR, dtype=B.DSPARK_BF16, table=PTR, max_pages=4, n_pages=9, page_size=16,
            cu=PTR, ctx=PTR, bs=2, rows=5, Hkv=2, D=128, window=0, n_sink=0, out_table=PTR, n_out_pages=9, k_out=PTR,
            v_out=OTHER, ws=PTR, ws_bytes=256, stream=None)
ATTEND = dict(q=PTR, q_stride=1024, dtype=B.DSPARK_BF16, k_cache=PTR, v_cache=PTR, kv_scale=PTR, table=PTR, max_pages=4,
              n_pages=9, page_size=16, cu=PTR, ctx=PTR, bs=2, rows=5, max_rows=3, Hq=8, Hkv=2, D=128, scale=0.1, window=0,
              n_sink=0, out=PTR, lse=None, k_scratch=PTR, v_scratch=OTHER, ws=PTR, ws_bytes=1 << 40, stream=None)
LOGPROBS = dict(logits=PTR, dtype=B.DSPARK_BF16, rows=16, V=64, cu=PTR, n=2, per=8, tokens=PTR, temperature=1.0, logprob=PTR,
                entropy=PTR, rank=PTR, top_ids=PTR, top_logprobs=PTR, top_n=5, ws=PTR, ws_bytes=1 << 40, stream=None)
SCALE = [("kv_scale", None, EINVAL), ("kv_scale", PTR + 1, EINVAL)]


@pytest.mark.parametrize("key,val,want", CACHE + SCALE + [
    ("k", None, EINVAL), ("v", None, EINVAL), ("k_stride", 250, EINVAL), ("v_stride", 12, EINVAL), ("q_out", None, EINVAL),
    ("q", None, EINVAL), ("q_out", PTR + 8, EINVAL), ("rot", 8, EINVAL), ("rot", 24, EINVAL), ("rot", 144, EINVAL),
    ("cos_sin", None, EINVAL), ("cos_sin", PTR + 4, EINVAL), ("max_pos", 0, EINVAL)])
def test_append_refuses(lib, key, val, want):  # noqa: F811
    assert _try(lib, "dspark_append_kv8", APPEND, {key: val}) == want


def test_append_refuses_strided_in_place(lib):  # noqa: F811
    assert _try(lib, "dspark_append_kv8", APPEND, {"q_out": PTR, "q_stride": 1536}) == EINVAL


@pytest.mark.parametrize("key,val,want", [c for c in CACHE if c[0] not in ("q", "q_stride", "Hq", "Hkv")] + SCALE + [
    ("Hkv", 0, EINVAL), ("window", -1, EINVAL), ("n_sink", -1, EINVAL), ("out_table", None, EINVAL), ("out_table", PTR + 2, EINVAL),
    ("n_out_pages", 0, EINVAL), ("k_out", None, EINVAL), ("v_out", None, EINVAL), ("k_out", PTR + 8, EINVAL), ("v_out", PTR, EINVAL)])
def test_read_refuses(lib, key, val, want):  # noqa: F811
    assert _try(lib, "dspark_read_kv8", READ, {key: val}) == want


@pytest.mark.parametrize("key,val,want", CACHE + SCALE + [
    ("q", None, EINVAL), ("out", None, EINVAL), ("out", PTR + 8, EINVAL), ("lse", PTR + 2, EINVAL), ("scale", float("inf"), EINVAL),
    ("scale", float("nan"), EINVAL), ("window", -1, EINVAL), ("n_sink", -1, EINVAL), ("max_rows", 0, EINVAL),
    ("k_scratch", None, EINVAL), ("v_scratch", None, EINVAL), ("k_scratch", PTR + 8, EINVAL), ("v_scratch", PTR, EINVAL)])
def test_attention_refuses(lib, key, val, want):  # noqa: F811
    assert _try(lib, "dspark_window_attention_kv8", ATTEND, {key: val}) == want


def test_attention_wants_its_workspace(lib):  # noqa: F811
    n = B.dspark_window_attention_workspace_bytes(8, 2, 128)
    assert _try(lib, "dspark_window_attention_kv8", ATTEND, {"ws_bytes": n - 1}) == EWS


@pytest.mark.parametrize("key,val,want", [
    ("logits", None, EINVAL), ("tokens", None, EINVAL), ("logprob", None, EINVAL), ("rows", 0, EINVAL), ("n", 0, EINVAL),
    ("per", 0, EINVAL), ("dtype", 5, EINVAL), ("V", 60, EINVAL), ("V", 0, EINVAL), ("V", 1 << 24, EUNSUP), ("top_n", -1, EINVAL),
    ("top_n", 33, EUNSUP), ("top_n", 0, EINVAL), ("top_ids", None, EINVAL), ("top_logprobs", None, EINVAL), ("n", 1 << 20, EUNSUP),
    ("n", 2 ** 31 - 1, EUNSUP), ("temperature", 0.0, EINVAL), ("temperature", -1.0, EINVAL), ("temperature", float("nan"), EINVAL),
    ("temperature", float("inf"), EINVAL), ("temperature", 1e-39, EINVAL), ("logits", PTR + 8, EINVAL), ("cu", PTR + 2, EINVAL),
    ("tokens", PTR + 2, EINVAL), ("rank", PTR + 1, EINVAL), ("ws", None, EWS), ("ws", PTR + 16, EWS), ("ws_bytes", 8, EWS)])
def test_logprobs_refuse(lib, key, val, want):  # noqa: F811
    assert _try(lib, "dspark_token_logprobs", LOGPROBS, {key: val}) == want


def test_logprobs_refuse_more_tokens_than_rows(lib):  # noqa: F811
    assert _try(lib, "dspark_token_logprobs", LOGPROBS, {"cu": None, "rows": 15}) == EINVAL


def test_logprobs_workspace_bytes(lib):  # noqa: F811
    assert B.dspark_token_logprobs_workspace_bytes(1, 64, 0) >= 256
    for bad in ((0, 64, 0), (1, 60, 0), (1, 64, 33), (1, 64, -1), (1 << 21, 64, 0), (1, 1 << 24, 0)):
        assert B.dspark_token_logprobs_workspace_bytes(*bad) == 0
        with pytest.raises(ValueError):
            B.alloc_logprobs_workspace(*bad, device="cpu")


def test_binding_refuses(lib):  # noqa: F811
    """The binding checks what the C ABI cannot see: types and shapes (CPU tensors: no call gets that far)."""
    i32, bf = torch.int32, torch.bfloat16
    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(F8)
    sc = torch.zeros(4, 2, 16, 2, dtype=torch.uint8)
    wide = torch.zeros(4, 2, 16, 64, dtype=bf)
    q = torch.zeros(3, 4, 64, dtype=bf)
    cu, ctx, table = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 5, dtype=i32)
    ws = torch.zeros(256, dtype=torch.uint8)
    bad_cache = (dict(k_cache=wide), dict(v_cache=wide), dict(v_cache=k[:3]), dict(kv_scale=sc[..., 0]), dict(kv_scale=sc[:3]),
                 dict(kv_scale=sc.int()), dict(cu_seqlens=cu.long()), dict(ctx_len=ctx[:1]), dict(page_table=table[:1]))
    attend = dict(q=q, k_cache=k, v_cache=k, kv_scale=sc, page_table=table, cu_seqlens=cu, ctx_len=ctx, max_rows=3, scale=1.0,
                  window=0, n_sink=0, out=torch.zeros_like(q), lse=None, k_scratch=None, v_scratch=None, ws=ws)
    for bad in bad_cache + (dict(q=q.float()), dict(out=q[:2]), dict(k_scratch=wide[:3], v_scratch=wide), dict(v_scratch=k),
                            dict(lse=torch.zeros(3, 5))):
        with pytest.raises(ValueError):
            B.dspark_window_attention_kv8(**{**attend, **bad})
    read = dict(k_cache=k, v_cache=k, kv_scale=sc, page_table=table, cu_seqlens=cu, ctx_len=ctx, rows=3, window=0, n_sink=0,
                out_table=table, k_out=wide, v_out=wide, ws=ws)
    for bad in bad_cache + (dict(out_table=table[:, :4]), dict(k_out=k), dict(v_out=wide[:2]), dict(k_out=wide[:, :1], v_out=wide[:, :1]),
                            dict(out_table=table.long())):
        with pytest.raises(ValueError):
            B.dspark_read_kv8(**{**read, **bad})
    kv = torch.zeros(3, 2, 64, dtype=bf)
    append = dict(q=q, k=kv, v=kv, cu_seqlens=cu, ctx_len=ctx, cos_sin=torch.zeros(9, 64), page_table=table, q_out=q, k_cache=k,
                  v_cache=k, kv_scale=sc, ws=ws)
    for bad in bad_cache + (dict(k=kv.float()), dict(v=kv[:2]), dict(q_out=None), dict(cos_sin=torch.zeros(9, 64, dtype=bf))):
        with pytest.raises((ValueError, B.DSparkError)):
            B.dspark_append_kv8(**{**append, **bad})
    x, t = torch.zeros(6, 64), torch.zeros(2, 3, dtype=i32)
    f, top = torch.zeros(2, 3), torch.zeros(2, 3, 4, dtype=i32)
    ask = dict(logits=x, cu_seqlens=cu, tokens=t, temperature=1.0, logprob=f, entropy=f, rank=t, top_ids=top,
               top_logprobs=top.float(), ws=ws)
    for bad in (dict(tokens=t.long()), dict(cu_seqlens=cu[:2]), dict(logprob=None), dict(logprob=f[:1]), dict(entropy=f.double()),
                dict(rank=f), dict(top_ids=top[:1]), dict(top_logprobs=top), dict(top_logprobs=top.float()[..., :3]),
                dict(tokens=t[0])):
        with pytest.raises(ValueError):
            B.dspark_token_logprobs(**{**ask, **bad})
    for call, args in ((B.dspark_window_attention_kv8, attend), (B.dspark_read_kv8, read), (B.dspark_append_kv8, append),
                       (B.dspark_token_logprobs, ask)):
        with pytest.raises(B.DSparkDeviceError):
            call(**args)
