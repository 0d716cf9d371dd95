"""Refusals of the target-side entry points: every bad argument is caught on the host, nothing is
launched (these run without a GPU; pointers are host buffers that no call may touch)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_markov_gb300 import binding as B  # noqa: E402
from speculative_decoding_draft_markov_gb300 import build as _build  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return B.lib()


_buf = ctypes.create_string_buffer(1 << 16)
PTR = (ctypes.addressof(_buf) + 4095) // 4096 * 4096  # 4096-byte aligned
OTHER = PTR + 8192
OK, EINVAL, EUNSUP, EWS = B.DSPARK_OK, B.DSPARK_EINVAL, B.DSPARK_EUNSUPPORTED, B.DSPARK_EWORKSPACE

APPEND = dict(q=PTR, q_stride=1024, k=PTR, k_stride=256, v=PTR, v_stride=256, dtype=B.DSPARK_BF16, cu=PTR, ctx=PTR, bs=2,
              rows=5, cos_sin=PTR, max_pos=100, rot=128, interleaved=0, table=PTR, max_pages=4, n_pages=9, page_size=16,
              Hq=8, Hkv=2, D=128, q_out=OTHER, k_cache=PTR, v_cache=PTR, ws=PTR, ws_bytes=256, stream=None)
ATTEND = dict(q=PTR, q_stride=1024, dtype=B.DSPARK_BF16, k_cache=PTR, v_cache=PTR, table=PTR, max_pages=4, n_pages=9,
              page_size=16, cu=PTR, ctx=PTR, bs=2, rows=5, max_rows=3, Hq=8, Hkv=2, D=128, scale=0.1, window=0, n_sink=0,
              out=PTR, lse=None, ws=PTR, ws_bytes=1 << 40, stream=None)
RULES = dict(logits=PTR, dtype=B.DSPARK_BF16, rows=5, V=64, cu=PTR, ids=PTR, bs=2, hist=PTR, repetition=PTR, frequency=PTR,
             presence=PTR, bias_start=PTR, bias_ids=PTR, bias_vals=PTR, n_bias=9, mask=PTR, out=OTHER, ws=PTR, ws_bytes=256,
             stream=None)
BUILD = dict(tokens=PTR, n_tokens=9, start=PTR, n_prompt=PTR, bs=2, V=64, hist=PTR, ws=PTR, ws_bytes=256, stream=None)
COMMIT = dict(out_tokens=PTR, bs=2, gamma=7, V=64, hist=PTR, ws=PTR, ws_bytes=256, stream=None)

CACHE = [("bs", 0, EINVAL), ("bs", 257, EUNSUP), ("rows", 0, EINVAL), ("max_pages", 0, EINVAL), ("n_pages", 0, EINVAL),
         ("page_size", 0, EINVAL), ("page_size", 4, EUNSUP), ("page_size", 24, EUNSUP), ("page_size", 8192, EUNSUP),
         ("dtype", B.DSPARK_F32, EUNSUP), ("dtype", 7, EINVAL), ("Hkv", 0, EINVAL), ("Hkv", 3, EINVAL), ("Hq", 0, EINVAL),
         ("D", 96, EUNSUP), ("cu", None, EINVAL), ("ctx", None, EINVAL), ("table", None, EINVAL), ("k_cache", None, EINVAL),
         ("v_cache", None, EINVAL), ("k_cache", PTR + 8, EINVAL), ("cu", PTR + 2, EINVAL), ("q", PTR + 2, EINVAL),
         ("q_stride", 1023, EINVAL), ("q_stride", 1028, EINVAL), ("ws", None, EWS), ("ws", PTR + 16, EWS),
         ("ws_bytes", 255, EWS)]


def _try(lib, name, args, over):
    return getattr(lib, name)(*dict(args, **over).values())


@pytest.mark.parametrize("key,val,want", CACHE + [
    ("k", None, EINVAL), ("v", None, EINVAL), ("k_stride", 250, EINVAL), ("v_stride", 12, EINVAL), ("q_out", None, EINVAL),
    ("q", None, EINVAL), ("q_out", PTR + 8, EINVAL), ("rot", 8, EINVAL), ("rot", 24, EINVAL), ("rot", 144, EINVAL),
    ("cos_sin", None, EINVAL), ("cos_sin", PTR + 4, EINVAL), ("max_pos", 0, EINVAL)])
def test_append_refuses(lib, key, val, want):
    assert _try(lib, "dspark_append_kv", APPEND, {key: val}) == want


def test_append_refuses_strided_in_place(lib):
    assert _try(lib, "dspark_append_kv", APPEND, {"q_out": PTR, "q_stride": 1536}) == EINVAL


@pytest.mark.parametrize("key,val,want", CACHE + [
    ("q", None, EINVAL), ("out", None, EINVAL), ("out", PTR + 8, EINVAL), ("lse", PTR + 2, EINVAL), ("scale", float("inf"), EINVAL),
    ("scale", float("nan"), EINVAL), ("window", -1, EINVAL), ("n_sink", -1, EINVAL), ("max_rows", 0, EINVAL)])
def test_attention_refuses(lib, key, val, want):
    assert _try(lib, "dspark_window_attention", ATTEND, {key: val}) == want


def test_attention_workspace_bytes(lib):
    n = B.dspark_window_attention_workspace_bytes(8, 2, 128)
    assert n >= 256
    assert _try(lib, "dspark_window_attention", ATTEND, {"ws_bytes": n - 1}) == EWS
    for bad in ((8, 3, 128), (0, 1, 128), (8, 2, 96), (256, 1, 64)):
        assert B.dspark_window_attention_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("key,val,want", [
    ("logits", None, EINVAL), ("out", None, EINVAL), ("cu", None, EINVAL), ("ids", None, EINVAL), ("rows", 0, EINVAL),
    ("dtype", 5, EINVAL), ("V", 60, EINVAL), ("V", 0, EINVAL), ("V", 1 << 24, EUNSUP), ("bs", 0, EINVAL), ("bs", 257, EUNSUP),
    ("hist", None, EINVAL), ("hist", PTR + 2, EINVAL), ("bias_ids", None, EINVAL), ("bias_start", None, EINVAL),
    ("bias_vals", None, EINVAL), ("n_bias", -1, EINVAL), ("bias_ids", PTR + 2, EINVAL), ("logits", PTR + 2, EINVAL), ("out", PTR + 2, EINVAL), ("mask", PTR + 1, EINVAL),
    ("ws", None, EWS), ("ws_bytes", 8, EWS)])
def test_rules_refuse(lib, key, val, want):
    assert _try(lib, "dspark_process_logits", RULES, {key: val}) == want


@pytest.mark.parametrize("key,val,want", [
    ("tokens", None, EINVAL), ("n_tokens", -1, EINVAL), ("start", None, EINVAL), ("n_prompt", None, EINVAL),
    ("hist", None, EINVAL), ("hist", PTR + 2, EINVAL), ("V", 12, EINVAL), ("V", 1 << 24, EUNSUP), ("bs", 257, EUNSUP),
    ("ws", None, EWS)])
def test_history_build_refuses(lib, key, val, want):
    assert _try(lib, "dspark_history_build", BUILD, {key: val}) == want


@pytest.mark.parametrize("key,val,want", [
    ("out_tokens", None, EINVAL), ("hist", None, EINVAL), ("gamma", 0, EINVAL), ("gamma", 17, EUNSUP), ("V", 12, EINVAL),
    ("bs", 0, EINVAL), ("ws", None, EWS)])
def test_history_commit_refuses(lib, key, val, want):
    assert _try(lib, "dspark_history_commit", COMMIT, {key: val}) == want


def test_binding_refuses():
    """The binding checks what the C ABI cannot see: types and shapes (CPU tensors: no call gets that far)."""
    i32, bf = torch.int32, torch.bfloat16
    k = torch.zeros(4, 2, 16, 64, dtype=bf)
    q = torch.zeros(3, 4, 64, dtype=bf)
    cu, ctx, table = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 5, dtype=i32)
    out, ws = torch.zeros_like(q), torch.zeros(256, dtype=torch.uint8)
    call = lambda **o: B.dspark_window_attention(**{**dict(  # noqa: E731
        q=q, k_cache=k, v_cache=k, page_table=table, cu_seqlens=cu, ctx_len=ctx, max_rows=3, scale=1.0, window=0, n_sink=0,
        out=out, lse=None, ws=ws), **o})
    for bad in (dict(cu_seqlens=cu.long()), dict(ctx_len=ctx.long()), dict(q=q.float()), dict(out=out[:2]),
                dict(v_cache=k[:3]), dict(page_table=table[:1]), dict(ctx_len=ctx[:1]), dict(lse=torch.zeros(3, 4, dtype=bf)),
                dict(lse=torch.zeros(3, 5)), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**bad)
    hist, toks = torch.zeros(2, 64, dtype=torch.int16), torch.zeros(2, 8, dtype=i32)
    for bad in (dict(hist=hist.int()), dict(out_tokens=toks.long()), dict(out_tokens=toks[:1])):
        with pytest.raises(ValueError):
            B.dspark_history_commit(**{**dict(out_tokens=toks, hist=hist, ws=ws), **bad})
    x = torch.zeros(3, 64)
    for bad in (dict(out=x[:2]), dict(out=x.to(bf)), dict(hist=hist.int()), dict(mask=torch.zeros(3, 3, dtype=i32)),
                dict(ids=cu.long()), dict(repetition=torch.ones(2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            B.dspark_process_logits(**{**dict(
                logits=x, cu_seqlens=cu, ids=cu, hist=hist, repetition=None, frequency=None, presence=None, bias_start=None,
                bias_ids=None, bias_vals=None, mask=None, out=x, ws=ws), **bad})
