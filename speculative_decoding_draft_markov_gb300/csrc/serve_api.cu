// C ABI of the target model's side of a step (paged caches, attention, logit rules, token history, log probabilities):
// host-side argument checks and launches.  Nothing here allocates memory.
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

using namespace dspark;

namespace {

inline bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA; }

inline int check_status_ws(const void* ws, size_t ws_bytes, size_t need = 256) {
  return !ws || !al(ws, 256) || ws_bytes < need ? DSPARK_EWORKSPACE : DSPARK_OK;
}

inline int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

int check_heads(int Hq, int Hkv, int D) {
  if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return DSPARK_EINVAL;
  return (D != 64 && D != 128) || Hq / Hkv > 128 || Hq > 65535 ? DSPARK_EUNSUPPORTED : DSPARK_OK;
}

// The paged cache and the packed rows, as both cache calls take them.
int check_cache(int dtype, const int32_t* cu, const int32_t* ctx, int bs, int rows, const int32_t* page_table,
                int max_pages, int n_pages, int page_size, const void* k_cache, const void* v_cache) {
  if (!cu || !ctx || !page_table || !k_cache || !v_cache) return DSPARK_EINVAL;
  if (bs < 1 || rows < 1 || max_pages < 1 || n_pages < 1 || page_size < 1) return DSPARK_EINVAL;
  if (dtype == DSPARK_F32) return DSPARK_EUNSUPPORTED;
  if (dtype != DSPARK_BF16) return DSPARK_EINVAL;
  if (bs > DSPARK_MAX_BS || page_size < 8 || page_size > 4096 || (page_size & (page_size - 1)))
    return DSPARK_EUNSUPPORTED;
  if (!al(k_cache, 16) || !al(v_cache, 16) || !al(cu, 4) || !al(ctx, 4) || !al(page_table, 4)) return DSPARK_EINVAL;
  return DSPARK_OK;
}

bool bad_rows(const void* p, int64_t stride, int width) {
  return !p || !al(p, 16) || stride < width || stride % 8 != 0;
}

}  // namespace

extern "C" {

int dspark_append_kv(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, int dtype, const int32_t* cu_seqlens, const int32_t* ctx_len, int bs, int rows,
                     const float* cos_sin, int max_pos, int rot, int interleaved, const int32_t* page_table,
                     int max_pages, int n_pages, int page_size, int Hq, int Hkv, int D, void* q_out, void* k_cache,
                     void* v_cache, void* ws, size_t ws_bytes, dspark_stream_t stream) {
  if (int e = check_cache(dtype, cu_seqlens, ctx_len, bs, rows, page_table, max_pages, n_pages, page_size, k_cache,
                          v_cache))
    return e;
  if (int e = check_heads(Hq, Hkv, D)) return e;
  if ((q == nullptr) != (q_out == nullptr)) return DSPARK_EINVAL;
  if (q && (bad_rows(q, q_stride, Hq * D) || !al(q_out, 16) || (q == q_out && q_stride != int64_t(Hq) * D)))
    return DSPARK_EINVAL;
  if (bad_rows(k, k_stride, Hkv * D) || bad_rows(v, v_stride, Hkv * D)) return DSPARK_EINVAL;
  if (!cos_sin || !al(cos_sin, 16) || max_pos < 1 || rot < 16 || rot > D || rot % 16 != 0) return DSPARK_EINVAL;
  if (int e = check_status_ws(ws, ws_bytes)) return e;
  return cuda_status(launch_append_kv(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, ctx_len, bs, rows, cos_sin,
                                      max_pos, rot, interleaved, page_table, max_pages, n_pages, log2_of(page_size),
                                      Hq, Hkv, D, q_out, k_cache, v_cache, static_cast<uint32_t*>(ws),
                                      reinterpret_cast<cudaStream_t>(stream)));
}

size_t dspark_window_attention_workspace_bytes(int Hq, int Hkv, int D) {
  return check_heads(Hq, Hkv, D) ? 0 : window_attention_ws_bytes(Hq, Hkv, D);
}

int dspark_window_attention(const void* q, int64_t q_stride, int dtype, const void* k_cache, const void* v_cache,
                            const int32_t* page_table, int max_pages, int n_pages, int page_size,
                            const int32_t* cu_seqlens, const int32_t* ctx_len, int bs, int rows, int max_rows, int Hq,
                            int Hkv, int D, float scale, int window, int n_sink, void* out, float* lse, void* ws,
                            size_t ws_bytes, dspark_stream_t stream) {
  if (int e = check_cache(dtype, cu_seqlens, ctx_len, bs, rows, page_table, max_pages, n_pages, page_size, k_cache,
                          v_cache))
    return e;
  if (int e = check_heads(Hq, Hkv, D)) return e;
  if (bad_rows(q, q_stride, Hq * D) || !out || !al(out, 16) || !al(lse, 4)) return DSPARK_EINVAL;
  if (q == out && q_stride != int64_t(Hq) * D) return DSPARK_EINVAL;  // other rows' queries would be overwritten
  if (!std::isfinite(scale) || window < 0 || n_sink < 0 || max_rows < 1) return DSPARK_EINVAL;
  if (int e = check_status_ws(ws, ws_bytes, window_attention_ws_bytes(Hq, Hkv, D))) return e;
  return cuda_status(launch_window_attention(q, q_stride, k_cache, v_cache, page_table, max_pages, n_pages,
                                             log2_of(page_size), cu_seqlens, ctx_len, bs, rows, max_rows, Hq, Hkv, D,
                                             scale, window, n_sink, out, lse, ws,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

static int check_vocab(int bs, int V) {
  if (bs < 1 || V < 8 || V % 8 != 0) return DSPARK_EINVAL;
  return bs > DSPARK_MAX_BS || V >= (1 << 24) ? DSPARK_EUNSUPPORTED : DSPARK_OK;
}

int dspark_process_logits(const void* logits, int dtype, int rows, int V, const int32_t* cu_seqlens,
                          const int32_t* ids, int bs, const int16_t* hist, const float* repetition,
                          const float* frequency, const float* presence, const int32_t* bias_start,
                          const int32_t* bias_ids, const float* bias_vals, int n_bias, const uint32_t* mask, void* out,
                          void* ws, size_t ws_bytes, dspark_stream_t stream) {
  if (!logits || !out || !cu_seqlens || !ids || rows < 1) return DSPARK_EINVAL;
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_EINVAL;
  if (int e = check_vocab(bs, V)) return e;
  if (!al(logits, 16) || !al(out, 16) || !al(hist, 16) || !al(mask, 4)) return DSPARK_EINVAL;
  if (!hist && (repetition || frequency || presence)) return DSPARK_EINVAL;  // penalties of what?
  if (!bias_start && (bias_ids || bias_vals)) return DSPARK_EINVAL;
  if (bias_start && n_bias != 0 && (!bias_ids || !bias_vals)) return DSPARK_EINVAL;
  if (n_bias < 0 || !al(bias_start, 4) || !al(bias_ids, 4) || !al(bias_vals, 4)) return DSPARK_EINVAL;
  if (!al(cu_seqlens, 4) || !al(ids, 4) || !al(repetition, 4) || !al(frequency, 4) || !al(presence, 4)) return DSPARK_EINVAL;
  if (int e = check_status_ws(ws, ws_bytes)) return e;
  return cuda_status(launch_process_logits(logits, dtype, rows, V, cu_seqlens, ids, bs, hist, repetition, frequency,
                                           presence, bias_start, bias_ids, bias_vals, n_bias, mask, out,
                                           static_cast<uint32_t*>(ws), reinterpret_cast<cudaStream_t>(stream)));
}

int dspark_history_build(const int32_t* tokens, int n_tokens, const int32_t* start, const int32_t* n_prompt, int bs,
                         int V, int16_t* hist, void* ws, size_t ws_bytes, dspark_stream_t stream) {
  if ((!tokens && n_tokens > 0) || n_tokens < 0 || !start || !n_prompt || !hist || !al(hist, 16)) return DSPARK_EINVAL;
  if (!al(tokens, 4) || !al(start, 4) || !al(n_prompt, 4)) return DSPARK_EINVAL;
  if (int e = check_vocab(bs, V)) return e;
  if (int e = check_status_ws(ws, ws_bytes)) return e;
  return cuda_status(launch_history_build(tokens, n_tokens, start, n_prompt, bs, V, hist, static_cast<uint32_t*>(ws),
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int dspark_history_commit(const int32_t* out_tokens, int bs, int gamma, int V, int16_t* hist, void* ws,
                          size_t ws_bytes, dspark_stream_t stream) {
  if (!out_tokens || !al(out_tokens, 4) || !hist || !al(hist, 16) || gamma < 1) return DSPARK_EINVAL;
  if (int e = check_vocab(bs, V)) return e;
  if (gamma > DSPARK_MAX_GAMMA) return DSPARK_EUNSUPPORTED;
  if (int e = check_status_ws(ws, ws_bytes)) return e;
  return cuda_status(launch_history_commit(out_tokens, bs, gamma, V, hist, static_cast<uint32_t*>(ws),
                                           reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------- the 8-bit cache, log probabilities

int dspark_append_kv8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      int dtype, const int32_t* cu_seqlens, const int32_t* ctx_len, int bs, int rows, const float* cos_sin,
                      int max_pos, int rot, int interleaved, const int32_t* page_table, int max_pages, int n_pages,
                      int page_size, int Hq, int Hkv, int D, void* q_out, void* k_cache, void* v_cache, uint8_t* kv_scale,
                      void* ws, size_t ws_bytes, dspark_stream_t stream) {
  if (int e = check_cache(dtype, cu_seqlens, ctx_len, bs, rows, page_table, max_pages, n_pages, page_size, k_cache,
                          v_cache))
    return e;
  if (int e = check_heads(Hq, Hkv, D)) return e;
  if (!kv_scale || !al(kv_scale, 16)) return DSPARK_EINVAL;
  if ((q == nullptr) != (q_out == nullptr)) return DSPARK_EINVAL;
  if (q && (bad_rows(q, q_stride, Hq * D) || !al(q_out, 16) || (q == q_out && q_stride != int64_t(Hq) * D)))
    return DSPARK_EINVAL;
  if (bad_rows(k, k_stride, Hkv * D) || bad_rows(v, v_stride, Hkv * D)) return DSPARK_EINVAL;
  if (!cos_sin || !al(cos_sin, 16) || max_pos < 1 || rot < 16 || rot > D || rot % 16 != 0) return DSPARK_EINVAL;
  if (int e = check_status_ws(ws, ws_bytes)) return e;
  return cuda_status(launch_append_kv8(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, ctx_len, bs, rows, cos_sin,
                                       max_pos, rot, interleaved, page_table, max_pages, n_pages, log2_of(page_size), Hq,
                                       Hkv, D, q_out, k_cache, v_cache, kv_scale, static_cast<uint32_t*>(ws),
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int dspark_read_kv8(const void* k_cache, const void* v_cache, const uint8_t* kv_scale, int dtype,
                    const int32_t* page_table, int max_pages, int n_pages, int page_size, const int32_t* cu_seqlens,
                    const int32_t* ctx_len, int bs, int rows, int Hkv, int D, int window, int n_sink,
                    const int32_t* out_table, int n_out_pages, void* k_out, void* v_out, void* ws, size_t ws_bytes,
                    dspark_stream_t stream) {
  if (int e = check_cache(dtype, cu_seqlens, ctx_len, bs, rows, page_table, max_pages, n_pages, page_size, k_cache,
                          v_cache))
    return e;
  if (int e = check_heads(Hkv, Hkv, D)) return e;
  if (!kv_scale || !al(kv_scale, 16) || !out_table || !al(out_table, 4) || n_out_pages < 1) return DSPARK_EINVAL;
  if (!k_out || !v_out || !al(k_out, 16) || !al(v_out, 16) || k_out == v_out) return DSPARK_EINVAL;
  if (window < 0 || n_sink < 0) return DSPARK_EINVAL;
  if (int e = check_status_ws(ws, ws_bytes)) return e;
  return cuda_status(launch_read_kv8(k_cache, v_cache, kv_scale, page_table, max_pages, n_pages, log2_of(page_size),
                                     cu_seqlens, ctx_len, bs, rows, Hkv, D, window, n_sink, out_table, n_out_pages, k_out,
                                     v_out, false, static_cast<uint32_t*>(ws), reinterpret_cast<cudaStream_t>(stream)));
}

int dspark_window_attention_kv8(const void* q, int64_t q_stride, int dtype, const void* k_cache, const void* v_cache,
                                const uint8_t* kv_scale, const int32_t* page_table, int max_pages, int n_pages,
                                int page_size, const int32_t* cu_seqlens, const int32_t* ctx_len, int bs, int rows,
                                int max_rows, int Hq, int Hkv, int D, float scale, int window, int n_sink, void* out,
                                float* lse, void* k_scratch, void* v_scratch, void* ws, size_t ws_bytes,
                                dspark_stream_t stream) {
  if (int e = check_cache(dtype, cu_seqlens, ctx_len, bs, rows, page_table, max_pages, n_pages, page_size, k_cache,
                          v_cache))
    return e;
  if (int e = check_heads(Hq, Hkv, D)) return e;
  if (!kv_scale || !al(kv_scale, 16)) return DSPARK_EINVAL;
  if (bad_rows(q, q_stride, Hq * D) || !out || !al(out, 16) || !al(lse, 4)) return DSPARK_EINVAL;
  if (q == out && q_stride != int64_t(Hq) * D) return DSPARK_EINVAL;  // other rows' queries would be overwritten
  if ((k_scratch == nullptr) != (v_scratch == nullptr) || !al(k_scratch, 16) || !al(v_scratch, 16)) return DSPARK_EINVAL;
  if (k_scratch && k_scratch == v_scratch) return DSPARK_EINVAL;
  if (!std::isfinite(scale) || window < 0 || n_sink < 0 || max_rows < 1) return DSPARK_EINVAL;
  if (int e = check_status_ws(ws, ws_bytes, window_attention_ws_bytes(Hq, Hkv, D))) return e;
  return cuda_status(launch_window_attention_kv8(q, q_stride, k_cache, v_cache, kv_scale, page_table, max_pages, n_pages,
                                                 log2_of(page_size), cu_seqlens, ctx_len, bs, rows, max_rows, Hq, Hkv, D,
                                                 scale, window, n_sink, out, lse, k_scratch, v_scratch, ws,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

static int check_items(int items, int V, int top_n) {
  if (items < 1 || V < 8 || V % 8 != 0 || top_n < 0) return DSPARK_EINVAL;
  return items > (1 << 20) || V >= (1 << 24) || top_n > DSPARK_MAX_TOP ? DSPARK_EUNSUPPORTED : DSPARK_OK;
}

size_t dspark_token_logprobs_workspace_bytes(int items, int V, int top_n) {
  return check_items(items, V, top_n) ? 0 : token_logprobs_ws_bytes(items, V, top_n);
}

int dspark_token_logprobs(const void* logits, int dtype, int rows, int V, const int32_t* cu_seqlens, int n, int per,
                          const int32_t* tokens, float temperature, float* logprob, float* entropy, int32_t* rank,
                          int32_t* top_ids, float* top_logprobs, int top_n, void* ws, size_t ws_bytes,
                          dspark_stream_t stream) {
  if (!logits || !tokens || !logprob || rows < 1 || n < 1 || per < 1) return DSPARK_EINVAL;
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_EINVAL;
  if (int64_t(n) * per > INT32_MAX) return DSPARK_EUNSUPPORTED;
  if (int e = check_items(n * per, V, top_n)) return e;
  if (!cu_seqlens && n * per > rows) return DSPARK_EINVAL;
  if (!al(logits, 16) || !al(cu_seqlens, 4) || !al(tokens, 4) || !al(logprob, 4) || !al(entropy, 4) || !al(rank, 4) ||
      !al(top_ids, 4) || !al(top_logprobs, 4))
    return DSPARK_EINVAL;
  if (top_n > 0 ? !top_ids || !top_logprobs : top_ids || top_logprobs) return DSPARK_EINVAL;
  if (!std::isfinite(temperature) || !(temperature > 0.f) || !std::isfinite(2.f / temperature)) return DSPARK_EINVAL;
  if (int e = check_status_ws(ws, ws_bytes, token_logprobs_ws_bytes(n * per, V, top_n))) return e;
  return cuda_status(launch_token_logprobs(logits, dtype, rows, V, cu_seqlens, n, tokens, per, temperature, logprob,
                                           entropy, rank, top_ids, top_logprobs, top_n, ws,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
