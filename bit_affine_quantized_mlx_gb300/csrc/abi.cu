// C-ABI entry points of liblily_q4: argument validation, workspace sizing and the
// host-only format helpers.  Compute is enqueued by the launchers in the other
// translation units; nothing here allocates device memory.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"

namespace lq4 {

int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev] = n;
  }
  return cached[dev];
}

int check_launch() {
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? LILY_Q4_OK : LILY_Q4_ERR_CUDA;
}

static bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

static bool width_ok(int v) {
  return v == 64 || v == 128 || v == 256 || v == 512 || v == 1024 || v == 2048;
}

static bool mat_ok(const lily_q4_mat &m) {
  return m.w && m.s && m.b && aligned(m.w, 16) && aligned(m.s, 16) && aligned(m.b, 16);
}

// Returns LILY_Q4_OK, INVALID_ARG or UNSUPPORTED.
static int check_layer(const lily_q4_moe_layer *L) {
  if (!L) return LILY_Q4_ERR_INVALID_ARG;
  if (L->hidden <= 0 || L->inter <= 0 || L->n_experts <= 0 || L->top_k <= 0)
    return LILY_Q4_ERR_INVALID_ARG;
  if (L->hidden % LILY_Q4_GROUP || L->inter % LILY_Q4_GROUP) return LILY_Q4_ERR_INVALID_ARG;
  if (L->top_k > L->n_experts) return LILY_Q4_ERR_INVALID_ARG;
  if (L->n_experts > 1024 || L->top_k > 16) return LILY_Q4_ERR_INVALID_ARG;
  if (L->has_shared != 0 && L->has_shared != 1) return LILY_Q4_ERR_INVALID_ARG;
  if (!mat_ok(L->gate) || !mat_ok(L->up) || !mat_ok(L->down)) return LILY_Q4_ERR_INVALID_ARG;
  if (L->shared_bits != 0 && L->shared_bits != 4 && L->shared_bits != 8) return LILY_Q4_ERR_INVALID_ARG;
  if (L->router_bits != 0 && L->router_bits != 16 && L->router_bits != 8) return LILY_Q4_ERR_INVALID_ARG;
  if (L->router_bits == 8) {
    if (!mat_ok(L->router_q8)) return LILY_Q4_ERR_INVALID_ARG;
  } else if (!L->router || !aligned(L->router, 16)) {
    return LILY_Q4_ERR_INVALID_ARG;
  }
  if (L->router_bias && !aligned(L->router_bias, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (L->has_shared) {
    if (!mat_ok(L->sh_gate) || !mat_ok(L->sh_up) || !mat_ok(L->sh_down))
      return LILY_Q4_ERR_INVALID_ARG;
    if (!L->shared_gate || !aligned(L->shared_gate, 16)) return LILY_Q4_ERR_INVALID_ARG;
  }
  if (!width_ok(L->hidden) || !width_ok(L->inter)) return LILY_Q4_ERR_UNSUPPORTED;
  return LILY_Q4_OK;
}

static int check_io(const uint16_t *x, uint16_t *y, int32_t *idx, float *w, void *ws) {
  if (!x || !y || !ws) return LILY_Q4_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  if ((idx && !aligned(idx, 4)) || (w && !aligned(w, 4))) return LILY_Q4_ERR_INVALID_ARG;
  return LILY_Q4_OK;
}

// ---------------------------------------------------------------- attention operators
static bool rows_ok(const Rows &r, int elem_bytes) {
  const int64_t step = 16 / elem_bytes;
  return r.p && aligned(r.p, 16) && r.ts % step == 0 && r.hs % step == 0;
}

static int check_cache(const lily_kv8_cache *C) {
  if (!C || !C->k || !C->v || !C->k_amax || !C->v_amax) return LILY_Q4_ERR_INVALID_ARG;
  if (!aligned(C->k, 16) || !aligned(C->v, 16) || !aligned(C->k_amax, 4) || !aligned(C->v_amax, 4))
    return LILY_Q4_ERR_INVALID_ARG;
  if (C->n_pages <= 0 || C->kv_heads <= 0 || C->kv_heads > 65535) return LILY_Q4_ERR_INVALID_ARG;
  if (C->page != 16 && C->page != 32 && C->page != 64 && C->page != 128) return LILY_Q4_ERR_UNSUPPORTED;
  if (C->head_dim != 64 && C->head_dim != 128 && C->head_dim != 256) return LILY_Q4_ERR_UNSUPPORTED;
  return LILY_Q4_OK;
}

// Bounds only: what sizes a workspace.
static int check_bounds(const lily_kv8_batch *b, int T) {
  if (!b || T < 0 || b->batch < 0 || b->table_pages < 0 || b->max_q < 0 || b->max_kv < 0)
    return LILY_Q4_ERR_INVALID_ARG;
  if (b->batch > kMaxBatch) return LILY_Q4_ERR_UNSUPPORTED;
  if (T > 0 && (b->batch == 0 || b->table_pages == 0 || b->max_q == 0)) return LILY_Q4_ERR_INVALID_ARG;
  return LILY_Q4_OK;
}

static int check_batch(const lily_kv8_batch *b, int T, void *ws, size_t ws_bytes) {
  const int rc = check_bounds(b, T);
  if (rc != LILY_Q4_OK) return rc;
  if (T == 0) return LILY_Q4_OK;
  if (!b->block_table || !b->q_start || !b->kv_len) return LILY_Q4_ERR_INVALID_ARG;
  if (!aligned(b->block_table, 4) || !aligned(b->q_start, 4) || !aligned(b->kv_len, 4))
    return LILY_Q4_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  return ws_bytes < kAlign ? LILY_Q4_ERR_WORKSPACE_TOO_SMALL : LILY_Q4_OK;
}

static int check_attention(const lily_kv8_cache *C, const lily_kv8_batch *b, int T, int q_heads) {
  int rc = check_cache(C);
  if (rc != LILY_Q4_OK) return rc;
  rc = check_bounds(b, T);
  if (rc != LILY_Q4_OK) return rc;
  if (q_heads <= 0 || q_heads % C->kv_heads) return LILY_Q4_ERR_INVALID_ARG;
  if (q_heads / C->kv_heads > 128) return LILY_Q4_ERR_UNSUPPORTED;
  return LILY_Q4_OK;
}

// ---------------------------------------------------------------- around the products of a step
// One row has no stride.
static bool flat_rows_ok(const void *p, int64_t ts, int elem_bytes, int rows) {
  return p && aligned(p, 16) && (rows <= 1 || ts % (16 / elem_bytes) == 0);
}
constexpr int kMaxRows = 1 << 30;  // the kernels count rows, and those of a tile past them, in 32 bits
// Rows that are written do not overlap.
static bool apart(int64_t ts, int rows, int cols) { return rows <= 1 || ts >= cols || ts <= -(int64_t)cols; }

static int check_mx(const lily_mx_mat *m) {
  if (!m || m->rows < 0 || m->cols <= 0 || m->cols % 32) return LILY_Q4_ERR_INVALID_ARG;
  if (m->bits != 8 && m->bits != 4) return LILY_Q4_ERR_UNSUPPORTED;
  if (m->rows == 0) return LILY_Q4_OK;
  if (!m->codes || !m->scales || !aligned(m->codes, 32) || !aligned(m->scales, 4))
    return LILY_Q4_ERR_INVALID_ARG;
  return LILY_Q4_OK;
}

static int check_mx_rows(const lily_mx_mat *m, int dtype, const void *x, int64_t ts) {
  const int rc = check_mx(m);
  if (rc != LILY_Q4_OK) return rc;
  if (dtype != LILY_BF16 && dtype != LILY_F16 && dtype != LILY_F32) return LILY_Q4_ERR_UNSUPPORTED;
  if (m->rows == 0) return LILY_Q4_OK;
  if ((int64_t)m->rows * m->cols > (int64_t)1 << 40) return LILY_Q4_ERR_UNSUPPORTED;  // what a grid counts
  return flat_rows_ok(x, ts, dtype == LILY_F32 ? 4 : 2, m->rows) ? LILY_Q4_OK : LILY_Q4_ERR_INVALID_ARG;
}

static int check_linear(const lily_mx_mat *W, const lily_mx_mat *x) {
  int rc = check_mx(W);
  if (rc == LILY_Q4_OK) rc = check_mx(x);
  if (rc != LILY_Q4_OK) return rc;
  if (W->cols != x->cols) return LILY_Q4_ERR_INVALID_ARG;
  return W->bits == 4 && W->cols % 128 == 0 && std::max(W->rows, x->rows) <= kMaxRows ? LILY_Q4_OK : LILY_Q4_ERR_UNSUPPORTED;
}

}  // namespace lq4

using namespace lq4;

extern "C" {

int lily_q4_version(void) { return 100; }

const char *lily_q4_status_string(int status) {
  switch (status) {
    case LILY_Q4_OK: return "ok";
    case LILY_Q4_ERR_INVALID_ARG: return "invalid argument";
    case LILY_Q4_ERR_UNSUPPORTED: return "unsupported shape";
    case LILY_Q4_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case LILY_Q4_ERR_CUDA: return "CUDA error";
    case LILY_Q4_ERR_TIMEOUT: return "device-side wait timed out";
    case LILY_Q4_ERR_INDEX: return "length or page number out of range, or no token to draw";
    default: return "unknown status";
  }
}

int lily_q4_pack(const uint8_t *q, int32_t N, int32_t K, uint32_t *w) {
  if (!q || !w || N < 0 || K <= 0 || K % 8) return LILY_Q4_ERR_INVALID_ARG;
  for (int64_t n = 0; n < N; ++n)
    for (int64_t m = 0; m < K / 8; ++m) {
      uint32_t word = 0;
      const uint8_t *src = q + n * K + 8 * m;
      for (int j = 7; j >= 0; --j) word = (word << 4) | (uint32_t)(src[j] & 0xF);
      w[n * (K / 8) + m] = word;
    }
  return LILY_Q4_OK;
}

int lily_q4_unpack(const uint32_t *w, int32_t N, int32_t K, uint8_t *q) {
  if (!q || !w || N < 0 || K <= 0 || K % 8) return LILY_Q4_ERR_INVALID_ARG;
  for (int64_t n = 0; n < N; ++n)
    for (int64_t m = 0; m < K / 8; ++m) {
      uint32_t word = w[n * (K / 8) + m];
      for (int j = 0; j < 8; ++j, word >>= 4) q[n * K + 8 * m + j] = (uint8_t)(word & 0xF);
    }
  return LILY_Q4_OK;
}

size_t lily_q4_gemv_argmax_workspace_bytes(int32_t N, int32_t K) {
  if (N <= 0 || K <= 0 || K % LILY_Q4_GROUP) return 0;
  return lm_ws_layout(N, K).total;
}

size_t lily_q8_gemv_argmax_workspace_bytes(int32_t N, int32_t K) {
  if (N <= 0 || K <= 0 || K % LILY_Q4_GROUP) return 0;
  return lm_ws_layout(N, K, 8).total;
}

size_t lily_q4_moe_workspace_bytes(const lily_q4_moe_layer *layer, int32_t T, int32_t prefill) {
  if (check_layer(layer) != LILY_Q4_OK || T <= 0) return 0;
  if (prefill) {
    if (T > 8192) return 0;
    return prefill_ws_layout(*layer, T).total;
  }
  if (T > 16) return 0;
  return decode_ws_layout(*layer, T).total;
}

int lily_q4_moe_launches(const lily_q4_moe_layer *layer, int32_t T, int32_t prefill) {
  if (check_layer(layer) != LILY_Q4_OK || T <= 0) return 0;
  if (prefill)
    return T <= 8192 && layer->hidden >= 128 && layer->inter >= 128 ? prefill_launch_count(*layer) : 0;
  return T <= 16 ? decode_launch_count(*layer, T) : 0;
}

int lily_q4_workspace_init(void *ws, size_t ws_bytes, lily_q4_stream_t stream) {
  if (!ws || ws_bytes < kAlign || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  return cudaMemsetAsync(ws, 0, ws_bytes, (cudaStream_t)stream) == cudaSuccess ? LILY_Q4_OK
                                                                              : LILY_Q4_ERR_CUDA;
}

int lily_q4_workspace_status(void *ws, lily_q4_stream_t stream) {
  if (!ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  int32_t hdr[kHdrIndexError + 1] = {0};
  if (cudaStreamSynchronize(st) != cudaSuccess) return LILY_Q4_ERR_CUDA;
  if (cudaMemcpy(hdr, ws, sizeof(hdr), cudaMemcpyDeviceToHost) != cudaSuccess)
    return LILY_Q4_ERR_CUDA;
  // what is reported is cleared; an index error beside a time-out waits for the next call
  for (const int w : {kHdrError, kHdrIndexError}) {
    if (hdr[w] == 0) continue;
    if (cudaMemset(static_cast<int32_t *>(ws) + w, 0, sizeof(int32_t)) != cudaSuccess)
      return LILY_Q4_ERR_CUDA;
    return w == kHdrError ? LILY_Q4_ERR_TIMEOUT : LILY_Q4_ERR_INDEX;
  }
  return LILY_Q4_OK;
}

int lily_q4_selftest_timeout(void *ws, size_t ws_bytes, int32_t which, lily_q4_stream_t stream) {
  if (which != 0 && which != 1) return LILY_Q4_ERR_INVALID_ARG;
  if (!ws && ws_bytes == 0) {  // the fixed scratch of lily_q4_gemv_argmax_noalloc
    const int rc = noalloc_scratch(&ws);
    if (rc != LILY_Q4_OK) return rc;
    ws_bytes = kAlign;
  }
  if (!ws || ws_bytes < kAlign || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  return selftest_wait(ws, which, (cudaStream_t)stream);
}

int lily_q4_gemv_argmax(const lily_q4_mat *W, int32_t N, int32_t K, const uint16_t *x,
                        int32_t *token, float *logits, void *ws, size_t ws_bytes,
                        lily_q4_stream_t stream) {
  if (!W || !mat_ok(*W) || N <= 0 || K <= 0 || K % LILY_Q4_GROUP) return LILY_Q4_ERR_INVALID_ARG;
  if (!x || !aligned(x, 16) || !token || !aligned(token, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (logits && !aligned(logits, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  if (!width_ok(K)) return LILY_Q4_ERR_UNSUPPORTED;
  if (ws_bytes < lm_ws_layout(N, K).total) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  return launch_gemv_argmax(*W, N, K, x, token, logits, ws, (cudaStream_t)stream);
}

int lily_q4_gemv_argmax_logprobs(const lily_q4_mat *W, int32_t N, int32_t K, const uint16_t *x,
                                 int32_t *token, float *lse, float *logprobs, void *ws,
                                 size_t ws_bytes, lily_q4_stream_t stream) {
  if (!W || !mat_ok(*W) || N <= 0 || K <= 0 || K % LILY_Q4_GROUP) return LILY_Q4_ERR_INVALID_ARG;
  if (!x || !aligned(x, 16) || !token || !aligned(token, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (!lse || !aligned(lse, 4) || (logprobs && !aligned(logprobs, 4))) return LILY_Q4_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  if (!width_ok(K)) return LILY_Q4_ERR_UNSUPPORTED;
  if (ws_bytes < lm_ws_layout(N, K).total) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  return launch_gemv_argmax(*W, N, K, x, token, logprobs, ws, (cudaStream_t)stream, lse);
}

int lily_q8_gemv_argmax(const lily_q4_mat *W, int32_t N, int32_t K, const uint16_t *x,
                        int32_t *token, float *logits, void *ws, size_t ws_bytes,
                        lily_q4_stream_t stream) {
  if (!W || !mat_ok(*W) || N <= 0 || K <= 0 || K % LILY_Q4_GROUP) return LILY_Q4_ERR_INVALID_ARG;
  if (!x || !aligned(x, 16) || !token || !aligned(token, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (logits && !aligned(logits, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  if (K != 512 && K != 1024 && K != 2048) return LILY_Q4_ERR_UNSUPPORTED;
  if (ws_bytes < lm_ws_layout(N, K, 8).total_argmax) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  return launch_q8_gemv_argmax(*W, N, K, x, token, logits, ws, (cudaStream_t)stream);
}

int lily_q8_gemv_argmax_logprobs(const lily_q4_mat *W, int32_t N, int32_t K, const uint16_t *x,
                                 int32_t *token, float *lse, float *logprobs, void *ws,
                                 size_t ws_bytes, lily_q4_stream_t stream) {
  if (!W || !mat_ok(*W) || N <= 0 || K <= 0 || K % LILY_Q4_GROUP) return LILY_Q4_ERR_INVALID_ARG;
  if (!x || !aligned(x, 16) || !token || !aligned(token, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (!lse || !aligned(lse, 4) || (logprobs && !aligned(logprobs, 4))) return LILY_Q4_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  if (K != 512 && K != 1024 && K != 2048) return LILY_Q4_ERR_UNSUPPORTED;
  if (ws_bytes < lm_ws_layout(N, K, 8).total) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  return launch_q8_gemv_argmax(*W, N, K, x, token, logprobs, ws, (cudaStream_t)stream, lse);
}

int lily_q4_moe_decode(const lily_q4_moe_layer *layer, const uint16_t *x, int32_t T,
                       uint16_t *y, int32_t *topk_idx, float *topk_w, void *ws,
                       size_t ws_bytes, lily_q4_stream_t stream) {
  int rc = check_layer(layer);
  if (rc != LILY_Q4_OK) return rc;
  if (T < 0 || T > 16) return LILY_Q4_ERR_INVALID_ARG;
  if (T == 0) return LILY_Q4_OK;
  rc = check_io(x, y, topk_idx, topk_w, ws);
  if (rc != LILY_Q4_OK) return rc;
  if (ws_bytes < decode_ws_layout(*layer, T).total) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  return launch_moe_decode(*layer, x, T, y, topk_idx, topk_w, ws, (cudaStream_t)stream);
}

int lily_q4_moe_prefill(const lily_q4_moe_layer *layer, const uint16_t *x, int32_t T,
                        uint16_t *y, int32_t *topk_idx, float *topk_w, void *ws,
                        size_t ws_bytes, lily_q4_stream_t stream) {
  int rc = check_layer(layer);
  if (rc != LILY_Q4_OK) return rc;
  if (T < 0 || T > 8192) return LILY_Q4_ERR_INVALID_ARG;
  if (T == 0) return LILY_Q4_OK;
  rc = check_io(x, y, topk_idx, topk_w, ws);
  if (rc != LILY_Q4_OK) return rc;
  if (ws_bytes < prefill_ws_layout(*layer, T).total) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  return launch_moe_prefill(*layer, x, T, y, topk_idx, topk_w, ws, (cudaStream_t)stream);
}

int lily_rope_turns(int32_t rotary_dim, double base, int32_t scaling, double factor,
                    double original_len, double slow, double fast, uint64_t *turns) {
  if (rotary_dim < 0 || rotary_dim > 256 || rotary_dim % 2) return LILY_Q4_ERR_INVALID_ARG;
  if (rotary_dim == 0) return LILY_Q4_OK;
  if (!turns || !(base > 0) || !(base < HUGE_VAL)) return LILY_Q4_ERR_INVALID_ARG;
  if (scaling != LILY_ROPE_NONE && scaling != LILY_ROPE_LINEAR && scaling != LILY_ROPE_YARN)
    return LILY_Q4_ERR_INVALID_ARG;
  if (scaling != LILY_ROPE_NONE && !(factor > 0 && factor < HUGE_VAL)) return LILY_Q4_ERR_INVALID_ARG;
  if (scaling == LILY_ROPE_YARN &&
      !(original_len > 0 && original_len < HUGE_VAL && fast > slow && fast < HUGE_VAL && slow > -HUGE_VAL))
    return LILY_Q4_ERR_INVALID_ARG;
  return rope_turns(rotary_dim, base, scaling, factor, original_len, slow, fast, turns);
}

int lily_qk_norm_rope(const lily_qk_rope *op, int32_t T, int32_t q_heads, int32_t k_heads,
                      const int32_t *pos, const void *q, int64_t q_ts, int64_t q_hs, void *q_out,
                      int64_t qo_ts, int64_t qo_hs, const void *k, int64_t k_ts, int64_t k_hs,
                      void *k_out, int64_t ko_ts, int64_t ko_hs, lily_q4_stream_t stream) {
  if (!op || T < 0 || q_heads < 0 || k_heads < 0) return LILY_Q4_ERR_INVALID_ARG;
  if (op->head_dim < 8 || op->head_dim > 256 || op->head_dim % 8) return LILY_Q4_ERR_UNSUPPORTED;
  if (op->rotary_dim < 0 || op->rotary_dim > op->head_dim || op->rotary_dim % 2)
    return LILY_Q4_ERR_INVALID_ARG;
  if (op->dtype != LILY_BF16 && op->dtype != LILY_F16) return LILY_Q4_ERR_UNSUPPORTED;
  if ((op->interleaved != 0 && op->interleaved != 1) || (op->normalize != 0 && op->normalize != 1))
    return LILY_Q4_ERR_INVALID_ARG;
  if (op->normalize && !(op->eps >= 0.f)) return LILY_Q4_ERR_INVALID_ARG;
  if ((op->q_weight && !aligned(op->q_weight, 16)) || (op->k_weight && !aligned(op->k_weight, 16)))
    return LILY_Q4_ERR_INVALID_ARG;
  if (op->rotary_dim > 0 && (!op->turns || !aligned(op->turns, 8))) return LILY_Q4_ERR_INVALID_ARG;
  if (T == 0 || (q_heads == 0 && k_heads == 0)) return LILY_Q4_OK;
  if (op->rotary_dim > 0 && (!pos || !aligned(pos, 4))) return LILY_Q4_ERR_INVALID_ARG;
  const Rows qi{const_cast<void *>(q), q_ts, q_hs}, qo{q_out, qo_ts, qo_hs};
  const Rows ki{const_cast<void *>(k), k_ts, k_hs}, ko{k_out, ko_ts, ko_hs};
  if (q_heads && (!rows_ok(qi, 2) || !rows_ok(qo, 2))) return LILY_Q4_ERR_INVALID_ARG;
  if (k_heads && (!rows_ok(ki, 2) || !rows_ok(ko, 2))) return LILY_Q4_ERR_INVALID_ARG;
  return launch_qk_norm_rope(*op, T, q_heads, k_heads, pos, qi, qo, ki, ko, (cudaStream_t)stream);
}

int lily_kv8_append(const lily_kv8_cache *cache, const lily_kv8_batch *batch, int32_t T, int32_t dtype,
                    const void *k, int64_t k_ts, int64_t k_hs, const void *v, int64_t v_ts,
                    int64_t v_hs, void *ws, size_t ws_bytes, lily_q4_stream_t stream) {
  int rc = check_cache(cache);
  if (rc != LILY_Q4_OK) return rc;
  if (dtype != LILY_BF16 && dtype != LILY_F16) return LILY_Q4_ERR_UNSUPPORTED;
  rc = check_batch(batch, T, ws, ws_bytes);
  if (rc != LILY_Q4_OK || T == 0) return rc;
  const Rows kr{const_cast<void *>(k), k_ts, k_hs}, vr{const_cast<void *>(v), v_ts, v_hs};
  if (!rows_ok(kr, 2) || !rows_ok(vr, 2)) return LILY_Q4_ERR_INVALID_ARG;
  return launch_kv8_append(*cache, *batch, T, dtype, kr, vr, ws, (cudaStream_t)stream);
}

int lily_kv8_read(const lily_kv8_cache *cache, const lily_kv8_batch *batch, int32_t T, int32_t dtype,
                  void *k_out, int64_t k_ts, int64_t k_hs, void *v_out, int64_t v_ts, int64_t v_hs,
                  void *ws, size_t ws_bytes, lily_q4_stream_t stream) {
  int rc = check_cache(cache);
  if (rc != LILY_Q4_OK) return rc;
  if (dtype != LILY_BF16 && dtype != LILY_F16 && dtype != LILY_F32) return LILY_Q4_ERR_UNSUPPORTED;
  rc = check_batch(batch, T, ws, ws_bytes);
  if (rc != LILY_Q4_OK || T == 0) return rc;
  const Rows kr{k_out, k_ts, k_hs}, vr{v_out, v_ts, v_hs};
  const int eb = dtype == LILY_F32 ? 4 : 2;
  if (!rows_ok(kr, eb) || !rows_ok(vr, eb)) return LILY_Q4_ERR_INVALID_ARG;
  return launch_kv8_read(*cache, *batch, T, dtype, kr, vr, ws, (cudaStream_t)stream);
}

size_t lily_kv8_attention_workspace_bytes(const lily_kv8_cache *cache, const lily_kv8_batch *batch,
                                          int32_t T, int32_t q_heads) {
  if (check_attention(cache, batch, T, q_heads) != LILY_Q4_OK) return 0;
  return kv8_attention_ws_bytes(*cache, *batch, T, q_heads);
}

int lily_kv8_attention(const lily_kv8_cache *cache, const lily_kv8_batch *batch, int32_t T,
                       int32_t q_heads, int32_t dtype, float scale, int32_t causal, int32_t window,
                       const void *q, int64_t q_ts, int64_t q_hs, void *out, int64_t o_ts,
                       int64_t o_hs, float *lse, void *ws, size_t ws_bytes, lily_q4_stream_t stream) {
  int rc = check_attention(cache, batch, T, q_heads);
  if (rc != LILY_Q4_OK) return rc;
  if (dtype != LILY_BF16 && dtype != LILY_F16) return LILY_Q4_ERR_UNSUPPORTED;
  if ((causal != 0 && causal != 1) || window < 0 || !(scale == scale) || !(fabsf(scale) < HUGE_VALF))
    return LILY_Q4_ERR_INVALID_ARG;
  rc = check_batch(batch, T, ws, ws_bytes);
  if (rc != LILY_Q4_OK || T == 0) return rc;
  const Rows qr{const_cast<void *>(q), q_ts, q_hs}, orow{out, o_ts, o_hs};
  if (!rows_ok(qr, 2) || !rows_ok(orow, 2) || (lse && !aligned(lse, 4))) return LILY_Q4_ERR_INVALID_ARG;
  const size_t need = kv8_attention_ws_bytes(*cache, *batch, T, q_heads);
  if (need == 0) return LILY_Q4_ERR_UNSUPPORTED;
  if (ws_bytes < need) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  const AttnShape s{T, q_heads, dtype, causal, window, scale};
  return launch_kv8_attention(*cache, *batch, s, qr, orow, lse, ws, (cudaStream_t)stream);
}

int lily_add_rms_norm(const lily_rms_norm *op, int32_t T, const void *x, int64_t x_ts, const void *add,
                      int64_t add_ts, void *sum, int64_t sum_ts, void *y, int64_t y_ts,
                      const lily_mx_mat *mx, lily_q4_stream_t stream) {
  if (!op || T < 0) return LILY_Q4_ERR_INVALID_ARG;
  if (op->width < 8 || op->width > 32768 || op->width % 8) return LILY_Q4_ERR_UNSUPPORTED;
  if (op->dtype != LILY_BF16 && op->dtype != LILY_F16) return LILY_Q4_ERR_UNSUPPORTED;
  if (!(op->eps >= 0.f && op->eps < HUGE_VALF) || !(fabsf(op->weight_offset) < HUGE_VALF)) return LILY_Q4_ERR_INVALID_ARG;
  if (op->weight && !aligned(op->weight, 16)) return LILY_Q4_ERR_INVALID_ARG;
  if (!sum && !y && !mx) return LILY_Q4_ERR_INVALID_ARG;
  if (mx) {
    const int rc = check_mx(mx);
    if (rc != LILY_Q4_OK) return rc;
    if (mx->cols != op->width || mx->rows < T) return LILY_Q4_ERR_INVALID_ARG;
  }
  if (T > kMaxRows) return LILY_Q4_ERR_UNSUPPORTED;
  if (T == 0) return LILY_Q4_OK;
  if (!flat_rows_ok(x, x_ts, 2, T) || (add && !flat_rows_ok(add, add_ts, 2, T))) return LILY_Q4_ERR_INVALID_ARG;
  if (sum && (!flat_rows_ok(sum, sum_ts, 2, T) || !apart(sum_ts, T, op->width))) return LILY_Q4_ERR_INVALID_ARG;
  if (y && (!flat_rows_ok(y, y_ts, 2, T) || !apart(y_ts, T, op->width))) return LILY_Q4_ERR_INVALID_ARG;
  if (sum && sum == y) return LILY_Q4_ERR_INVALID_ARG;
  // in place row by row
  if (T > 1 && ((sum && sum == x && sum_ts != x_ts) || (sum && sum == add && sum_ts != add_ts) || (y && y == x && y_ts != x_ts) ||
                (y && y == add && y_ts != add_ts)))
    return LILY_Q4_ERR_INVALID_ARG;
  return launch_add_rms_norm(*op, T, x, x_ts, add, add_ts, sum, sum_ts, y, y_ts, mx, (cudaStream_t)stream);
}

int lily_mx_quantize(const lily_mx_mat *m, int32_t dtype, const void *x, int64_t x_ts, lily_q4_stream_t stream) {
  const int rc = check_mx_rows(m, dtype, x, x_ts);
  if (rc != LILY_Q4_OK || m->rows == 0) return rc;
  return launch_mx_blocks(*m, dtype, const_cast<void *>(x), x_ts, false, (cudaStream_t)stream);
}

int lily_mx_read(const lily_mx_mat *m, int32_t dtype, void *x, int64_t x_ts, lily_q4_stream_t stream) {
  const int rc = check_mx_rows(m, dtype, x, x_ts);
  if (rc != LILY_Q4_OK || m->rows == 0) return rc;
  if (!apart(x_ts, m->rows, m->cols)) return LILY_Q4_ERR_INVALID_ARG;
  return launch_mx_blocks(*m, dtype, x, x_ts, true, (cudaStream_t)stream);
}

size_t lily_mx4_linear_workspace_bytes(const lily_mx_mat *W, const lily_mx_mat *x) {
  return check_linear(W, x) == LILY_Q4_OK ? kAlign : 0;
}

int lily_mx4_linear(const lily_mx_mat *W, const lily_mx_mat *x, int32_t dtype, void *out, int64_t out_ts,
                    void *ws, size_t ws_bytes, lily_q4_stream_t stream) {
  const int rc = check_linear(W, x);
  if (rc != LILY_Q4_OK) return rc;
  if (dtype != LILY_BF16 && dtype != LILY_F16 && dtype != LILY_F32) return LILY_Q4_ERR_UNSUPPORTED;
  if (W->rows == 0 || x->rows == 0) return LILY_Q4_OK;
  if (!out || !aligned(out, dtype == LILY_F32 ? 4 : 2) || !ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  if (ws_bytes < kAlign) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  // output tiles are counted in 32 bits; there are at least 16 rows in one
  if (((int64_t)W->rows + 127) / 128 * (((int64_t)x->rows + 15) / 16) > INT32_MAX) return LILY_Q4_ERR_UNSUPPORTED;
  if (!apart(out_ts, x->rows, W->rows)) return LILY_Q4_ERR_INVALID_ARG;
  return launch_mx4_linear(*W, *x, dtype, out, out_ts, ws, (cudaStream_t)stream);
}

size_t lily_sample_workspace_bytes(int32_t B, int32_t V) {
  return B >= 0 && V > 0 && V <= kSampleMaxVocab ? kAlign : 0;
}

int lily_sample(const lily_sampling *op, int32_t B, int32_t V, int32_t dtype, const void *logits, int64_t ts,
                const float *u, int32_t *token, float *prob, int32_t *kept, void *ws, size_t ws_bytes,
                lily_q4_stream_t stream) {
  if (!op || B < 0 || V <= 0) return LILY_Q4_ERR_INVALID_ARG;
  if (V > kSampleMaxVocab || B > 1 << 24) return LILY_Q4_ERR_UNSUPPORTED;
  if (dtype != LILY_BF16 && dtype != LILY_F16 && dtype != LILY_F32) return LILY_Q4_ERR_UNSUPPORTED;
  for (const void *p : {(const void *)op->temperature, (const void *)op->top_k, (const void *)op->top_p,
                        (const void *)op->min_p, (const void *)prob, (const void *)kept})
    if (!aligned(p, 4)) return LILY_Q4_ERR_INVALID_ARG;
  if (B == 0) return LILY_Q4_OK;
  if (!logits || !aligned(logits, dtype == LILY_F32 ? 4 : 2) || !u || !aligned(u, 4) || !token || !aligned(token, 4))
    return LILY_Q4_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return LILY_Q4_ERR_INVALID_ARG;
  if (ws_bytes < kAlign) return LILY_Q4_ERR_WORKSPACE_TOO_SMALL;
  return launch_sample(*op, B, V, dtype, logits, ts, u, token, prob, kept, ws, (cudaStream_t)stream);
}

int lily_q4_call(int32_t which, const void *words) {
  // how many words each call has, and which of them stand for 32-bit numbers and have to be such
  struct Shape {
    int words, ints[6];
  };
  static const Shape kShapes[] = {{18, {1, 2, 3, 0}}, {13, {2, 3, 0}}, {13, {2, 3, 0}}, {18, {2, 3, 4, 6, 7, 0}},
                                  {0, {0}},           {0, {0}},        {0, {0}},        {0, {0}},
                                  {12, {1, 0}},       {5, {1, 0}},     {5, {1, 0}},    {8, {2, 0}},
                                  {13, {1, 2, 3, 0}}};
  if (!words || which < 0 || which >= (int)(sizeof(kShapes) / sizeof(kShapes[0])) || !kShapes[which].words)
    return LILY_Q4_ERR_INVALID_ARG;
  int64_t w[18];  // the words may be unaligned
  memcpy(w, words, kShapes[which].words * sizeof(int64_t));
  for (const int *i = kShapes[which].ints; *i; ++i)
    if (w[*i] != (int32_t)w[*i]) return LILY_Q4_ERR_INVALID_ARG;
  auto ptr = [&](int i) { return reinterpret_cast<void *>(w[i]); };
  auto i32 = [&](int i) { return (int32_t)w[i]; };
  auto stream = [&](int i) { return reinterpret_cast<lily_q4_stream_t>(w[i]); };
  const auto *cache = reinterpret_cast<const lily_kv8_cache *>(w[0]);
  const auto *batch = reinterpret_cast<const lily_kv8_batch *>(w[1]);
  switch (which) {
    case LILY_CALL_QK_NORM_ROPE:
      return lily_qk_norm_rope(reinterpret_cast<const lily_qk_rope *>(w[0]), i32(1), i32(2), i32(3),
                               static_cast<const int32_t *>(ptr(4)), ptr(5), w[6], w[7], ptr(8), w[9], w[10],
                               ptr(11), w[12], w[13], ptr(14), w[15], w[16], stream(17));
    case LILY_CALL_KV8_APPEND:
      return lily_kv8_append(cache, batch, i32(2), i32(3), ptr(4), w[5], w[6], ptr(7), w[8], w[9], ptr(10),
                             (size_t)w[11], stream(12));
    case LILY_CALL_KV8_READ:
      return lily_kv8_read(cache, batch, i32(2), i32(3), ptr(4), w[5], w[6], ptr(7), w[8], w[9], ptr(10),
                           (size_t)w[11], stream(12));
    case LILY_CALL_ADD_RMS_NORM:
      return lily_add_rms_norm(reinterpret_cast<const lily_rms_norm *>(w[0]), i32(1), ptr(2), w[3], ptr(4), w[5],
                               ptr(6), w[7], ptr(8), w[9], static_cast<const lily_mx_mat *>(ptr(10)), stream(11));
    case LILY_CALL_MX_QUANTIZE:
      return lily_mx_quantize(reinterpret_cast<const lily_mx_mat *>(w[0]), i32(1), ptr(2), w[3], stream(4));
    case LILY_CALL_MX_READ:
      return lily_mx_read(reinterpret_cast<const lily_mx_mat *>(w[0]), i32(1), ptr(2), w[3], stream(4));
    case LILY_CALL_MX4_LINEAR:
      return lily_mx4_linear(reinterpret_cast<const lily_mx_mat *>(w[0]), reinterpret_cast<const lily_mx_mat *>(w[1]),
                             i32(2), ptr(3), w[4], ptr(5), (size_t)w[6], stream(7));
    case LILY_CALL_SAMPLE:
      return lily_sample(reinterpret_cast<const lily_sampling *>(w[0]), i32(1), i32(2), i32(3), ptr(4), w[5],
                         static_cast<const float *>(ptr(6)), static_cast<int32_t *>(ptr(7)),
                         static_cast<float *>(ptr(8)), static_cast<int32_t *>(ptr(9)), ptr(10), (size_t)w[11], stream(12));
    default: {
      double scale;
      memcpy(&scale, &w[5], sizeof(scale));
      return lily_kv8_attention(cache, batch, i32(2), i32(3), i32(4), (float)scale, i32(6), i32(7), ptr(8), w[9],
                                w[10], ptr(11), w[12], w[13], static_cast<float *>(ptr(14)), ptr(15), (size_t)w[16],
                                stream(17));
    }
  }
}

}  // extern "C"
