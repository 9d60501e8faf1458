// C ABI of the serving calls: argument validation and dispatch (include/gptq.h).
#include "common.cuh"

namespace gptq {

gptq_status qk_norm_rope_launch(const void* Q, const void* K, int in_dtype, long long T, int hq, int hk, int D,
                                long long ldq, long long ldk, const float* wq, const float* wk, float eps,
                                const float* cosv, const float* sinv, long long n_pos, int rot, int interleaved,
                                const int* positions, void* Qo, void* Ko, int out_dtype, long long ldqo,
                                long long ldko, cudaStream_t s);
gptq_status kv_append_launch(const void* K, const void* V, int dtype, long long T, int H, int D, long long ldk,
                             long long ldv, const long long* slots, void* pool, long long num_pages, int page,
                             cudaStream_t s);
gptq_status kv_read_launch(const void* pool, long long num_pages, int page, int H, int D, const long long* slots,
                           long long T, void* K, void* V, int dtype, long long ldk, long long ldv, cudaStream_t s);
size_t kv_attention_workspace_bytes(long long total_q, int Hq, int H, int D, long long batch, long long max_q);
gptq_status kv_attention_launch(const void* Q, int dtype, long long total_q, int Hq, int H, int D, long long ldq,
                                const int* cu_q, const int* kv_lens, const int* table, long long ldt,
                                long long table_width, long long batch, long long max_q, const void* pool,
                                long long num_pages, int page, float sm_scale, int causal, long long window, void* O,
                                long long ldo, float* lse, void* ws, cudaStream_t s);
size_t adapter_workspace_bytes(long long m, long long d, int bits, int group_size, long long T, int rank);
gptq_status adapter_linear_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m,
                                  long long d, int bits, int group_size, const uint16_t* X, long long T, long long ldx,
                                  const uint16_t* A, const uint16_t* B, const float* alpha, long long n_adapters,
                                  int rank, const int* ids, void* Y, int y_dtype, long long ldy, void* ws,
                                  cudaStream_t s);
bool tensor_maps_available();

namespace {
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int elem_bytes(int dtype) { return dtype == GPTQ_F32 ? 4 : 2; }
// Keys of a sequence: a tile of keys past them still has 32-bit numbers.
constexpr int64_t kMaxKeys = 0x7FFFFF00;
bool any_dtype(int dtype) { return dtype == GPTQ_F32 || dtype == GPTQ_BF16 || dtype == GPTQ_F16; }

// Rows of `width` elements with token stride ld that 16-byte accesses may read.
bool rows_ok(const void* p, int dtype, long long ld, long long width) {
  return p && aligned(p, 16) && ld >= width && (ld * elem_bytes(dtype)) % 16 == 0;
}

gptq_status check_cache(const void* pool, int64_t num_pages, int page_size, int n_kv_heads, int head_dim) {
  if (!pool || !aligned(pool, 16)) return set_error(GPTQ_ERR_INVALID_ARG, "pool must be a 16-byte aligned pointer");
  if (num_pages < 1 || num_pages > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "num_pages out of range");
  if (page_size < 16 || page_size > 256 || page_size % 16)
    return set_error(GPTQ_ERR_INVALID_ARG, "page_size must be a multiple of 16 in [16, 256]");
  if (n_kv_heads < 1 || n_kv_heads > 65535) return set_error(GPTQ_ERR_INVALID_ARG, "n_kv_heads out of range");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return set_error(GPTQ_ERR_UNSUPPORTED, "this build runs head_dim 64, 128 or 256 in the cache");
  return GPTQ_OK;
}

gptq_status check_packed(const uint32_t* qweight, const float* scales, const float* zeros, int64_t m, int64_t d,
                         int bits, int group_size) {
  if (!qweight || !scales || !zeros) return set_error(GPTQ_ERR_INVALID_ARG, "NULL pointer");
  if (m < 1 || m > ((int64_t)1 << 30) || d < 32 || d > 65536 || d % 32)
    return set_error(GPTQ_ERR_INVALID_ARG, "m >= 1 and d a multiple of 32 in [32, 65536] are required");
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return set_error(GPTQ_ERR_INVALID_ARG, "bits must be 2, 3, 4 or 8");
  if (group_size != -1 && (group_size < 32 || group_size % 32 || d % group_size))
    return set_error(GPTQ_ERR_INVALID_ARG, "group_size must be -1 or a multiple of 32 that divides d");
  const size_t qa = (bits == 4 || bits == 8) ? 16 : (bits == 2 ? 8 : 4);
  if (!aligned(qweight, qa) || !aligned(scales, 4) || !aligned(zeros, 4))
    return set_error(GPTQ_ERR_INVALID_ARG, "qweight misaligned (16 bytes for 4 and 8 bits, 8 for 2)");
  return GPTQ_OK;
}
}  // namespace

}  // namespace gptq

using namespace gptq;

extern "C" {

gptq_status gptq_qk_norm_rope(const void* Q, const void* K, int in_dtype, int64_t T, int n_q_heads, int n_k_heads,
                              int head_dim, int64_t ldq, int64_t ldk, const float* wq, const float* wk, float eps,
                              const float* cos_table, const float* sin_table, int64_t n_positions, int rot_dim,
                              int interleaved, const int32_t* positions, void* Qo, void* Ko, int out_dtype,
                              int64_t ldqo, int64_t ldko, gptq_stream_t stream) {
  clear_error();
  if (!any_dtype(in_dtype) || !any_dtype(out_dtype)) return set_error(GPTQ_ERR_INVALID_ARG, "unknown dtype");
  if (T < 0 || T > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "T out of range");
  if (n_q_heads < 1 || n_k_heads < 0 || n_q_heads > 65535 || n_k_heads > 65535)
    return set_error(GPTQ_ERR_INVALID_ARG, "head counts out of range");
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return set_error(GPTQ_ERR_INVALID_ARG, "head_dim must be a multiple of 8 in [8, 256]");
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
    return set_error(GPTQ_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [0, head_dim]");
  if (!(eps >= 0.0f) || eps > 1e30f) return set_error(GPTQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (T == 0) return GPTQ_OK;
  if (!rows_ok(Q, in_dtype, ldq, (int64_t)n_q_heads * head_dim) ||
      !rows_ok(Qo, out_dtype, ldqo, (int64_t)n_q_heads * head_dim))
    return set_error(GPTQ_ERR_INVALID_ARG, "Q and Qo need 16-byte aligned rows of n_q_heads * head_dim values");
  if (n_k_heads && (!rows_ok(K, in_dtype, ldk, (int64_t)n_k_heads * head_dim) ||
                    !rows_ok(Ko, out_dtype, ldko, (int64_t)n_k_heads * head_dim)))
    return set_error(GPTQ_ERR_INVALID_ARG, "K and Ko need 16-byte aligned rows of n_k_heads * head_dim values");
  if ((wq && !aligned(wq, 16)) || (wk && !aligned(wk, 16)))
    return set_error(GPTQ_ERR_INVALID_ARG, "wq and wk must be 16-byte aligned");
  if (rot_dim) {
    if (!cos_table || !sin_table || !positions || !aligned(cos_table, 16) || !aligned(sin_table, 16))
      return set_error(GPTQ_ERR_INVALID_ARG, "a rotation needs positions and 16-byte aligned tables");
    if (n_positions < 1) return set_error(GPTQ_ERR_INVALID_ARG, "n_positions must be at least 1");
  }
  return qk_norm_rope_launch(Q, K, in_dtype, T, n_q_heads, n_k_heads, head_dim, ldq, ldk, wq, wk, eps, cos_table,
                             sin_table, n_positions, rot_dim, interleaved != 0, positions, Qo, Ko, out_dtype, ldqo,
                             ldko, reinterpret_cast<cudaStream_t>(stream));
}

gptq_status gptq_kv_append(const void* K, const void* V, int kv_dtype, int64_t T, int n_kv_heads, int head_dim,
                           int64_t ldk, int64_t ldv, const int64_t* slots, void* pool, int64_t num_pages, int page_size,
                           gptq_stream_t stream) {
  clear_error();
  if (gptq_status st = check_cache(pool, num_pages, page_size, n_kv_heads, head_dim)) return st;
  if (!any_dtype(kv_dtype)) return set_error(GPTQ_ERR_INVALID_ARG, "unknown dtype");
  if (T < 0 || T > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "T out of range");
  if (T == 0) return GPTQ_OK;
  if (!slots) return set_error(GPTQ_ERR_INVALID_ARG, "slots is NULL");
  const int64_t width = (int64_t)n_kv_heads * head_dim;
  if (!rows_ok(K, kv_dtype, ldk, width) || !rows_ok(V, kv_dtype, ldv, width))
    return set_error(GPTQ_ERR_INVALID_ARG, "K and V need 16-byte aligned rows of n_kv_heads * head_dim values");
  return kv_append_launch(K, V, kv_dtype, T, n_kv_heads, head_dim, ldk, ldv,
                          reinterpret_cast<const long long*>(slots), pool, num_pages, page_size,
                          reinterpret_cast<cudaStream_t>(stream));
}

gptq_status gptq_kv_read(const void* pool, int64_t num_pages, int page_size, int n_kv_heads, int head_dim,
                         const int64_t* slots, int64_t T, void* K, void* V, int kv_dtype, int64_t ldk, int64_t ldv,
                         gptq_stream_t stream) {
  clear_error();
  if (gptq_status st = check_cache(pool, num_pages, page_size, n_kv_heads, head_dim)) return st;
  if (!any_dtype(kv_dtype)) return set_error(GPTQ_ERR_INVALID_ARG, "unknown dtype");
  if (T < 0 || T > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "T out of range");
  if (T == 0) return GPTQ_OK;
  if (!slots) return set_error(GPTQ_ERR_INVALID_ARG, "slots is NULL");
  const int64_t width = (int64_t)n_kv_heads * head_dim;
  if (!rows_ok(K, kv_dtype, ldk, width) || !rows_ok(V, kv_dtype, ldv, width))
    return set_error(GPTQ_ERR_INVALID_ARG, "K and V need 16-byte aligned rows of n_kv_heads * head_dim values");
  return kv_read_launch(pool, num_pages, page_size, n_kv_heads, head_dim, reinterpret_cast<const long long*>(slots), T,
                        K, V, kv_dtype, ldk, ldv, reinterpret_cast<cudaStream_t>(stream));
}

size_t gptq_kv_attention_workspace_size(int64_t total_q, int n_q_heads, int n_kv_heads, int head_dim, int64_t batch,
                                        int64_t max_q) {
  if (total_q < 0 || total_q > 0x7FFFFFFF || n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads > 65535 ||
      n_q_heads % n_kv_heads || batch < 1 || batch > 65535 || max_q < 1 || max_q > 0x7FFFFFFF)
    return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return kv_attention_workspace_bytes(total_q, n_q_heads, n_kv_heads, head_dim, batch, max_q);
}

gptq_status gptq_kv_attention(const void* Q, int q_dtype, int64_t total_q, int n_q_heads, int n_kv_heads, int head_dim,
                              int64_t ldq, const int32_t* cu_q, const int32_t* kv_lens, const int32_t* block_table,
                              int64_t ldt, int64_t table_width, int64_t batch, int64_t max_q, const void* pool,
                              int64_t num_pages, int page_size, float sm_scale, int causal, int64_t window, void* O,
                              int64_t ldo, float* lse, void* ws, size_t ws_bytes, gptq_stream_t stream) {
  clear_error();
  if (gptq_status st = check_cache(pool, num_pages, page_size, n_kv_heads, head_dim)) return st;
  if (q_dtype != GPTQ_BF16 && q_dtype != GPTQ_F16)
    return set_error(GPTQ_ERR_INVALID_ARG, "q_dtype must be GPTQ_BF16 or GPTQ_F16");
  if (n_q_heads < n_kv_heads || n_q_heads > 65535 || n_q_heads % n_kv_heads)
    return set_error(GPTQ_ERR_INVALID_ARG, "n_q_heads must be a multiple of n_kv_heads");
  if (total_q < 0 || total_q > 0x7FFFFFFF || batch < 0 || batch > 65535 || max_q < 0 || max_q > 0x7FFFFFFF)
    return set_error(GPTQ_ERR_INVALID_ARG, "total_q, batch or max_q out of range");
  if (!(sm_scale > 0.0f) || sm_scale > 1e30f) return set_error(GPTQ_ERR_INVALID_ARG, "sm_scale must be positive and finite");
  if (window < 0) return set_error(GPTQ_ERR_INVALID_ARG, "window must be >= 0");
  if (table_width < 0 || table_width > kMaxKeys / page_size || ldt < table_width)
    return set_error(GPTQ_ERR_INVALID_ARG, "table_width * page_size must be at most 2^31 - 256 and ldt cover the table");
  if (total_q == 0 || batch == 0 || max_q == 0) return GPTQ_OK;
  if (!cu_q || !kv_lens || (table_width && !block_table)) return set_error(GPTQ_ERR_INVALID_ARG, "NULL pointer");
  const int64_t width = (int64_t)n_q_heads * head_dim;
  if (!rows_ok(Q, q_dtype, ldq, width) || !rows_ok(O, q_dtype, ldo, width))
    return set_error(GPTQ_ERR_INVALID_ARG, "Q and O need 16-byte aligned rows of n_q_heads * head_dim values");
  const size_t need = kv_attention_workspace_bytes(total_q, n_q_heads, n_kv_heads, head_dim, batch, max_q);
  if (!ws || !aligned(ws, 256)) return set_error(GPTQ_ERR_INVALID_ARG, "ws must be 256-byte aligned");
  if (ws_bytes < need) return set_error(GPTQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", ws_bytes, need);
  return kv_attention_launch(Q, q_dtype, total_q, n_q_heads, n_kv_heads, head_dim, ldq, cu_q, kv_lens, block_table, ldt,
                             table_width, batch, max_q, pool, num_pages, page_size, sm_scale, causal != 0, window, O,
                             ldo, lse, ws, reinterpret_cast<cudaStream_t>(stream));
}

size_t gptq_adapter_workspace_size(int64_t m, int64_t d, int bits, int group_size, int64_t T, int rank) {
  if (m < 1 || m > ((int64_t)1 << 30) || d < 32 || d > 65536 || d % 32 || T < 0 || T > 0x7FFFFFFF) return 0;
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return 0;
  if (group_size != -1 && (group_size < 32 || group_size % 32 || d % group_size)) return 0;
  if (rank < 8 || rank > 128 || rank % 8) return 0;
  return adapter_workspace_bytes(m, d, bits, group_size, T, rank);
}

gptq_status gptq_adapter_linear(const uint32_t* qweight, const float* scales, const float* zeros, int64_t m, int64_t d,
                                int bits, int group_size, const uint16_t* X, int64_t T, int64_t ldx, const uint16_t* A,
                                const uint16_t* B, const float* alpha, int64_t n_adapters, int rank, const int32_t* ids,
                                void* Y, int y_dtype, int64_t ldy, void* ws, size_t ws_bytes, gptq_stream_t stream) {
  clear_error();
  if (gptq_status st = check_packed(qweight, scales, zeros, m, d, bits, group_size)) return st;
  if (y_dtype != GPTQ_F32 && y_dtype != GPTQ_BF16)
    return set_error(GPTQ_ERR_INVALID_ARG, "y_dtype must be GPTQ_F32 or GPTQ_BF16");
  if (rank < 8 || rank > 128 || rank % 8) return set_error(GPTQ_ERR_INVALID_ARG, "rank must be a multiple of 8 in [8, 128]");
  if (n_adapters < 0 || n_adapters > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "n_adapters out of range");
  if (T < 0 || T > 0x7FFFFFFF || ldx < d || ldx % 8 || ldy < m) return set_error(GPTQ_ERR_INVALID_ARG, "bad T, ldx or ldy");
  if (((T + 127) / 128) * ((m + 127) / 128) > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "too many output tiles");
  if (T == 0) return GPTQ_OK;
  if (!X || !Y || !aligned(X, 16)) return set_error(GPTQ_ERR_INVALID_ARG, "X must be 16-byte aligned, Y not NULL");
  if (n_adapters > 0 && (!A || !B || !ids || !aligned(A, 16) || !aligned(B, 16)))
    return set_error(GPTQ_ERR_INVALID_ARG, "adapters need ids and 16-byte aligned A and B");
  const size_t need = adapter_workspace_bytes(m, d, bits, group_size, T, rank);
  if (!ws || !aligned(ws, 256)) return set_error(GPTQ_ERR_INVALID_ARG, "ws must be 256-byte aligned");
  if (ws_bytes < need) return set_error(GPTQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", ws_bytes, need);
  if (!tensor_maps_available()) return set_error(GPTQ_ERR_UNSUPPORTED, "the tensor-map encoder is not available");
  return adapter_linear_launch(qweight, scales, zeros, m, d, bits, group_size, X, T, ldx, A, B, alpha, n_adapters, rank,
                               n_adapters > 0 ? ids : nullptr, Y, y_dtype, ldy, ws,
                               reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
