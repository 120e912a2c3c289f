// serving_api.cu — the C ABI of the serving-side operators: argument validation, workspace
// layout, stream-ordered launches.  Nothing is allocated and no call synchronises the host.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "serving.h"

namespace {

dspark_status fail(dspark_status code, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return dspark::record_error(code, msg);
}

dspark_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? DSPARK_OK : fail(DSPARK_CUDA_ERROR, "%s: %s", what, cudaGetErrorString(e));
}

#define CHECK_PTR(p)                                                              \
  do {                                                                            \
    if ((p) == nullptr) return fail(DSPARK_INVALID_ARG, "null pointer: %s", #p); \
  } while (0)
#define CHECK_ALIGN(p, n)                                                                     \
  do {                                                                                        \
    if ((reinterpret_cast<uintptr_t>(p) & ((n) - 1u)) != 0)                                   \
      return fail(DSPARK_INVALID_ARG, "%s must start on a %d-byte boundary", #p, (int)(n)); \
  } while (0)
#define CHECK(call)                             \
  do {                                          \
    const dspark_status st_ = (call);           \
    if (st_ != DSPARK_OK) return st_;           \
  } while (0)

bool is_float_type(int d) { return d == DSPARK_F32 || d == DSPARK_BF16 || d == DSPARK_F16; }
bool is_half_type(int d) { return d == DSPARK_BF16 || d == DSPARK_F16; }
size_t size_of(int d) { return d == DSPARK_F32 ? 4 : (d == DSPARK_E4M3 ? 1 : 2); }

dspark_status check_workspace(void* workspace, size_t ws_bytes, size_t need) {
  CHECK_PTR(workspace);
  CHECK_ALIGN(workspace, 256);
  if (ws_bytes < need) return fail(DSPARK_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", ws_bytes, need);
  return DSPARK_OK;
}

// ------------------------------------------------------------------ token log probabilities

dspark_status check_logits(int N, int V, int64_t row_stride, int dtype, float temperature) {
  if (N < 0 || V < 1) return fail(DSPARK_INVALID_ARG, "sizes must be positive (N=%d V=%d)", N, V);
  if (V > dspark::kMaxLogprobV) return fail(DSPARK_UNSUPPORTED_SHAPE, "V=%d exceeds %d", V, dspark::kMaxLogprobV);
  if (!is_float_type(dtype)) return fail(DSPARK_INVALID_ARG, "bad dtype %d", dtype);
  if (row_stride < V) return fail(DSPARK_INVALID_ARG, "row_stride %lld is below V=%d", (long long)row_stride, V);
  if (!(temperature > 0.f) || !isfinite(temperature) || !isfinite(1.4426951f / temperature))
    return fail(DSPARK_INVALID_ARG, "temperature must be positive and finite");
  return DSPARK_OK;
}

// ----------------------------------------------------------------------------- paged cache

struct CacheLayout {
  size_t counts, hole, mover, rank, total;
};

CacheLayout cache_layout(int num_pages) {
  CacheLayout L;
  const size_t list = dspark::align256(4 * (size_t)num_pages);
  L.counts = 256;
  L.hole = L.counts + 256;
  L.mover = L.hole + list;
  L.rank = L.mover + list;
  L.total = L.rank + list;
  return L;
}

dspark_status check_geometry(int R, int num_pages, int page_size, int max_pages, int64_t table_stride) {
  if (R < 1 || num_pages < 1 || page_size < 1 || max_pages < 1)
    return fail(DSPARK_INVALID_ARG, "sizes must be positive (R=%d num_pages=%d page_size=%d max_pages=%d)", R,
                num_pages, page_size, max_pages);
  if (R > dspark::kMaxSlots) return fail(DSPARK_UNSUPPORTED_SHAPE, "R=%d exceeds %d", R, dspark::kMaxSlots);
  if (num_pages > dspark::kMaxPages)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "num_pages=%d exceeds %d", num_pages, dspark::kMaxPages);
  // (a tile's positions go past the last page by less than 256 before they are tested)
  if ((int64_t)max_pages * page_size >= ((int64_t)1 << 31) - 256)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "max_pages * page_size must be below 2^31 - 256");
  if (table_stride < max_pages)
    return fail(DSPARK_INVALID_ARG, "table_stride %lld is below max_pages=%d", (long long)table_stride, max_pages);
  return DSPARK_OK;
}

dspark_status check_tables(const dspark::CacheTables& t, void* workspace, size_t ws_bytes) {
  CHECK(check_geometry(t.R, t.num_pages, t.page_size, t.max_pages, t.table_stride));
  CHECK_PTR(t.page_table);
  CHECK_PTR(t.seq_len);
  CHECK_PTR(t.ref_count);
  return check_workspace(workspace, ws_bytes, cache_layout(t.num_pages).total);
}

dspark::CacheTables tables(int R, int num_pages, int page_size, int max_pages, int64_t table_stride,
                           int32_t* page_table, int32_t* seq_len, int32_t* ref_count, void* workspace) {
  return dspark::CacheTables{R,       num_pages, page_size, max_pages, table_stride, page_table,
                             seq_len, ref_count, static_cast<dspark::DeviceStatus*>(workspace)};
}

dspark_status take_pools(dspark::PagePools& out, int n_pools, void* const* pools, size_t page_bytes) {
  out.n = 0;
  out.page_bytes = 0;
  if (n_pools < 0) return fail(DSPARK_INVALID_ARG, "n_pools=%d is negative", n_pools);
  if (n_pools > dspark::kMaxPools)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "n_pools=%d exceeds %d", n_pools, dspark::kMaxPools);
  if (n_pools == 0) return DSPARK_OK;
  CHECK_PTR(pools);
  if (page_bytes == 0 || page_bytes % 16 != 0)
    return fail(DSPARK_INVALID_ARG, "page_bytes=%zu must be a positive multiple of 16", page_bytes);
  for (int i = 0; i < n_pools; ++i) {
    CHECK_PTR(pools[i]);
    CHECK_ALIGN(pools[i], 16);
    out.base[i] = pools[i];
  }
  out.n = n_pools;
  out.page_bytes = page_bytes;
  return DSPARK_OK;
}

dspark_status check_rows(int D, int dtype_io, int dtype_kv, const void* k_pool, const void* v_pool,
                         int64_t page_stride, int64_t head_stride, int64_t token_stride, const float* k_scale,
                         const float* v_scale) {
  if (D < 16 || D > 256 || D % 16 != 0)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "D=%d must be a multiple of 16 in 16..256", D);
  if (!is_half_type(dtype_io)) return fail(DSPARK_INVALID_ARG, "bad dtype %d: bf16 or fp16 is wanted", dtype_io);
  if (dtype_kv != dtype_io && dtype_kv != DSPARK_E4M3)
    return fail(DSPARK_INVALID_ARG, "dtype_kv=%d must be %d or DSPARK_E4M3", dtype_kv, dtype_io);
  CHECK_PTR(k_pool);
  CHECK_PTR(v_pool);
  CHECK_ALIGN(k_pool, 16);
  CHECK_ALIGN(v_pool, 16);
  const int64_t unit = 16 / (int64_t)size_of(dtype_kv);
  if (page_stride % unit || head_stride % unit || token_stride % unit || page_stride < 0 || head_stride < 0 ||
      token_stride < 0)
    return fail(DSPARK_INVALID_ARG, "the pools' strides must be multiples of 16 bytes");
  if (dtype_kv == DSPARK_E4M3) {
    CHECK_PTR(k_scale);
    CHECK_PTR(v_scale);
  } else if (k_scale != nullptr || v_scale != nullptr) {
    return fail(DSPARK_INVALID_ARG, "k_scale and v_scale go with an e4m3 cache");
  }
  return DSPARK_OK;
}

dspark_status check_strided(const void* p, int64_t stride_token, int64_t stride_head, const char* what) {
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0)
    return fail(DSPARK_INVALID_ARG, "%s must start on a 16-byte boundary", what);
  if (stride_token % 8 || stride_head % 8 || stride_token < 0 || stride_head < 0)
    return fail(DSPARK_INVALID_ARG, "the strides of %s must be multiples of 16 bytes", what);
  return DSPARK_OK;
}

// What both attention calls ask of their arguments (but for the bound of the queries).
dspark_status check_attention(int T, int R, int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages,
                              int64_t table_stride, int window, float scale) {
  CHECK(check_geometry(R, num_pages, page_size, max_pages, table_stride));
  if (T < 0 || Hq < 1 || Hkv < 1 || window < 0)
    return fail(DSPARK_INVALID_ARG, "sizes must be positive (T=%d Hq=%d Hkv=%d window=%d)", T, Hq, Hkv, window);
  if (Hq % Hkv != 0) return fail(DSPARK_INVALID_ARG, "Hq=%d must be a multiple of Hkv=%d", Hq, Hkv);
  if (Hq / Hkv > 64) return fail(DSPARK_UNSUPPORTED_SHAPE, "Hq / Hkv = %d exceeds 64", Hq / Hkv);
  if ((int64_t)T * Hq > INT32_MAX) return fail(DSPARK_UNSUPPORTED_SHAPE, "T * Hq must be below 2^31");
  if (!isfinite(scale)) return fail(DSPARK_INVALID_ARG, "scale must be finite");
  return DSPARK_OK;
}

// --------------------------------------------------------------------------- rotary positions

dspark_status check_turn(int D, int rot_dim, int interleaved, const int64_t* rates, float magnitude) {
  if (rot_dim < 2 || rot_dim > D || rot_dim % 2 != 0)
    return fail(DSPARK_INVALID_ARG, "rot_dim=%d must be even and lie in 2..D=%d", rot_dim, D);
  if (interleaved != 0 && interleaved != 1) return fail(DSPARK_INVALID_ARG, "interleaved=%d must be 0 or 1", interleaved);
  CHECK_PTR(rates);
  if (!isfinite(magnitude)) return fail(DSPARK_INVALID_ARG, "magnitude must be finite");
  return DSPARK_OK;
}

dspark_status append(int T, int R, int Hq, int Hkv, int D, int rot_dim, int interleaved, int num_pages, int page_size,
                     int max_pages, int dtype_in, int dtype_kv, const void* q, int64_t q_stride_token,
                     int64_t q_stride_head, const void* k, const void* v, int64_t in_stride_token,
                     int64_t in_stride_head, void* q_out, int64_t q_out_stride_token, int64_t q_out_stride_head,
                     void* k_pool, void* v_pool, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                     const int32_t* page_table, int64_t table_stride, const int32_t* seq_len, const int32_t* q_start,
                     const int32_t* granted, const float* k_scale, const float* v_scale, const int64_t* rates,
                     float magnitude, void* workspace, size_t ws_bytes, void* stream) {
  CHECK(check_geometry(R, num_pages, page_size, max_pages, table_stride));
  if (T < 0 || Hq < 0 || Hkv < 1)
    return fail(DSPARK_INVALID_ARG, "sizes must be positive (T=%d Hq=%d Hkv=%d)", T, Hq, Hkv);
  CHECK(check_rows(D, dtype_in, dtype_kv, k_pool, v_pool, page_stride, head_stride, token_stride, k_scale, v_scale));
  CHECK(check_turn(D, rot_dim, interleaved, rates, magnitude));
  if (((int64_t)Hq + 2 * (int64_t)Hkv) * D > (1 << 26))
    return fail(DSPARK_UNSUPPORTED_SHAPE, "(Hq + 2 Hkv) * D must be at most 2^26");
  if ((page_stride == 0 && num_pages > 1) || (head_stride == 0 && Hkv > 1) || (token_stride == 0 && page_size > 1))
    return fail(DSPARK_INVALID_ARG, "rows of a pool that is written to must not lie on one another");
  CHECK_PTR(page_table);
  CHECK_PTR(seq_len);
  CHECK_PTR(q_start);
  CHECK(check_workspace(workspace, ws_bytes, 256));
  if (T == 0) return DSPARK_OK;
  CHECK_PTR(k);
  CHECK_PTR(v);
  CHECK(check_strided(k, in_stride_token, in_stride_head, "k"));
  CHECK(check_strided(v, in_stride_token, in_stride_head, "v"));
  if (Hq > 0) {
    CHECK_PTR(q);
    CHECK_PTR(q_out);
    CHECK(check_strided(q, q_stride_token, q_stride_head, "q"));
    CHECK(check_strided(q_out, q_out_stride_token, q_out_stride_head, "q_out"));
    if ((q_out_stride_token < D && T > 1) || (q_out_stride_head < D && Hq > 1))
      return fail(DSPARK_INVALID_ARG, "rows of q_out must not lie on one another");
    if (q_out == q && ((T > 1 && q_out_stride_token != q_stride_token) || (Hq > 1 && q_out_stride_head != q_stride_head)))
      return fail(DSPARK_INVALID_ARG, "queries turned in place have the strides of q");
  }
  dspark::AppendArgs a = {};
  a.T = T; a.R = R; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.rot = rot_dim; a.interleaved = interleaved;
  a.num_pages = num_pages; a.page_size = page_size; a.max_pages = max_pages; a.dtype_in = dtype_in; a.dtype_kv = dtype_kv;
  a.q = q; a.q_token = q_stride_token; a.q_head = q_stride_head; a.k = k; a.v = v; a.in_token = in_stride_token;
  a.in_head = in_stride_head; a.q_out = q_out; a.q_out_token = q_out_stride_token; a.q_out_head = q_out_stride_head;
  a.k_pool = k_pool; a.v_pool = v_pool; a.page_stride = page_stride; a.head_stride = head_stride;
  a.token_stride = token_stride; a.page_table = page_table; a.table_stride = table_stride; a.seq_len = seq_len;
  a.q_start = q_start; a.granted = granted; a.k_scale = k_scale; a.v_scale = v_scale; a.rates = rates;
  a.magnitude = magnitude; a.status = static_cast<dspark::DeviceStatus*>(workspace);
  return launched(dspark::launch_cache_append(a, static_cast<cudaStream_t>(stream)), "cache_append");
}

}  // namespace

extern "C" {

dspark_status dspark_token_logprobs(int N, int V, int64_t row_stride, int dtype, const void* logits,
                                    const int32_t* tokens, float temperature, int top_k, float* logprob_out,
                                    float* entropy_out, float* lse_out, int32_t* top_ids_out,
                                    float* top_logprobs_out, void* stream) {
  CHECK(check_logits(N, V, row_stride, dtype, temperature));
  if (top_k < 0 || top_k > V) return fail(DSPARK_INVALID_ARG, "top_k=%d must lie in 0..V", top_k);
  if (top_k > dspark::kMaxTopK) return fail(DSPARK_UNSUPPORTED_SHAPE, "top_k=%d exceeds %d", top_k, dspark::kMaxTopK);
  if (N == 0) return DSPARK_OK;
  CHECK_PTR(logits);
  CHECK_ALIGN(logits, size_of(dtype));
  CHECK_PTR(tokens);
  CHECK_PTR(logprob_out);
  CHECK_PTR(entropy_out);
  CHECK_PTR(lse_out);
  if (top_k > 0) {
    CHECK_PTR(top_ids_out);
    CHECK_PTR(top_logprobs_out);
  }
  dspark::LogprobArgs a = {};
  a.N = N; a.V = V; a.row_stride = row_stride; a.dtype = dtype; a.logits = logits; a.tokens = tokens;
  a.inv_temp = 1.f / temperature; a.top_k = top_k; a.logprob_out = logprob_out; a.entropy_out = entropy_out;
  a.lse_out = lse_out; a.top_ids_out = top_ids_out; a.top_logprobs_out = top_logprobs_out;
  return launched(dspark::launch_token_logprobs(a, static_cast<cudaStream_t>(stream)), "token_logprobs");
}

dspark_status dspark_token_logprobs_backward(int N, int V, int64_t row_stride, int64_t grad_stride, int dtype,
                                             const void* logits, const int32_t* tokens, float temperature,
                                             const float* lse, const float* entropy, const float* grad_logprob,
                                             const float* grad_entropy, void* grad_out, void* stream) {
  CHECK(check_logits(N, V, row_stride, dtype, temperature));
  if (grad_stride < V) return fail(DSPARK_INVALID_ARG, "grad_stride %lld is below V=%d", (long long)grad_stride, V);
  if (N == 0) return DSPARK_OK;
  CHECK_PTR(logits);
  CHECK_ALIGN(logits, size_of(dtype));
  CHECK_PTR(tokens);
  CHECK_PTR(lse);
  CHECK_PTR(entropy);
  CHECK_PTR(grad_logprob);
  CHECK_PTR(grad_out);
  CHECK_ALIGN(grad_out, size_of(dtype));
  if (grad_out == logits && grad_stride != row_stride)
    return fail(DSPARK_INVALID_ARG, "a gradient in the logits' place has the logits' row stride");
  dspark::LogprobArgs a = {};
  a.N = N; a.V = V; a.row_stride = row_stride; a.grad_stride = grad_stride; a.dtype = dtype; a.logits = logits;
  a.tokens = tokens; a.inv_temp = 1.f / temperature; a.lse = lse; a.entropy = entropy;
  a.grad_logprob = grad_logprob; a.grad_entropy = grad_entropy; a.grad_out = grad_out;
  return launched(dspark::launch_token_logprobs_backward(a, static_cast<cudaStream_t>(stream)),
                  "token_logprobs_backward");
}

size_t dspark_cache_workspace_size(int R, int num_pages) {
  if (R < 1 || num_pages < 1 || R > dspark::kMaxSlots || num_pages > dspark::kMaxPages) return 0;
  return cache_layout(num_pages).total;
}

dspark_status dspark_cache_fork(int F, int R, int num_pages, int page_size, int max_pages, int64_t table_stride,
                                int32_t* page_table, int32_t* seq_len, int32_t* ref_count, const int32_t* src,
                                const int32_t* dst, void* workspace, size_t ws_bytes, void* stream) {
  const dspark::CacheTables t =
      tables(R, num_pages, page_size, max_pages, table_stride, page_table, seq_len, ref_count, workspace);
  CHECK(check_tables(t, workspace, ws_bytes));
  if (F < 0 || F > R) return fail(DSPARK_INVALID_ARG, "F=%d must lie in 0..R", F);
  if (F == 0) return DSPARK_OK;
  CHECK_PTR(src);
  CHECK_PTR(dst);
  return launched(dspark::launch_cache_fork(t, F, src, dst, static_cast<cudaStream_t>(stream)), "cache_fork");
}

dspark_status dspark_cache_reserve(int R, int num_pages, int page_size, int max_pages, int64_t table_stride,
                                   int32_t* page_table, int32_t* seq_len, int32_t* ref_count, const int32_t* n_new,
                                   int32_t* granted_out, int32_t* copies_out, int n_pools, void* const* pools,
                                   size_t page_bytes, void* workspace, size_t ws_bytes, void* stream) {
  const dspark::CacheTables t =
      tables(R, num_pages, page_size, max_pages, table_stride, page_table, seq_len, ref_count, workspace);
  CHECK(check_tables(t, workspace, ws_bytes));
  CHECK_PTR(n_new);
  CHECK_PTR(granted_out);
  CHECK_PTR(copies_out);
  dspark::PagePools p;
  CHECK(take_pools(p, n_pools, pools, page_bytes));
  return launched(
      dspark::launch_cache_reserve(t, n_new, granted_out, copies_out, p, static_cast<cudaStream_t>(stream)),
      "cache_reserve");
}

dspark_status dspark_cache_write(int T, int R, int Hkv, int D, int num_pages, int page_size, int max_pages,
                                 int dtype_in, int dtype_kv, const void* k, const void* v, int64_t in_stride_token,
                                 int64_t in_stride_head, void* k_pool, void* v_pool, int64_t page_stride,
                                 int64_t head_stride, int64_t token_stride, const int32_t* page_table,
                                 int64_t table_stride, const int32_t* seq_len, const int32_t* q_start,
                                 const int32_t* granted, const float* k_scale, const float* v_scale, void* workspace,
                                 size_t ws_bytes, void* stream) {
  CHECK(check_geometry(R, num_pages, page_size, max_pages, table_stride));
  if (T < 0 || Hkv < 1) return fail(DSPARK_INVALID_ARG, "sizes must be positive (T=%d Hkv=%d)", T, Hkv);
  CHECK(check_rows(D, dtype_in, dtype_kv, k_pool, v_pool, page_stride, head_stride, token_stride, k_scale, v_scale));
  if ((page_stride == 0 && num_pages > 1) || (head_stride == 0 && Hkv > 1) || (token_stride == 0 && page_size > 1))
    return fail(DSPARK_INVALID_ARG, "rows of a pool that is written to must not lie on one another");
  CHECK_PTR(page_table);
  CHECK_PTR(seq_len);
  CHECK_PTR(q_start);
  CHECK(check_workspace(workspace, ws_bytes, 256));
  if (T == 0) return DSPARK_OK;
  CHECK_PTR(k);
  CHECK_PTR(v);
  CHECK(check_strided(k, in_stride_token, in_stride_head, "k"));
  CHECK(check_strided(v, in_stride_token, in_stride_head, "v"));
  dspark::CacheWriteArgs a = {};
  a.T = T; a.R = R; a.Hkv = Hkv; a.D = D; a.num_pages = num_pages; a.page_size = page_size; a.max_pages = max_pages;
  a.dtype_in = dtype_in; a.dtype_kv = dtype_kv; a.k = k; a.v = v; a.in_stride_token = in_stride_token;
  a.in_stride_head = in_stride_head; a.k_pool = k_pool; a.v_pool = v_pool; a.page_stride = page_stride;
  a.head_stride = head_stride; a.token_stride = token_stride; a.page_table = page_table;
  a.table_stride = table_stride; a.seq_len = seq_len; a.q_start = q_start; a.granted = granted; a.k_scale = k_scale;
  a.v_scale = v_scale; a.status = static_cast<dspark::DeviceStatus*>(workspace);
  return launched(dspark::launch_cache_write(a, static_cast<cudaStream_t>(stream)), "cache_write");
}

dspark_status dspark_cache_truncate(int R, int num_pages, int page_size, int max_pages, int64_t table_stride,
                                    int32_t* page_table, int32_t* seq_len, int32_t* ref_count,
                                    const int32_t* new_len, void* workspace, size_t ws_bytes, void* stream) {
  const dspark::CacheTables t =
      tables(R, num_pages, page_size, max_pages, table_stride, page_table, seq_len, ref_count, workspace);
  CHECK(check_tables(t, workspace, ws_bytes));
  CHECK_PTR(new_len);
  return launched(dspark::launch_cache_truncate(t, new_len, static_cast<cudaStream_t>(stream)), "cache_truncate");
}

dspark_status dspark_cache_compact(int R, int num_pages, int page_size, int max_pages, int64_t table_stride,
                                   int32_t* page_table, const int32_t* seq_len, int32_t* ref_count,
                                   int32_t* n_moves_out, int n_pools, void* const* pools, size_t page_bytes,
                                   void* workspace, size_t ws_bytes, void* stream) {
  const dspark::CacheTables t = tables(R, num_pages, page_size, max_pages, table_stride, page_table,
                                       const_cast<int32_t*>(seq_len), ref_count, workspace);
  CHECK(check_tables(t, workspace, ws_bytes));
  CHECK_PTR(n_moves_out);
  dspark::PagePools p;
  CHECK(take_pools(p, n_pools, pools, page_bytes));
  const CacheLayout L = cache_layout(num_pages);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const dspark::CompactLists lists = {
      reinterpret_cast<int32_t*>(ws + L.counts), reinterpret_cast<int32_t*>(ws + L.hole),
      reinterpret_cast<int32_t*>(ws + L.mover), reinterpret_cast<int32_t*>(ws + L.rank)};
  return launched(dspark::launch_cache_compact(t, lists, n_moves_out, p, static_cast<cudaStream_t>(stream)),
                  "cache_compact");
}

size_t dspark_paged_attention_workspace_size(int T, int R, int Hq, int Hkv, int D, int max_q) {
  if (T < 0 || R < 1 || R > dspark::kMaxSlots || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 64 || D < 16 ||
      D > 256 || D % 16 != 0 || max_q < 1 || max_q > dspark::kMaxQueries)
    return 0;
  return 256 + dspark::paged_attention_scratch(T, R, Hq, Hkv, D, max_q);
}

dspark_status dspark_paged_attention(int T, int R, int Hq, int Hkv, int D, int num_pages, int page_size,
                                     int max_pages, int max_q, int dtype_q, int dtype_kv, const void* q,
                                     int64_t q_stride_token, int64_t q_stride_head, const void* k_pool,
                                     const void* v_pool, int64_t page_stride, int64_t head_stride,
                                     int64_t token_stride, const int32_t* page_table, int64_t table_stride,
                                     const int32_t* seq_len, const int32_t* q_start, float scale,
                                     const float* k_scale, const float* v_scale, int window, void* out,
                                     float* lse_out, void* workspace, size_t ws_bytes, void* stream) {
  return dspark_paged_attention_granted(T, R, Hq, Hkv, D, num_pages, page_size, max_pages, max_q, dtype_q, dtype_kv, q,
                                        q_stride_token, q_stride_head, k_pool, v_pool, page_stride, head_stride,
                                        token_stride, page_table, table_stride, seq_len, q_start, nullptr, scale,
                                        k_scale, v_scale, window, out, lse_out, workspace, ws_bytes, stream);
}

dspark_status dspark_paged_attention_granted(int T, int R, int Hq, int Hkv, int D, int num_pages, int page_size,
                                             int max_pages, int max_q, int dtype_q, int dtype_kv, const void* q,
                                             int64_t q_stride_token, int64_t q_stride_head, const void* k_pool,
                                             const void* v_pool, int64_t page_stride, int64_t head_stride,
                                             int64_t token_stride, const int32_t* page_table, int64_t table_stride,
                                             const int32_t* seq_len, const int32_t* q_start, const int32_t* granted,
                                             float scale, const float* k_scale, const float* v_scale, int window,
                                             void* out, float* lse_out, void* workspace, size_t ws_bytes,
                                             void* stream) {
  CHECK(check_attention(T, R, Hq, Hkv, D, num_pages, page_size, max_pages, table_stride, window, scale));
  if (max_q < 1) return fail(DSPARK_INVALID_ARG, "max_q=%d must be positive", max_q);
  if (max_q > dspark::kMaxQueries)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "max_q=%d exceeds %d", max_q, dspark::kMaxQueries);
  CHECK(check_rows(D, dtype_q, dtype_kv, k_pool, v_pool, page_stride, head_stride, token_stride, k_scale, v_scale));
  CHECK_PTR(page_table);
  CHECK_PTR(seq_len);
  CHECK_PTR(q_start);
  CHECK(check_workspace(workspace, ws_bytes, dspark_paged_attention_workspace_size(T, R, Hq, Hkv, D, max_q)));
  if (T == 0) return DSPARK_OK;
  CHECK_PTR(q);
  CHECK_PTR(out);
  CHECK_ALIGN(out, 16);
  CHECK(check_strided(q, q_stride_token, q_stride_head, "q"));
  dspark::AttentionArgs a = {};
  a.T = T; a.R = R; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.D = D; a.num_pages = num_pages;
  a.page_size = page_size; a.max_pages = max_pages; a.max_q = max_q; a.dtype_q = dtype_q; a.dtype_kv = dtype_kv; a.q = q;
  a.q_stride_token = q_stride_token; a.q_stride_head = q_stride_head; a.k_pool = k_pool; a.v_pool = v_pool;
  a.page_stride = page_stride; a.head_stride = head_stride; a.token_stride = token_stride;
  a.page_table = page_table; a.table_stride = table_stride; a.seq_len = seq_len; a.q_start = q_start;
  a.granted = granted; a.scale = scale; a.k_scale = k_scale; a.v_scale = v_scale; a.out = out; a.lse_out = lse_out;
  // a window as long as the table hides nothing; kept below it, position - window stays within 32 bits
  a.window = window < (int64_t)max_pages * page_size ? window : 0;
  a.status = static_cast<dspark::DeviceStatus*>(workspace);
  return launched(dspark::launch_paged_attention(a, static_cast<unsigned char*>(workspace) + 256,
                                                 static_cast<cudaStream_t>(stream)),
                  "paged_attention");
}

size_t dspark_chunk_attention_workspace_size(int T, int R, int Hq, int Hkv, int D) {
  if (T < 0 || R < 1 || R > dspark::kMaxSlots || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 64 || D < 16 ||
      D > 256 || D % 16 != 0)
    return 0;
  return 256 + dspark::chunk_attention_scratch(Hq, Hkv, D);
}

dspark_status dspark_chunk_attention(int T, int R, int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages,
                                     int dtype_q, int dtype_kv, const void* q, int64_t q_stride_token,
                                     int64_t q_stride_head, const void* k_pool, const void* v_pool, int64_t page_stride,
                                     int64_t head_stride, int64_t token_stride, const int32_t* page_table,
                                     int64_t table_stride, const int32_t* seq_len, const int32_t* q_start,
                                     const int32_t* granted, float scale, const float* k_scale, const float* v_scale,
                                     int window, void* out, float* lse_out, void* workspace, size_t ws_bytes,
                                     void* stream) {
  CHECK(check_attention(T, R, Hq, Hkv, D, num_pages, page_size, max_pages, table_stride, window, scale));
  if (window >= (int64_t)max_pages * page_size) window = 0;  // (all that a table can hold)
  // (a query that lies as far before its context as there are rows sees nothing: its window begins further back yet)
  if ((int64_t)T + window >= ((int64_t)1 << 31) - 1024)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "T + window = %lld must be below 2^31 - 1024", (long long)T + window);
  CHECK(check_rows(D, dtype_q, dtype_kv, k_pool, v_pool, page_stride, head_stride, token_stride, k_scale, v_scale));
  CHECK_PTR(page_table);
  CHECK_PTR(seq_len);
  CHECK_PTR(q_start);
  CHECK(check_workspace(workspace, ws_bytes, dspark_chunk_attention_workspace_size(T, R, Hq, Hkv, D)));
  if (T == 0) return DSPARK_OK;
  CHECK_PTR(q);
  CHECK_PTR(out);
  CHECK_ALIGN(out, 16);
  CHECK(check_strided(q, q_stride_token, q_stride_head, "q"));
  dspark::AttentionArgs a = {};
  a.T = T; a.R = R; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.D = D; a.num_pages = num_pages;
  a.page_size = page_size; a.max_pages = max_pages; a.max_q = T; a.dtype_q = dtype_q; a.dtype_kv = dtype_kv; a.q = q;
  a.q_stride_token = q_stride_token; a.q_stride_head = q_stride_head; a.k_pool = k_pool; a.v_pool = v_pool;
  a.page_stride = page_stride; a.head_stride = head_stride; a.token_stride = token_stride;
  a.page_table = page_table; a.table_stride = table_stride; a.seq_len = seq_len; a.q_start = q_start;
  a.granted = granted; a.scale = scale; a.k_scale = k_scale; a.v_scale = v_scale; a.out = out; a.lse_out = lse_out;
  a.window = window;
  a.status = static_cast<dspark::DeviceStatus*>(workspace);
  return launched(dspark::launch_chunk_attention(a, static_cast<unsigned char*>(workspace) + 256,
                                                 static_cast<cudaStream_t>(stream)),
                  "chunk_attention");
}

dspark_status dspark_rotary(int T, int H, int D, int rot_dim, int dtype, int interleaved, int inverse, const void* x,
                            int64_t x_stride_token, int64_t x_stride_head, const int32_t* positions,
                            const int64_t* rates, float magnitude, void* out, int64_t out_stride_token,
                            int64_t out_stride_head, void* stream) {
  if (T < 0 || H < 1 || D < 1) return fail(DSPARK_INVALID_ARG, "sizes must be positive (T=%d H=%d D=%d)", T, H, D);
  if (!is_float_type(dtype)) return fail(DSPARK_INVALID_ARG, "bad dtype %d", dtype);
  CHECK(check_turn(D, rot_dim, interleaved, rates, magnitude));
  if (inverse != 0 && inverse != 1) return fail(DSPARK_INVALID_ARG, "inverse=%d must be 0 or 1", inverse);
  if (D > dspark::kMaxRotaryDim)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "D=%d exceeds %d", D, dspark::kMaxRotaryDim);
  if ((int64_t)H * D > (1 << 26)) return fail(DSPARK_UNSUPPORTED_SHAPE, "H * D must be at most 2^26");
  if (x_stride_token < 0 || x_stride_head < 0 || out_stride_token < 0 || out_stride_head < 0)
    return fail(DSPARK_INVALID_ARG, "strides must not be negative");
  if ((out_stride_token < D && T > 1) || (out_stride_head < D && H > 1))
    return fail(DSPARK_INVALID_ARG, "rows of out must not lie on one another");
  if (T == 0) return DSPARK_OK;
  CHECK_PTR(x);
  CHECK_PTR(positions);
  CHECK_PTR(out);
  CHECK_ALIGN(x, size_of(dtype));
  CHECK_ALIGN(out, size_of(dtype));
  if (out == x && ((T > 1 && out_stride_token != x_stride_token) || (H > 1 && out_stride_head != x_stride_head)))
    return fail(DSPARK_INVALID_ARG, "a result in the place of x has the strides of x");
  const dspark::RotaryArgs a = {T, H, D, rot_dim, dtype, interleaved, inverse, x, x_stride_token, x_stride_head, positions,
                                rates, magnitude, out, out_stride_token, out_stride_head};
  return launched(dspark::launch_rotary(a, static_cast<cudaStream_t>(stream)), "rotary");
}

dspark_status dspark_cache_append(int T, int R, int Hq, int Hkv, int D, int rot_dim, int interleaved, int num_pages,
                                  int page_size, int max_pages, int dtype_in, int dtype_kv, const void* q,
                                  int64_t q_stride_token, int64_t q_stride_head, const void* k, const void* v,
                                  int64_t in_stride_token, int64_t in_stride_head, void* q_out,
                                  int64_t q_out_stride_token, int64_t q_out_stride_head, void* k_pool, void* v_pool,
                                  int64_t page_stride, int64_t head_stride, int64_t token_stride,
                                  const int32_t* page_table, int64_t table_stride, const int32_t* seq_len,
                                  const int32_t* q_start, const int32_t* granted, const float* k_scale,
                                  const float* v_scale, const int64_t* rates, float magnitude, void* workspace,
                                  size_t ws_bytes, void* stream) {
  if (rot_dim >= 2 && rot_dim <= D && rot_dim % 2 == 0 && rot_dim % 16 != 0)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "rot_dim=%d must be a multiple of 16 (dspark_cache_append_any takes it)", rot_dim);
  return append(T, R, Hq, Hkv, D, rot_dim, interleaved, num_pages, page_size, max_pages, dtype_in, dtype_kv, q,
                q_stride_token, q_stride_head, k, v, in_stride_token, in_stride_head, q_out, q_out_stride_token,
                q_out_stride_head, k_pool, v_pool, page_stride, head_stride, token_stride, page_table, table_stride,
                seq_len, q_start, granted, k_scale, v_scale, rates, magnitude, workspace, ws_bytes, stream);
}

dspark_status dspark_cache_append_any(int T, int R, int Hq, int Hkv, int D, int rot_dim, int interleaved, int num_pages,
                                      int page_size, int max_pages, int dtype_in, int dtype_kv, const void* q,
                                      int64_t q_stride_token, int64_t q_stride_head, const void* k, const void* v,
                                      int64_t in_stride_token, int64_t in_stride_head, void* q_out,
                                      int64_t q_out_stride_token, int64_t q_out_stride_head, void* k_pool, void* v_pool,
                                      int64_t page_stride, int64_t head_stride, int64_t token_stride,
                                      const int32_t* page_table, int64_t table_stride, const int32_t* seq_len,
                                      const int32_t* q_start, const int32_t* granted, const float* k_scale,
                                      const float* v_scale, const int64_t* rates, float magnitude, void* workspace,
                                      size_t ws_bytes, void* stream) {
  return append(T, R, Hq, Hkv, D, rot_dim, interleaved, num_pages, page_size, max_pages, dtype_in, dtype_kv, q,
                q_stride_token, q_stride_head, k, v, in_stride_token, in_stride_head, q_out, q_out_stride_token,
                q_out_stride_head, k_pool, v_pool, page_stride, head_stride, token_stride, page_table, table_stride,
                seq_len, q_start, granted, k_scale, v_scale, rates, magnitude, workspace, ws_bytes, stream);
}

dspark_status dspark_adjust_logits(int N, int V, int R, int dtype, const void* logits, int64_t row_stride,
                                   const int32_t* tokens, const int32_t* q_start, const int32_t* history,
                                   int64_t history_stride, int history_width, const int32_t* history_len,
                                   const int32_t* prompt_len, const float* repetition, const float* frequency,
                                   const float* presence, int n_bias, const int32_t* bias_ids, const float* bias,
                                   const uint32_t* mask, int64_t mask_stride, int mask_rows, const int32_t* mask_row,
                                   void* out, int64_t out_stride, void* stream) {
  if (N < 0 || V < 1 || R < 1) return fail(DSPARK_INVALID_ARG, "sizes must be positive (N=%d V=%d R=%d)", N, V, R);
  if (V > dspark::kMaxLogprobV) return fail(DSPARK_UNSUPPORTED_SHAPE, "V=%d exceeds %d", V, dspark::kMaxLogprobV);
  if (R > dspark::kMaxSlots) return fail(DSPARK_UNSUPPORTED_SHAPE, "R=%d exceeds %d", R, dspark::kMaxSlots);
  if (!is_float_type(dtype)) return fail(DSPARK_INVALID_ARG, "bad dtype %d", dtype);
  if (row_stride < V) return fail(DSPARK_INVALID_ARG, "row_stride %lld is below V=%d", (long long)row_stride, V);
  if (out_stride < V) return fail(DSPARK_INVALID_ARG, "out_stride %lld is below V=%d", (long long)out_stride, V);
  const int64_t entries = (history != nullptr ? history_width : 0) + (int64_t)N;  // (counted in 29 bits)
  if (entries >= 1 << 29)
    return fail(DSPARK_UNSUPPORTED_SHAPE, "history_width + N = %lld must be below 2^29", (long long)entries);
  if (history != nullptr) {
    if (history_width < 0 || history_stride < history_width)
      return fail(DSPARK_INVALID_ARG, "history_stride %lld is below history_width=%d", (long long)history_stride, history_width);
    CHECK_PTR(history_len);
  }
  if (n_bias < 0) return fail(DSPARK_INVALID_ARG, "n_bias=%d is negative", n_bias);
  if (n_bias > dspark::kMaxBias) return fail(DSPARK_UNSUPPORTED_SHAPE, "n_bias=%d exceeds %d", n_bias, dspark::kMaxBias);
  if (n_bias > 0) {
    CHECK_PTR(bias_ids);
    CHECK_PTR(bias);
  }
  if (mask != nullptr) {
    if (mask_rows < 0 || mask_stride < (V + 31) / 32)
      return fail(DSPARK_INVALID_ARG, "a mask has mask_rows=%d rows of at least %d words", mask_rows, (V + 31) / 32);
    if (mask_row == nullptr && mask_rows < N)
      return fail(DSPARK_INVALID_ARG, "without mask_row there is a mask row for each of the %d rows, got %d", N, mask_rows);
  } else if (mask_row != nullptr && mask_rows != 0) {  // (a mask without rows may have no address: no row goes by it)
    return fail(DSPARK_INVALID_ARG, "mask_row goes with a mask");
  }
  if (N == 0) return DSPARK_OK;
  CHECK_PTR(logits);
  CHECK_ALIGN(logits, size_of(dtype));
  CHECK_PTR(q_start);
  CHECK_PTR(out);
  CHECK_ALIGN(out, size_of(dtype));
  if (out == logits && out_stride != row_stride)
    return fail(DSPARK_INVALID_ARG, "a result in the logits' place has the logits' row stride");
  const dspark::AdjustArgs a = {N, V, R, dtype, logits, row_stride, tokens, q_start, history, history_stride, history_width,
                                history_len, prompt_len, repetition, frequency, presence, n_bias, bias_ids, bias, mask,
                                mask_stride, mask_rows, mask_row, out, out_stride};
  return launched(dspark::launch_adjust_logits(a, static_cast<cudaStream_t>(stream)), "adjust_logits");
}

}  // extern "C"
