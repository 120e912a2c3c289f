// serving.h — argument blocks and launcher declarations of the serving-side operators
// (token log probabilities, the paged cache, attention over it).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dspark {

struct DeviceStatus;

struct LogprobArgs {
  int N, V;
  int64_t row_stride, grad_stride;
  int dtype;
  const void* logits;
  const int32_t* tokens;
  float inv_temp;
  int top_k;
  float* logprob_out;
  float* entropy_out;
  float* lse_out;
  int32_t* top_ids_out;
  float* top_logprobs_out;
  // backward
  const float* lse;
  const float* entropy;
  const float* grad_logprob;
  const float* grad_entropy;
  void* grad_out;
};

constexpr int kMaxTopK = 32;
constexpr int kMaxLogprobV = 1 << 20;

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t s);
cudaError_t launch_token_logprobs_backward(const LogprobArgs& a, cudaStream_t s);

// The tables of a paged cache.
struct CacheTables {
  int R, num_pages, page_size, max_pages;
  int64_t table_stride;
  int32_t* page_table;
  int32_t* seq_len;
  int32_t* ref_count;
  DeviceStatus* status;
};

constexpr int kMaxSlots = 8192;
constexpr int kMaxPages = 1 << 22;
constexpr int kMaxPools = 512;

// Pools of which whole pages are copied; the pairs live on the device.
struct PagePools {
  int n;
  size_t page_bytes;
  void* base[kMaxPools];
};

struct CompactLists {
  int32_t* counts;  // [0]: pages in use, [1]: moves
  int32_t* hole;    // i-th free page below the number of pages in use
  int32_t* mover;   // i-th used page at or past it
  int32_t* rank;    // [num_pages] i of a moving page
};

cudaError_t launch_cache_fork(const CacheTables& t, int F, const int32_t* src, const int32_t* dst, cudaStream_t s);
cudaError_t launch_cache_reserve(const CacheTables& t, const int32_t* n_new, int32_t* granted, int32_t* copies,
                                 const PagePools& pools, cudaStream_t s);
cudaError_t launch_cache_truncate(const CacheTables& t, const int32_t* new_len, cudaStream_t s);
cudaError_t launch_cache_compact(const CacheTables& t, const CompactLists& l, int32_t* n_moves, const PagePools& pools,
                                 cudaStream_t s);

struct CacheWriteArgs {
  int T, R, Hkv, D, num_pages, page_size, max_pages, dtype_in, dtype_kv;
  const void* k;
  const void* v;
  int64_t in_stride_token, in_stride_head;
  void* k_pool;
  void* v_pool;
  int64_t page_stride, head_stride, token_stride;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* seq_len;
  const int32_t* q_start;
  const int32_t* granted;
  const float* k_scale;
  const float* v_scale;
  DeviceStatus* status;
};
cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t s);

struct AttentionArgs {
  int T, R, Hq, Hkv, G, D, num_pages, page_size, max_pages, max_q, dtype_q, dtype_kv;  // G = Hq / Hkv
  const void* q;
  int64_t q_stride_token, q_stride_head;
  const void* k_pool;
  const void* v_pool;
  int64_t page_stride, head_stride, token_stride;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* seq_len;
  const int32_t* q_start;
  const int32_t* granted;  // may be null
  float scale;
  const float* k_scale;
  const float* v_scale;
  int window;
  void* out;
  float* lse_out;
  DeviceStatus* status;
};
constexpr int kMaxQueries = 128;
size_t paged_attention_scratch(int T, int R, int Hq, int Hkv, int D, int max_q);
cudaError_t launch_paged_attention(const AttentionArgs& a, void* scratch, cudaStream_t s);

}  // namespace dspark
