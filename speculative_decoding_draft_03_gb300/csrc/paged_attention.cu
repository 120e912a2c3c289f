// paged_attention.cu — attention of each request's last tokens over its paged key-value cache.
#include "serving.cuh"

namespace dspark {
namespace {

enum { kBadLen = 50, kBadPage = 51, kBadQueries = 52 };

template <typename T>
__device__ __forceinline__ float value(const T* p) { return (float)*p; }

template <typename TQ, typename TKV>
__global__ void __launch_bounds__(128) attention_kernel(AttentionArgs a) {
  griddep_wait();
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (long long)a.T * a.Hq) return;
  const int t = (int)(w / a.Hq), hq = (int)(w % a.Hq), h = hq / (a.Hq / a.Hkv);
  const int r = upper_bound(a.q_start, a.R + 1, t) - 1;
  if (r < 0 || r >= a.R) return;
  const int n = a.q_start[r + 1] - a.q_start[r], i = t - a.q_start[r];
  const int len = a.seq_len[r];
  if (n > a.max_q || i >= n || a.q_start[r] < 0 || a.q_start[r + 1] > a.T || len < 0 ||
      len > a.max_pages * a.page_size) {
    if (lane == 0) report_bad_input(a.status, kBadQueries);
    return;
  }
  const int last = len - n + i, first = a.window > 0 ? max(0, last - a.window + 1) : 0;
  constexpr int kPer = 8;
  float q[kPer], o[kPer];
  const float c = a.scale * (a.k_scale ? a.k_scale[h] : 1.f);
  for (int e = 0; e < kPer; ++e) {
    const int d = lane + 32 * e;
    q[e] = d < a.D ? value(static_cast<const TQ*>(a.q) + t * a.q_stride_token + hq * a.q_stride_head + d) : 0.f;
    o[e] = 0.f;
  }
  float m = -INFINITY, s = 0.f;
  for (int j = first; j <= last; ++j) {
    const int page = a.page_table[r * a.table_stride + j / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) report_bad_input(a.status, kBadPage);
      continue;
    }
    const int64_t at = page * a.page_stride + h * a.head_stride + (j % a.page_size) * a.token_stride;
    const TKV* k = static_cast<const TKV*>(a.k_pool) + at;
    const TKV* v = static_cast<const TKV*>(a.v_pool) + at;
    float x = 0.f;
    for (int e = 0; e < kPer; ++e)
      if (lane + 32 * e < a.D) x = fmaf(q[e], value(k + lane + 32 * e), x);
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    x *= c;
    const float m2 = fmaxf(m, x);
    const float f = m2 == -INFINITY ? 1.f : expf(m - m2), p = x == -INFINITY ? 0.f : expf(x - m2);
    s = s * f + p;
    for (int e = 0; e < kPer; ++e)
      if (lane + 32 * e < a.D) o[e] = fmaf(p, value(v + lane + 32 * e), o[e] * f);
    m = m2;
  }
  const float g = s == 0.f ? 0.f : (a.v_scale ? a.v_scale[h] : 1.f) / s;
  for (int e = 0; e < kPer; ++e)
    if (lane + 32 * e < a.D)
      static_cast<TQ*>(a.out)[((size_t)t * a.Hq + hq) * a.D + lane + 32 * e] = (TQ)(s == 0.f ? 0.f : o[e] * g);
  if (lane == 0 && a.lse_out) a.lse_out[(size_t)t * a.Hq + hq] = s == 0.f ? -INFINITY : m + logf(s);
}

}  // namespace

size_t paged_attention_scratch(int, int, int, int, int, int) { return 0; }

cudaError_t launch_paged_attention(const AttentionArgs& a, void*, cudaStream_t s) {
  const dim3 grid((unsigned)(((long long)a.T * a.Hq + 3) / 4));
  const bool q8 = a.dtype_kv == DSPARK_E4M3;
  auto* k = a.dtype_q == DSPARK_BF16
                ? (q8 ? attention_kernel<__nv_bfloat16, __nv_fp8_e4m3> : attention_kernel<__nv_bfloat16, __nv_bfloat16>)
                : (q8 ? attention_kernel<__half, __nv_fp8_e4m3> : attention_kernel<__half, __half>);
  return launch_chained(k, grid, dim3(128), 0, s, 1, a);
}

}  // namespace dspark
