// logprob.cu — log probabilities of given tokens, with entropy and the best alternatives,
// and their gradient.
#include "serving.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;
constexpr float kLargeLse = 1024.f;  // an lse beyond it is known to 2^-14 at best

template <typename T>
__device__ __forceinline__ float value(T x) { return (float)x; }

// Base-2 softmax statistics about the largest logit m: s = sum 2^u, w = sum 2^u u with
// u = (x - m) c, c = log2(e) / T.  The difference is taken before the product, so logits near
// the ends of the type's range (masks of its lowest value) neither overflow nor lose u.
struct Softmax {
  float m, s, w;
};
__device__ __forceinline__ Softmax merge(Softmax a, Softmax b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, 0.f, 0.f};
  const float da = fmaxf((a.m - m) * c, -200.f), db = fmaxf((b.m - m) * c, -200.f), fa = exp2f(da), fb = exp2f(db);
  return {m, a.s * fa + b.s * fb, (a.w + da * a.s) * fa + (b.w + db * b.s) * fb};
}

// The whole row's statistics, the same in every thread; `bad`: it holds a NaN or +inf.
template <typename T>
__device__ Softmax row_softmax(const T* row, int V, float c, Softmax* part, bool& bad) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Softmax st = {-INFINITY, 0.f, 0.f};
  bad = false;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    const float x = value(row[v]);
    bad |= !(x < INFINITY);
    st = merge(st, {x, x == -INFINITY ? 0.f : 1.f, 0.f}, c);
  }
  for (int d = 16; d; d >>= 1) {
    const Softmax o = {__shfl_xor_sync(~0u, st.m, d), __shfl_xor_sync(~0u, st.s, d), __shfl_xor_sync(~0u, st.w, d)};
    st = merge(st, o, c);
  }
  __syncthreads();
  if (lane == 0) part[warp] = st;
  bad = __syncthreads_or(bad);
  st = part[0];
  for (int w = 1; w < kThreads / 32; ++w) st = merge(st, part[w], c);
  return st;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_kernel(LogprobArgs a) {
  __shared__ Softmax part[kThreads / 32];
  __shared__ float best_v[kThreads / 32];
  __shared__ int best_i[kThreads / 32];
  const int n = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  const int tok = a.tokens[n];
  const float nan = __int_as_float(0x7FC00000);
  if (tok < 0 || tok >= a.V) {
    if (threadIdx.x == 0) a.logprob_out[n] = a.entropy_out[n] = a.lse_out[n] = nan;
    if (threadIdx.x < a.top_k) {
      a.top_ids_out[(size_t)n * a.top_k + threadIdx.x] = -1;
      a.top_logprobs_out[(size_t)n * a.top_k + threadIdx.x] = nan;
    }
    return;
  }
  const T* row = static_cast<const T*>(a.logits) + n * a.row_stride;
  const float c = a.inv_temp * kLog2e;
  bool bad;
  const Softmax st = row_softmax(row, a.V, c, part, bad);
  const bool none = st.m == -INFINITY;
  const float l2 = log2f(st.s);
  auto logprob = [&](float x) { return bad ? nan : (none ? -INFINITY : fmaf(x - st.m, a.inv_temp, -l2 * kLn2)); };
  if (threadIdx.x == 0) {
    a.logprob_out[n] = logprob(value(row[tok]));
    a.entropy_out[n] = bad ? nan : (none ? 0.f : (l2 - st.w / st.s) * kLn2);
    a.lse_out[n] = bad ? nan : (none ? -INFINITY : fmaf(st.m, a.inv_temp, l2 * kLn2));
  }
  float last_v = INFINITY;
  int last_i = -1;
  for (int k = 0; k < a.top_k; ++k) {  // the best element after the last one taken
    float bv = -INFINITY;
    int bi = a.V;
    for (int v = threadIdx.x; v < a.V; v += kThreads) {
      const float x = value(row[v]);
      const bool after = x < last_v || (x == last_v && v > last_i);
      if (after && (x > bv || bi == a.V)) bv = x, bi = v;
    }
    for (int d = 16; d; d >>= 1) {
      const float ov = __shfl_xor_sync(~0u, bv, d);
      const int oi = __shfl_xor_sync(~0u, bi, d);
      if (oi < a.V && (bi == a.V || ov > bv || (ov == bv && oi < bi))) bv = ov, bi = oi;
    }
    __syncthreads();
    if (lane == 0) best_v[warp] = bv, best_i[warp] = bi;
    __syncthreads();
    bv = best_v[0], bi = best_i[0];
    for (int w = 1; w < kThreads / 32; ++w)
      if (best_i[w] < a.V && (bi == a.V || best_v[w] > bv || (best_v[w] == bv && best_i[w] < bi)))
        bv = best_v[w], bi = best_i[w];
    last_v = bv, last_i = bi;
    if (threadIdx.x == 0) {
      a.top_ids_out[(size_t)n * a.top_k + k] = bad ? -1 : bi;
      a.top_logprobs_out[(size_t)n * a.top_k + k] = logprob(bv);
    }
  }
}

template <typename T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_backward_kernel(LogprobArgs a) {
  griddep_wait();
  const int n = blockIdx.x, tok = a.tokens[n];
  const T* row = static_cast<const T*>(a.logits) + n * a.row_stride;
  T* out = static_cast<T*>(a.grad_out) + n * a.grad_stride;
  const float lse = a.lse[n], H = a.entropy[n];
  const bool none = tok < 0 || tok >= a.V || lse == -INFINITY;
  const float gl = a.grad_logprob[n], ge = a.grad_entropy ? a.grad_entropy[n] : 0.f;
  // ln p = (x - at) / T - log_sum.  A large lse (masks of the type's lowest value in the whole
  // row) has no digits left for the sum beside the maximum: the two are taken again.
  float at = 0.f, log_sum = 0.f;
  __shared__ Softmax part[kThreads / 32];
  const bool apart = !none && fabsf(lse) > kLargeLse;
  if (apart) {
    bool bad;
    const Softmax st = row_softmax(row, a.V, a.inv_temp * kLog2e, part, bad);
    at = st.m;
    log_sum = log2f(st.s) * kLn2;
  }
  for (int v = threadIdx.x; v < a.V; v += kThreads) {
    float d = 0.f;
    if (!none) {
      const float x = value(row[v]);
      const float lp = apart ? (x - at) * a.inv_temp - log_sum : fmaf(x, a.inv_temp, -lse);
      const float p = exp2f(lp * kLog2e);
      d = -p * gl - (p == 0.f ? 0.f : ge * p * (lp + H));
      if (v == tok) d += gl;
      d *= a.inv_temp;
    }
    out[v] = rounded<T>(d);
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t s) {
  auto* k = a.dtype == DSPARK_F32 ? logprob_kernel<float>
                                  : (a.dtype == DSPARK_BF16 ? logprob_kernel<__nv_bfloat16> : logprob_kernel<__half>);
  return launch_chained(k, dim3(a.N), dim3(kThreads), 0, s, 1, a);
}

cudaError_t launch_token_logprobs_backward(const LogprobArgs& a, cudaStream_t s) {
  auto* k = a.dtype == DSPARK_F32
                ? logprob_backward_kernel<float>
                : (a.dtype == DSPARK_BF16 ? logprob_backward_kernel<__nv_bfloat16> : logprob_backward_kernel<__half>);
  return launch_chained(k, dim3(a.N), dim3(kThreads), 0, s, 1, a);
}

}  // namespace dspark
