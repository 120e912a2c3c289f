// adjust.cu — logits adjusted before a token is taken from them: penalties for what a request has
// seen and answered, biases, and grammar masks.
//
// For row i of a slot's block, over the sequence history ++ tokens fed in up to row i (entries below
// prompt_len are the prompt's, the others answers):
//   x' = x / rho if x > 0 else x rho, for an id that is in the sequence;
//   x' -= frequency n + presence 1[n > 0], n: how often the id was answered;  x' += bias;
//   x' = -inf where the row's mask has a 0.
//   * A CTA takes a slice of the ids of one slot, for all the slot's rows: it counts the whole history's
//     ids of its slice in shared memory (a word per id: answers, and a bit for the prompt), then streams
//     its slice of the rows, one after the other, adding each row's own token before it.  A bit per id
//     says whether a count or a bias is there at all, so that the rest is a copy.
//   * In place, pieces that nothing touches are neither read nor written.
// What bounds it: device memory (each logit is read and written once), and, where histories are long
// against a slice's rows, the counting (every slice reads the whole history, from L2).
#include <algorithm>

#include "serving.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;  // rows that share one count, at most
constexpr uint32_t kPrompt = 0x80000000u;

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }

// n bits (up to 32) of a bit array from bit `at` on; words past the last are 0.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int count, int at) {
  const int w = at >> 5;
  const uint32_t lo = words[w], hi = w + 1 < count ? words[w + 1] : 0u;
  return __funnelshift_r(lo, hi, at & 31);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ AdjustArgs a, int slice) {
  extern __shared__ __align__(16) uint32_t smem[];
  constexpr int E = 16 / (int)sizeof(T);
  const int tid = threadIdx.x, r = blockIdx.y, v0 = blockIdx.x * slice, nv = min(slice, a.V - v0);
  const int words = (slice + 31) / 32;
  uint32_t* counts = smem;                                           // [slice]
  float* biases = reinterpret_cast<float*>(smem + slice);            // [slice], where there are any
  uint32_t* touched = smem + (a.n_bias > 0 ? 2 * slice : slice);     // [words] a bit per id
  griddep_wait();
  griddep_allow_next();
  const int q0 = min(max(a.q_start[r], 0), a.N), q1 = min(max(a.q_start[r + 1], q0), a.N);
  const int hist = a.history == nullptr ? 0 : min(max(a.history_len[r], 0), a.history_width);
  const int prompt = a.prompt_len == nullptr ? 0 : a.prompt_len[r];
  const float rho = a.repetition == nullptr ? 1.f : a.repetition[r];
  const float freq = a.frequency == nullptr ? 0.f : a.frequency[r], pres = a.presence == nullptr ? 0.f : a.presence[r];
  const int32_t* history = a.history + r * a.history_stride;

  auto count = [&](int id, bool answered) {  // (several threads may count the same id)
    const uint32_t at = (uint32_t)(id - v0);
    if (id < v0 || at >= (uint32_t)nv) return;
    if (answered) atomicAdd(counts + at, 1u);
    else atomicOr(counts + at, kPrompt);
    atomicOr(touched + (at >> 5), 1u << (at & 31));
  };
  auto adjusted = [&](float x, int at) {  // an id that is counted or biased
    const uint32_t c = counts[at];
    if (c != 0) {
      x = x > 0.f ? __fdiv_rn(x, rho) : x * rho;
      const uint32_t n = c & ~kPrompt;
      if (n != 0) x = x - freq * (float)n - pres;
    }
    return a.n_bias > 0 ? x + biases[at] : x;
  };

  for (int first = blockIdx.z * kRows; first < q1 - q0; first += gridDim.z * kRows) {
    const int last = min(first + kRows, q1 - q0);
    __syncthreads();  // the rows before no longer read the counts
    for (int i = tid; i < (int)(touched - smem) + words; i += kThreads) smem[i] = 0;
    __syncthreads();
    for (int i = tid; i < hist; i += kThreads) count(history[i], i >= prompt);
    if (a.tokens != nullptr)
      for (int i = tid; i < first; i += kThreads) count(a.tokens[q0 + i], hist + i >= prompt);
    if (tid >= kThreads - 32 && a.n_bias > 0) {
      // the biases by one warp, 32 at a time; an id that is there more than once gets their sum, in order
      const int lane = tid & 31;
      for (int i = 0; i < a.n_bias; i += 32) {
        const int id = i + lane < a.n_bias ? a.bias_ids[(int64_t)r * a.n_bias + i + lane] : -1;
        const float b = i + lane < a.n_bias ? a.bias[(int64_t)r * a.n_bias + i + lane] : 0.f;
        const bool mine = id >= v0 && id - v0 < nv;
        uint32_t same = __match_any_sync(~0u, mine ? id : -1 - lane);
        const bool leader = mine && (same & ((1u << lane) - 1)) == 0;
        float sum = mine ? biases[id - v0] : 0.f;
        while (__any_sync(~0u, leader && same != 0)) {
          const int from = leader && same != 0 ? __ffs(same) - 1 : lane;
          const float other = __shfl_sync(~0u, b, from);
          if (leader && same != 0) sum += other;
          same &= same - 1;
        }
        if (leader) {
          biases[id - v0] = sum;
          atomicOr(touched + ((id - v0) >> 5), 1u << ((id - v0) & 31));
        }
        __syncwarp();
      }
    }
    for (int i = first; i < last; ++i) {
      __syncthreads();
      if (tid == 0 && a.tokens != nullptr) count(a.tokens[q0 + i], hist + i >= prompt);
      __syncthreads();
      const int n = q0 + i;
      const T* x = static_cast<const T*>(a.logits) + (int64_t)n * a.row_stride + v0;
      T* y = static_cast<T*>(a.out) + (int64_t)n * a.out_stride + v0;
      const int m = a.mask == nullptr ? -1 : (a.mask_row == nullptr ? n : a.mask_row[n]);
      const uint32_t* mask = m >= 0 && m < a.mask_rows ? a.mask + (int64_t)m * a.mask_stride : nullptr;
      const int mask_words = (a.V + 31) / 32;
      auto single = [&](int at) {
        const bool allowed = mask == nullptr || ((mask[(v0 + at) >> 5] >> ((v0 + at) & 31)) & 1u);
        const bool there = (touched[at >> 5] >> (at & 31)) & 1u;
        if (!allowed) y[at] = rounded<T>(-INFINITY);
        else if (there) y[at] = rounded<T>(adjusted(value(x[at]), at));
        else if (x != y) y[at] = x[at];
      };
      // whole pieces between ids `head` and `head` + E `pieces`, where both rows agree on what is aligned
      const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15u), head = min(nv, off ? (16 - off) / (int)sizeof(T) : 0);
      const bool agree = off == (int)(reinterpret_cast<uintptr_t>(y) & 15u);
      const int pieces = agree ? (nv - head) / E : 0, tail = agree ? head + pieces * E : 0;
      if (agree && tid < head) single(tid);
      for (int k = tail + tid; k < nv; k += kThreads) single(k);
      for (int p = tid; p < pieces; p += kThreads) {
        const int at = head + p * E;
        constexpr uint32_t kAll = (1u << E) - 1;
        const uint32_t there = bits_at(touched, words, at) & kAll;
        const uint32_t allowed = mask == nullptr ? kAll : bits_at(mask, mask_words, v0 + at) & kAll;
        if (x == y && there == 0 && allowed == kAll) continue;
        union {
          uint4 raw;
          T e[E];
        } u;
        u.raw = load_once16(x + at);
        if (there != 0 || allowed != kAll) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if ((there >> e) & 1u) u.e[e] = rounded<T>(adjusted(value(u.e[e]), at + e));
            if (!((allowed >> e) & 1u)) u.e[e] = rounded<T>(-INFINITY);
          }
        }
        store16(y + at, u.raw);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const AdjustArgs& a, cudaStream_t s) {
  constexpr int kSlice = 8192;
  const int slice = std::min(kSlice, (a.V + 31) / 32 * 32), slices = (a.V + slice - 1) / slice;
  const int groups = std::max(1, std::min(4096, a.N / (a.R * kRows)));
  const size_t smem = ((size_t)slice * (a.n_bias > 0 ? 2 : 1) + (slice + 31) / 32) * 4;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(adjust_kernel<T>, (2 * (size_t)kSlice + kSlice / 32) * 4, done);
  if (e != cudaSuccess) return e;
  return launch_chained(adjust_kernel<T>, dim3(slices, a.R, groups), dim3(kThreads), smem, s, 1, a, slice);
}

}  // namespace

cudaError_t launch_adjust_logits(const AdjustArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case DSPARK_F32: return launch<float>(a, s);
    case DSPARK_BF16: return launch<__nv_bfloat16>(a, s);
    default: return launch<__half>(a, s);
  }
}

}  // namespace dspark
