// adjust.cu — logits adjusted before a token is taken from them: penalties for what a request has
// seen and answered, biases, and grammar masks.
//
// For row i of a slot's block, over the sequence history ++ tokens fed in up to row i (entries below
// prompt_len are the prompt's, the others answers):
//   x' = x / rho if x > 0 else x rho, for an id that is in the sequence;
//   x' -= frequency n + presence 1[n > 0], n: how often the id was answered;  x' += bias;
//   x' = -inf where the row's mask has a 0.
// Two kernels:
//   * The rows are copied, masks applied: 16 bytes a thread, four at a time.  (In place it has the masked ids
//     alone to write, and without a mask it is not launched.)
//   * Then the few ids that change.  A CTA takes a slice of the ids of one slot, for up to eight of the slot's
//     rows: it counts the whole history's ids of its slice in shared memory (a word per id: answers, and a bit
//     for the prompt); lists the ids that were counted; and adjusts them, an id a thread over all rows, with the
//     block's tokens counted as it comes to their rows.  Large slices read the history few times.
// (One kernel that did both slice by slice had each of its phases wait for memory on its own: 154 rows of 151936
// bf16 logits with histories of 1 K to 8 K tokens 41 us, 36 so; 182 rows of 50257 fp32 ones with histories of up
// to 32 K and 300 biases 86 us, 50 so.)
// What bounds it: device memory in the first (each logit is read and written once: 16.7 of the 36 us), in the
// second the chain from a slot's length over its history to its logits, whose lines are read for an id each: in
// place without masks, where the second is alone, these cases take 20.5 and 39 us.
#include <algorithm>

#include "serving.cuh"

namespace dspark {
namespace {

constexpr int kCopyThreads = 256, kCopyAhead = 4;
constexpr int kThreads = 1024;
constexpr int kRows = 8;  // rows that share one count, at most
constexpr int kMinSlice = 2048, kMaxSlice = 65536;  // (its ids are listed in 16 bits)
constexpr size_t kMaxSmem = 210 * 1024;
// A word per id: how often it was answered, whether the prompt has it, whether a row's own token is it, whether
// it has a bias.
constexpr uint32_t kPrompt = 1u << 31, kOwn = 1u << 30, kBiased = 1u << 29, kAnswers = kBiased - 1;

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }

// 32 bits of a bit array from bit `at` on; words past the last are 0.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int count, int at) {
  const int w = at >> 5;
  const uint32_t lo = words[w], hi = w + 1 < count ? words[w + 1] : 0u;
  return __funnelshift_r(lo, hi, at & 31);
}

__device__ __forceinline__ const uint32_t* mask_of(const AdjustArgs& a, int n) {
  const int m = a.mask == nullptr ? -1 : (a.mask_row == nullptr ? n : a.mask_row[n]);
  return m >= 0 && m < a.mask_rows ? a.mask + (int64_t)m * a.mask_stride : nullptr;
}

template <typename T>
__global__ void __launch_bounds__(kCopyThreads) mask_kernel(const __grid_constant__ AdjustArgs a, int chunks) {
  constexpr int E = 16 / (int)sizeof(T), kPieces = kCopyThreads * kCopyAhead;  // of a CTA
  constexpr uint32_t kAll = (1u << E) - 1;
  griddep_wait();
  griddep_allow_next();
  const int n = blockIdx.x / chunks, c = blockIdx.x - n * chunks, tid = threadIdx.x, words = (a.V + 31) / 32;
  if (n < a.q_start[0] || n >= a.q_start[a.R]) return;  // of no slot
  const T* x = static_cast<const T*>(a.logits) + (int64_t)n * a.row_stride;
  T* y = static_cast<T*>(a.out) + (int64_t)n * a.out_stride;
  const uint32_t* mask = mask_of(a, n);
  const bool in_place = a.out == a.logits;
  // whole pieces, where both rows agree on what is aligned
  const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15u), head = min(a.V, off ? (16 - off) / (int)sizeof(T) : 0);
  const int pieces = off == (int)(reinterpret_cast<uintptr_t>(y) & 15u) ? (a.V - head) / E : 0;
  union Piece {
    uint4 raw;
    T e[E];
  } u[kCopyAhead];
  uint32_t allowed[kCopyAhead];
#pragma unroll
  for (int j = 0; j < kCopyAhead; ++j) {
    const int p = c * kPieces + j * kCopyThreads + tid;
    allowed[j] = 0;
    if (p >= pieces) continue;
    if (!in_place) u[j].raw = load_once16(x + head + p * E);
    allowed[j] = mask == nullptr ? kAll : bits_at(mask, words, head + p * E) & kAll;
  }
#pragma unroll
  for (int j = 0; j < kCopyAhead; ++j) {
    const int p = c * kPieces + j * kCopyThreads + tid;
    if (p >= pieces || (in_place && allowed[j] == kAll)) continue;
    if (in_place) u[j].raw = load_once16(x + head + p * E);
    if (allowed[j] != kAll) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (!((allowed[j] >> e) & 1u)) u[j].e[e] = rounded<T>(-INFINITY);
    }
    store16(y + head + p * E, u[j].raw);
  }
  // what is left before and after them (the whole row where they do not agree)
  const int first = pieces > 0 ? head : 0, tail = first + pieces * E;
  for (int k = c * kCopyThreads + tid; k < first + a.V - tail; k += chunks * kCopyThreads) {
    const int v = k < first ? k : tail + k - first;
    if (mask != nullptr && !((mask[v >> 5] >> (v & 31)) & 1u)) y[v] = rounded<T>(-INFINITY);
    else if (!in_place) y[v] = x[v];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ AdjustArgs a, int slice, uint32_t per_slices) {
  extern __shared__ __align__(16) uint32_t counts[];  // [slice]
  uint32_t* marked = counts + slice;                             // [slice / 32] a bit per id that was counted
  uint16_t* list = reinterpret_cast<uint16_t*>(marked + slice / 32);  // the counted ids: no more than were counted
  __shared__ int bias_id[kThreads];
  __shared__ float bias_of[kThreads];
  __shared__ const uint32_t* masks[kRows];
  __shared__ int tokens[kRows], answered[kRows];  // the rows' tokens, as ids of the slice; whether they are answers
  __shared__ int listed, twice;
  const int tid = threadIdx.x, r = blockIdx.x, mine = blockIdx.y, slices = gridDim.y;
  // Slices take turns by 32 ids (a vocabulary's frequent ids are neighbours, and this spreads them): where an id
  // stands in this slice, or -1; and back.  per_slices: 2^32 / slices, rounded up.
  auto place_of = [&](int id) {
    if ((uint32_t)id >= (uint32_t)a.V) return -1;
    const uint32_t turn = (uint32_t)id >> 5, round = slices == 1 ? turn : __umulhi(turn, per_slices);  // (exact: turn < 2^15)
    return (int)(turn - round * slices) == mine ? (int)(round << 5 | (id & 31)) : -1;
  };
  auto id_at = [&](int at) { return ((at >> 5) * slices + mine) * 32 + (at & 31); };
  // (Also before the inputs are read, though what wrote them was complete before any row was copied: what earlier grids
  // wrote is there for a grid that has waited itself.  Counting beside the copy saved 2 us of 36, or 0.6 of 6.6.)
  griddep_wait();
  const int q0 = min(max(a.q_start[r], 0), a.N), q1 = min(max(a.q_start[r + 1], q0), a.N);
  const int hist = a.history == nullptr ? 0 : min(max(a.history_len[r], 0), a.history_width);
  const int prompt = a.prompt_len == nullptr ? 0 : a.prompt_len[r];
  const float rho = a.repetition == nullptr ? 1.f : a.repetition[r];
  const float freq = a.frequency == nullptr ? 0.f : a.frequency[r], pres = a.presence == nullptr ? 0.f : a.presence[r];
  const int32_t* history = a.history + r * a.history_stride;
  const int my_bias = tid < a.n_bias ? place_of(a.bias_ids[(int64_t)r * a.n_bias + tid]) : -1;
  const float my_value = tid < a.n_bias ? a.bias[(int64_t)r * a.n_bias + tid] : 0.f;
  const bool biased = my_bias >= 0;

  // (several threads may count the same id; the first marks it, unless it has a bias and is listed with that)
  auto mark = [&](int at) { atomicOr(marked + (at >> 5), 1u << (at & 31)); };
  auto count = [&](int id, bool answer) {
    const int at = place_of(id);
    if (at < 0) return;
    if ((answer ? atomicAdd(counts + at, 1u) : atomicOr(counts + at, kPrompt)) == 0) mark(at);
  };

  for (int first = blockIdx.z * kRows; first < q1 - q0; first += gridDim.z * kRows) {
    const int n_rows = min(kRows, q1 - q0 - first);
    __syncthreads();  // the rows before no longer read the counts
    for (int i = 4 * tid; i < slice; i += 4 * kThreads) *reinterpret_cast<uint4*>(counts + i) = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < slice / 32; i += kThreads) marked[i] = 0;
    if (tid < n_rows) {
      const int n = q0 + first + tid;
      masks[tid] = mask_of(a, n);
      tokens[tid] = a.tokens == nullptr ? -1 : place_of(a.tokens[n]);
      answered[tid] = hist + first + tid >= prompt;
    }
    bias_id[tid] = my_bias;
    bias_of[tid] = my_value;
    if (tid == 0) listed = 0, twice = 0;
    __syncthreads();
    if (a.n_bias > 0) {
      if (biased && atomicOr(counts + my_bias, kBiased) != 0) twice = 1;
      __syncthreads();
    }
    // the history, 16 bytes a thread at a time where it is aligned
    const int lead = min(hist, (int)((16 - (reinterpret_cast<uintptr_t>(history) & 15u)) & 15u) / 4), quads = (hist - lead) / 4;
    int4 next = make_int4(-1, -1, -1, -1);
    if (tid < quads) next = *reinterpret_cast<const int4*>(history + lead + 4 * tid);
#pragma unroll 1
    for (int i = tid; i < quads; i += kThreads) {
      const int at = lead + 4 * i;
      const int4 h = next;
      if (i + kThreads < quads) next = *reinterpret_cast<const int4*>(history + at + 4 * kThreads);
      count(h.x, at >= prompt), count(h.y, at + 1 >= prompt), count(h.z, at + 2 >= prompt), count(h.w, at + 3 >= prompt);
    }
    if (tid < lead) count(history[tid], tid >= prompt);
    for (int i = lead + 4 * quads + tid; i < hist; i += kThreads) count(history[i], i >= prompt);
    if (a.tokens != nullptr)
      for (int i = tid; i < first; i += kThreads) count(a.tokens[q0 + i], hist + i >= prompt);
    if (tid < n_rows && tokens[tid] >= 0 && atomicOr(counts + tokens[tid], kOwn) == 0) mark(tokens[tid]);
    // where an id has several biases: their sum, in order, with the first
    if (a.n_bias > 0) {
      bool leads = biased;
      float sum = my_value;
      if (biased && twice) {
        sum = 0.f;
        for (int j = 0; j < a.n_bias; ++j) {
          if (bias_id[j] != my_bias) continue;
          if (j < tid) leads = false;
          sum += bias_of[j];
        }
      }
      __syncthreads();
      if (!leads) bias_id[tid] = -1;
      bias_of[tid] = sum;
    }
    __syncthreads();
    // the marked ids, listed a word of 32 a thread (neighbours stay together: they share lines of the logits)
    const int lane = tid & 31;
    for (int w = tid; w - lane < slice / 32; w += kThreads) {
      uint32_t bits = w < slice / 32 ? marked[w] : 0u;
      int to = __popc(bits), from = 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, to, d);
        if (lane >= d) to += o;
      }
      if (lane == 31) from = atomicAdd(&listed, to);
      to += __shfl_sync(~0u, from, 31) - __popc(bits);
      for (; bits != 0; bits &= bits - 1) list[to++] = (uint16_t)(32 * w + __ffs(bits) - 1);
    }
    __syncthreads();
    // an id of a row a thread, in a loop as short as can be (unrolled over the rows it waited for instructions)
    const int per_row = listed + a.n_bias;
#pragma unroll 1
    for (int k = tid; k < per_row * n_rows; k += kThreads) {
      const int i = k / per_row, e = k - i * per_row;
      const int at = e < listed ? list[e] : bias_id[e - listed];
      if (at < 0) continue;
      const int id = id_at(at);
      T* y = static_cast<T*>(a.out) + (int64_t)(q0 + first + i) * a.out_stride + id;  // (as the copy has left it)
      float z = value(*y);
      const uint32_t* mask = masks[i];
      const uint32_t allowed = mask == nullptr ? ~0u : mask[id >> 5];
      const uint32_t c = counts[at];
      uint32_t n = c & kAnswers;
      bool seen = n != 0 || (c & kPrompt) != 0;
      if (c & kOwn)
        for (int j = 0; j <= i; ++j)
          if (tokens[j] == at) seen = true, n += answered[j];
      if (seen) z = z > 0.f ? __fdiv_rn(z, rho) : z * rho;
      if (n != 0) z = z - freq * (float)n - pres;
      if (e >= listed) z += bias_of[e - listed];
      if ((allowed >> (id & 31)) & 1u) *y = rounded<T>(z);
    }
  }
}

// The slices of a slot's ids: as few as shared memory allows (each reads the slot's history), or as many as still
// run at once on as many SMs.
int slice_of(const AdjustArgs& a, int n) { return ((a.V + 31) / 32 + n - 1) / n * 32; }
size_t smem_of(const AdjustArgs& a, int n) {
  const int slice = slice_of(a, n);
  const long long most = std::min<long long>(slice, (a.history == nullptr ? 0 : a.history_width) + (long long)a.N);
  return 4 * (size_t)slice + 4 * (size_t)((slice / 32 + 3) / 4 * 4) + (2 * (size_t)most + 15) / 16 * 16;
}
int slices_of(const AdjustArgs& a, int groups) {
  int n = 1;
  while (slice_of(a, n) > kMaxSlice || smem_of(a, n) > kMaxSmem) ++n;
  while ((long long)a.R * groups * (n + 1) <= sm_count() && slice_of(a, n + 1) >= kMinSlice) ++n;
  return n;
}

template <typename T>
cudaError_t launch(const AdjustArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(adjust_kernel<T>, kMaxSmem, done);
  if (e != cudaSuccess) return e;
  if (a.out != a.logits || a.mask != nullptr) {
    constexpr int kIds = kCopyThreads * kCopyAhead * (16 / (int)sizeof(T));
    const int chunks = (a.V + kIds - 1) / kIds;
    if ((long long)chunks * a.N > INT32_MAX) return cudaErrorInvalidValue;
    if ((e = launch_chained(mask_kernel<T>, dim3(chunks * a.N), dim3(kCopyThreads), 0, s, 1, a, chunks)) != cudaSuccess) return e;
  }
  const int groups = std::max(1, std::min(4096, a.N / (a.R * kRows))), n = slices_of(a, groups);
  const uint32_t per_slices = (uint32_t)(((1ull << 32) + n - 1) / n);
  return launch_chained(adjust_kernel<T>, dim3(a.R, n, groups), dim3(kThreads), smem_of(a, n), s, 1, a, slice_of(a, n), per_slices);
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
