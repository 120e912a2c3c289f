// logprob.cu — log probabilities of given tokens, with entropy and the best alternatives,
// and their gradient.
//
// Forward.  One pass over a row, by a thread-block cluster whose CTAs take contiguous slices
// and join through distributed shared memory (no scratch, no second launch).  A thread keeps
// base-2 softmax statistics about a running reference, r ~ max of x c (c = log2(e) / T):
//   s = sum 2^u, w = sum 2^u u, u = x c - r;  lse = (r + log2 s) ln 2,
//   entropy = (log2 s - w / s) ln 2,  ln p_v = (x_v c - r - log2 s) ln 2.
// The best K ids come from the same pass.  Each 512-byte segment of the row leaves its
// largest key in shared memory; the K best elements lie in the K segments with the largest
// maxima (an element of any other segment has K larger ones before it; among equal maxima the
// earlier segments), so only those few segments are read again, from the L2 cache.
// What bounds it: the copy rate of the device memory.
//
// Backward.  Elementwise, one read and one write of the row.
#include <cooperative_groups.h>

#include "serving.cuh"

namespace dspark {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLargeLse = 1024.f;  // an lse beyond it is known to 2^-14 at best
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 4;           // 16-byte pieces in flight per thread
constexpr int kSegs = 32;            // segments that are read again, at most (>= kMaxTopK)
constexpr int kCand = 256;           // candidates that are ranked by counting, at most

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A 16-byte piece of a row as floats.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float value(float x) { return x; }
  static __device__ __forceinline__ float rounded(float x) { return x; }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 rounded(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Piece<__half> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float value(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half rounded(float x) { return __float2half_rn(x); }
};

// A row as 16-byte pieces on 16-byte boundaries: piece i holds the elements i n - shift ..,
// of which those below 0 or past V are not part of the row (and are not read).
template <typename T>
struct Row {
  const T* at;
  int V, shift, pieces;
  __device__ __forceinline__ Row(const void* base, int64_t offset, int V_) : at(static_cast<const T*>(base) + offset), V(V_) {
    shift = (int)((reinterpret_cast<uintptr_t>(at) & 15) / sizeof(T));
    pieces = (V + shift + Piece<T>::n - 1) / Piece<T>::n;
  }
  __device__ __forceinline__ int first(int piece) const { return piece * Piece<T>::n - shift; }
  __device__ __forceinline__ bool whole(int piece) const {
    const int e = first(piece);
    return e >= 0 && e + Piece<T>::n <= V;
  }
  // the elements outside the row as -inf
  __device__ __forceinline__ void load(int piece, float (&x)[Piece<T>::n]) const {
    const int e = first(piece);
    if (whole(piece)) {
      Piece<T>::unpack(load_once16(at + e), x);
      return;
    }
#pragma unroll
    for (int i = 0; i < Piece<T>::n; ++i) x[i] = e + i >= 0 && e + i < V ? Piece<T>::value(at[e + i]) : -INFINITY;
  }
};

// ------------------------------------------------------------------- statistics of a row

// Softmax statistics about the reference r (in base 2).  r is held at kLowRef or above: a
// thread that saw only masked ids has sums of 0 about it.
constexpr float kLowRef = -1e30f, kHighRef = 1e30f;
struct Stats2 {
  float r, s, w;
};
__device__ __forceinline__ Stats2 join(Stats2 a, Stats2 b) {
  const float r = fmaxf(a.r, b.r), da = fmaxf(a.r - r, -200.f), db = fmaxf(b.r - r, -200.f), fa = ex2(da), fb = ex2(db);
  return {r, a.s * fa + b.s * fb, fmaf(da, a.s, a.w) * fa + fmaf(db, b.s, b.w) * fb};
}
__device__ __forceinline__ Stats2 warp_join(Stats2 a) {
#pragma unroll
  for (int d = 16; d; d >>= 1)
    a = join(a, {__shfl_xor_sync(~0u, a.r, d), __shfl_xor_sync(~0u, a.s, d), __shfl_xor_sync(~0u, a.w, d)});
  return a;
}

// Statistics about the largest logit m, the difference taken before the product: right for any
// finite logits (masks of the type's lowest value neither overflow nor lose u), at twice the
// arithmetic.  For the rows whose statistics above do not hold.
struct Softmax {
  float m, s, w;
};
__device__ __forceinline__ Softmax merge(Softmax a, Softmax b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, 0.f, 0.f};
  const float da = fmaxf((a.m - m) * c, -200.f), db = fmaxf((b.m - m) * c, -200.f), fa = exp2f(da), fb = exp2f(db);
  return {m, a.s * fa + b.s * fb, (a.w + da * a.s) * fa + (b.w + db * b.s) * fb};
}

// By one CTA; the result in every thread.  `bad`: the row holds a NaN or +inf.
template <typename T>
__device__ __noinline__ Softmax row_softmax(const T* row, int V, float c, Softmax* part, bool& bad) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Softmax st = {-INFINITY, 0.f, 0.f};
  bad = false;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    const float x = Piece<T>::value(row[v]);
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
  for (int w = 1; w < kWarps; ++w) st = merge(st, part[w], c);
  return st;
}

// ------------------------------------------------------------------------ the best K

// Order-preserving code of a logit (-0 as +0); elements outside the row have code 0, below
// -inf's.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
constexpr uint32_t kLowestKey = 0x007FFFFFu;  // of -inf

struct Best {
  uint32_t key;
  int id;
};
__device__ __forceinline__ bool before(Best a, Best b) { return a.key > b.key || (a.key == b.key && a.id < b.id); }

struct TopShared {
  Best cand[kCand];
  Best result[kMaxTopK];
  int segs[kSegs];
  int count[2][kWarps];
  int n_segs, n_cand, ties;
  Best warp_best[kWarps];
};

// Block-wide sum of `mine`; `turn` alternates the two buffers, so one barrier is enough.
__device__ __forceinline__ int block_sum(int mine, int (*count)[kWarps], int& turn) {
  const int n = __reduce_add_sync(~0u, mine);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) count[turn][threadIdx.x >> 5] = n;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += count[turn][w];
  return sum;
}

// A key with between K and `most` of the counted keys at or above it, or (ties) the K-th
// largest key itself with more than `most`.  count(k) counts keys >= k over the block; lo has
// at least K, hi fewer.
template <typename Count>
__device__ __forceinline__ uint32_t bisect(uint32_t lo, uint32_t hi, int K, int most, int& n_lo, Count count) {
  while (n_lo > most && hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int n = count(mid);
    if (n >= K) lo = mid, n_lo = n;
    else hi = mid;
  }
  return lo;
}

// The K best elements of the CTA's slice (segments [seg0, seg0 + n)), into sh.result, fewer if
// the slice has fewer (the rest: key 0).  seg_key: the segments' largest keys.
template <typename T>
__device__ void slice_best(const Row<T>& row, int seg0, int n, const uint32_t* seg_key, int K, TopShared& sh) {
  constexpr int VE = Piece<T>::n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int turn = 0;
  if (threadIdx.x < kMaxTopK) sh.result[threadIdx.x] = {0u, 0x7FFFFFFF};
  if (threadIdx.x == 0) sh.n_segs = sh.n_cand = 0;
  uint32_t top = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) top = max(top, seg_key[i]);
  top = __reduce_max_sync(~0u, top);
  if (lane == 0) sh.warp_best[warp].key = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max(top, sh.warp_best[w].key);

  // 1. the segments worth another look
  uint32_t floor_key = kLowestKey;
  int n_at = n;
  if (n > kSegs) {
    floor_key = bisect(kLowestKey, top + 1, K, kSegs, n_at, [&](uint32_t k) {
      int c = 0;
      for (int i = threadIdx.x; i < n; i += kThreads) c += seg_key[i] >= k;
      return block_sum(c, sh.count, turn);
    });
  }
  if (n_at <= kSegs) {
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (seg_key[i] >= floor_key) sh.segs[atomicAdd(&sh.n_segs, 1)] = i;
  } else if (warp == 0) {
    // more segments share the K-th largest maximum: those above it, then the first of them
    int taken = 0;
    for (int pass = 0; pass < 2; ++pass)
      for (int i0 = 0; i0 < n && taken < K; i0 += 32) {
        const int i = i0 + lane;
        const bool take = i < n && (pass == 0 ? seg_key[i] > floor_key : seg_key[i] == floor_key);
        const uint32_t m = __ballot_sync(~0u, take);
        const int place = taken + __popc(m & ((1u << lane) - 1u));
        if (take && place < K) sh.segs[place] = i;
        taken = min(K, taken + __popc(m));
      }
    if (lane == 0) sh.n_segs = taken;
  }
  __syncthreads();

  // 2. their elements, in registers
  constexpr int kMine = kSegs / kWarps;
  const int segs = sh.n_segs;
  uint32_t key[kMine][VE];
  int id0[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int k = j * kWarps + warp;
    float x[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) key[j][i] = 0;
    id0[j] = 0;
    if (k < segs) {
      const int piece = (seg0 + sh.segs[k]) * 32 + lane;
      id0[j] = row.first(piece);
      if (piece < row.pieces) {
        row.load(piece, x);
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (id0[j] + i >= 0 && id0[j] + i < row.V) key[j][i] = key_of(x[i]);
      }
    }
  }

  // 3. a threshold that leaves few of them
  auto at_least = [&](uint32_t k) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < kMine; ++j)
#pragma unroll
      for (int i = 0; i < VE; ++i) c += key[j][i] >= k;
    return block_sum(c, sh.count, turn);
  };
  int n_el = at_least(floor_key);
  if (n_el > kCand) floor_key = bisect(floor_key, top + 1, K, kCand, n_el, at_least);
  if (n_el <= kCand) {
#pragma unroll
    for (int j = 0; j < kMine; ++j)
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (key[j][i] >= floor_key) sh.cand[atomicAdd(&sh.n_cand, 1)] = {key[j][i], id0[j] + i};
    __syncthreads();
    // 4. each candidate's place is the number of those before it
    if (threadIdx.x < n_el) {
      const Best mine = sh.cand[threadIdx.x];
      int place = 0;
      for (int i = 0; i < n_el; ++i) place += before(sh.cand[i], mine);
      if (place < K) sh.result[place] = mine;
    }
    __syncthreads();
    return;
  }
  // Many elements share the K-th largest logit: take the best one K times.
  Best last = {0xFFFFFFFFu, -1};
  for (int k = 0; k < K; ++k) {
    Best b = {0u, 0x7FFFFFFF};
#pragma unroll
    for (int j = 0; j < kMine; ++j)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const Best e = {key[j][i], id0[j] + i};
        if (e.key != 0 && before(last, e) && before(e, b)) b = e;
      }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const Best e = {__shfl_xor_sync(~0u, b.key, d), __shfl_xor_sync(~0u, b.id, d)};
      if (before(e, b)) b = e;
    }
    __syncthreads();
    if (lane == 0) sh.warp_best[warp] = b;
    __syncthreads();
    b = sh.warp_best[0];
    for (int w = 1; w < kWarps; ++w)
      if (before(sh.warp_best[w], b)) b = sh.warp_best[w];
    if (threadIdx.x == 0) sh.result[k] = b;
    last = b;
  }
  __syncthreads();
}

// --------------------------------------------------------------------------- forward

// One cluster per row.  Dynamic shared memory: a key per segment of the slice (top_k > 0).
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(LogprobArgs a, int slice) {
  constexpr int VE = Piece<T>::n;
  extern __shared__ uint32_t seg_key[];
  __shared__ Stats2 part[kWarps];
  __shared__ Softmax slow_part[kWarps];
  __shared__ Stats2 mine;
  __shared__ TopShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int n = blockIdx.x / ctas, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_allow_next();
  const int tok = a.tokens[n];
  const float nan = __int_as_float(0x7FC00000);
  if (tok < 0 || tok >= a.V) {  // the whole cluster
    if (rank == 0) {
      if (threadIdx.x == 0) a.logprob_out[n] = a.entropy_out[n] = a.lse_out[n] = nan;
      if (TOP && threadIdx.x < a.top_k) {
        a.top_ids_out[(size_t)n * a.top_k + threadIdx.x] = -1;
        a.top_logprobs_out[(size_t)n * a.top_k + threadIdx.x] = nan;
      }
    }
    return;
  }
  const Row<T> row(a.logits, n * a.row_stride, a.V);
  const float c = a.inv_temp * kLog2e;
  const int segs = (row.pieces + 31) / 32, seg0 = min(rank * slice, segs), seg1 = min(seg0 + slice, segs);

  Stats2 st = {kLowRef, 0.f, 0.f};
  for (int g0 = seg0 + warp; g0 < seg1; g0 += kWarps * kUnroll) {
    float x[kUnroll][VE];
    const int last = g0 + (kUnroll - 1) * kWarps;
    if (last < seg1 && row.first(g0 * 32) >= 0 && row.first(last * 32 + 32) <= row.V) {
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u] = load_once16(row.at + row.first((g0 + u * kWarps) * 32 + lane));
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) Piece<T>::unpack(v[u], x[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int piece = (g0 + u * kWarps) * 32 + lane;
        if (g0 + u * kWarps < seg1 && piece < row.pieces) {
          row.load(piece, x[u]);
        } else {
#pragma unroll
          for (int i = 0; i < VE; ++i) x[u][i] = -INFINITY;
        }
      }
    }
    float most = -INFINITY;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float m = x[u][0];
#pragma unroll
      for (int i = 1; i < VE; ++i) m = fmaxf(m, x[u][i]);
      most = fmaxf(most, m);
      if (TOP) {
        const uint32_t k = __reduce_max_sync(~0u, key_of(m));
        if (lane == 0 && g0 + u * kWarps < seg1) seg_key[g0 + u * kWarps - seg0] = k;
      }
    }
    const float r = fmaxf(st.r, most * c), d = st.r - r, f = ex2(d);
    st.w = fmaf(fmaxf(d, -200.f), st.s, st.w) * f;
    st.s *= f;
    st.r = r;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float e = fmaf(x[u][i], c, -r), p = ex2(e);
        st.s += p;
        st.w = fmaf(p, fmaxf(e, -200.f), st.w);
      }
  }
  st = warp_join(st);
  if (lane == 0) part[warp] = st;
  __syncthreads();
  st = part[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) st = join(st, part[w]);
  if (TOP) slice_best(row, seg0, seg1 - seg0, seg_key, a.top_k, sh);
  if (ctas > 1) {
    if (threadIdx.x == 0) mine = st;
    cluster.sync();
    if (rank != 0) {
      cluster.sync();  // its shared memory is read until then
      return;
    }
    for (int r = 1; r < ctas; ++r) st = join(st, *cluster.map_shared_rank(&mine, r));
    if (TOP) {
      const int total = ctas * a.top_k;  // <= 8 * 32 = kCand
      if (threadIdx.x < total)
        sh.cand[threadIdx.x] = cluster.map_shared_rank(&sh, threadIdx.x / a.top_k)->result[threadIdx.x % a.top_k];
      __syncthreads();
      if (threadIdx.x < total) {
        const Best me = sh.cand[threadIdx.x];
        int place = 0;
        for (int i = 0; i < total; ++i) place += before(sh.cand[i], me);
        if (me.key != 0 && place < a.top_k) sh.result[place] = me;
      }
      __syncthreads();
    }
    cluster.sync();
  }

  // ln p of a logit: (x c - r - log2 s) ln 2, or from the careful statistics
  float l2 = log2f(st.s);
  const float x_tok = Piece<T>::value(row.at[tok]);
  const bool plain = st.s > 0.f && st.r < kHighRef && st.r > kLowRef;  // (false where s is NaN)
  if (plain) {
    auto logprob = [&](float x) {
      const float y = (fmaf(x, c, -st.r) - l2) * kLn2;
      // (a masked id's lowest value passes the range in base 2, not in base e)
      return y > -INFINITY ? y : fmaf(x, a.inv_temp, -(st.r + l2) * kLn2);
    };
    if (threadIdx.x == 0) {
      a.logprob_out[n] = logprob(x_tok);
      a.entropy_out[n] = (l2 - st.w / st.s) * kLn2;
      a.lse_out[n] = (st.r + l2) * kLn2;
    }
    if (TOP && threadIdx.x < a.top_k) {
      const Best b = sh.result[threadIdx.x];
      a.top_ids_out[(size_t)n * a.top_k + threadIdx.x] = b.id;
      a.top_logprobs_out[(size_t)n * a.top_k + threadIdx.x] = logprob(value_of(b.key));
    }
    return;
  }
  bool bad;
  const Softmax sm = row_softmax(row.at, a.V, c, slow_part, bad);
  const bool none = sm.m == -INFINITY;
  l2 = log2f(sm.s);
  auto logprob = [&](float x) { return bad ? nan : (none ? -INFINITY : fmaf(x - sm.m, a.inv_temp, -l2 * kLn2)); };
  if (threadIdx.x == 0) {
    a.logprob_out[n] = logprob(x_tok);
    a.entropy_out[n] = bad ? nan : (none ? 0.f : (l2 - sm.w / sm.s) * kLn2);
    a.lse_out[n] = bad ? nan : (none ? -INFINITY : fmaf(sm.m, a.inv_temp, l2 * kLn2));
  }
  if (TOP && threadIdx.x < a.top_k) {
    const Best b = sh.result[threadIdx.x];
    a.top_ids_out[(size_t)n * a.top_k + threadIdx.x] = bad ? -1 : b.id;
    a.top_logprobs_out[(size_t)n * a.top_k + threadIdx.x] = logprob(value_of(b.key));
  }
}

// --------------------------------------------------------------------------- backward

constexpr int kBackPieces = 2;  // 16-byte pieces per thread

// grid: (pieces of a row / (256 x kBackPieces), rows).  `together`: a row's logits and its
// gradient lie alike on the 16-byte grid.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_backward_kernel(LogprobArgs a) {
  constexpr int VE = Piece<T>::n;
  __shared__ Softmax part[kWarps];
  griddep_wait();
  griddep_allow_next();
  const int n = blockIdx.y, tok = a.tokens[n];
  const Row<T> row(a.logits, n * a.row_stride, a.V);
  const Row<T> out(a.grad_out, n * a.grad_stride, a.V);
  T* to = const_cast<T*>(out.at);
  const float lse = a.lse[n], H = a.entropy[n];
  const bool none = tok < 0 || tok >= a.V || lse == -INFINITY;
  const float gl = a.grad_logprob[n], ge = a.grad_entropy ? a.grad_entropy[n] : 0.f;
  // ln p = (x - at) / T - log_sum.  A large lse (masks of the type's lowest value in the whole
  // row) has no digits left for the sum beside the maximum: the two are taken again, by one
  // CTA that then writes the whole row (which may lie in the logits' place).
  float at = 0.f, log_sum = lse;
  const bool apart = !none && fabsf(lse) > kLargeLse;
  if (apart) {
    if (blockIdx.x != 0) return;
    bool bad;
    const Softmax st = row_softmax(row.at, a.V, a.inv_temp * kLog2e, part, bad);
    at = st.m;
    log_sum = log2f(st.s) * kLn2;
  }
  const float A = fmaf(ge, H, gl);
  auto gradient = [&](float x, int v) {
    // ln p held above -300, where p is 0 whatever the mask's value: 0 x -inf does not arise
    const float lp = fmaxf(apart ? (x - at) * a.inv_temp - log_sum : fmaf(x, a.inv_temp, -log_sum), -300.f);
    const float d = -ex2(lp * kLog2e) * fmaf(ge, lp, A) * a.inv_temp;
    return none ? 0.f : (v == tok ? fmaf(gl, a.inv_temp, d) : d);
  };
  if (apart) {
    for (int v = threadIdx.x; v < a.V; v += kThreads)
      to[v] = Piece<T>::rounded(gradient(Piece<T>::value(row.at[v]), v));
    return;
  }
  const int piece0 = blockIdx.x * (kThreads * kBackPieces) + threadIdx.x;
  if (row.shift == out.shift) {
#pragma unroll
    for (int u = 0; u < kBackPieces; ++u) {
      const int piece = piece0 + u * kThreads;
      if (piece >= row.pieces) return;
      const int e = row.first(piece);
      float x[VE];
      if (none) {
#pragma unroll
        for (int i = 0; i < VE; ++i) x[i] = 0.f;
      } else {
        row.load(piece, x);
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) x[i] = gradient(x[i], e + i);
      if (row.whole(piece)) {
        store16(to + e, Piece<T>::pack(x));
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (e + i >= 0 && e + i < a.V) to[e + i] = Piece<T>::rounded(x[i]);
      }
    }
    return;
  }
  const int e0 = blockIdx.x * (kThreads * kBackPieces * VE) - row.shift;
  for (int v = max(e0, 0) + threadIdx.x; v < min(e0 + kThreads * kBackPieces * VE, a.V); v += kThreads)
    to[v] = Piece<T>::rounded(gradient(none ? 0.f : Piece<T>::value(row.at[v]), v));
}

template <typename T>
cudaError_t forward(const LogprobArgs& a, cudaStream_t s) {
  const int pieces = (a.V + 2 * Piece<T>::n - 2) / Piece<T>::n, segs = (pieces + 31) / 32;  // at most, any shift
  // CTAs per row: enough rows keep every SM busy by themselves; few are split over a cluster
  // while a slice keeps its threads in work
  int ctas = 1;
  while (ctas < 8 && (long long)a.N * ctas < 4ll * sm_count() && segs > ctas * 2 * kWarps) ctas *= 2;
  const int slice = (segs + ctas - 1) / ctas;
  const size_t smem = a.top_k > 0 ? sizeof(uint32_t) * slice : 0;
  auto* kernel = a.top_k > 0 ? logprob_kernel<T, true> : logprob_kernel<T, false>;
  return launch_chained(kernel, dim3((unsigned)a.N * ctas), dim3(kThreads), smem, s, ctas, a, slice);
}

template <typename T>
cudaError_t backward(const LogprobArgs& a, cudaStream_t s) {
  const int pieces = (a.V + 2 * Piece<T>::n - 2) / Piece<T>::n;
  const unsigned x = (pieces + kThreads * kBackPieces - 1) / (kThreads * kBackPieces);
  for (int n0 = 0; n0 < a.N; n0 += 65535) {  // a grid's limit of rows
    LogprobArgs b = a;
    b.N = min(a.N - n0, 65535);
    b.logits = static_cast<const T*>(a.logits) + n0 * a.row_stride;
    b.grad_out = static_cast<T*>(a.grad_out) + n0 * a.grad_stride;
    b.tokens += n0;
    b.lse += n0;
    b.entropy += n0;
    b.grad_logprob += n0;
    if (b.grad_entropy) b.grad_entropy += n0;
    const cudaError_t e = launch_chained(logprob_backward_kernel<T>, dim3(x, b.N), dim3(kThreads), 0, s, 1, b);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t s) {
  return a.dtype == DSPARK_F32 ? forward<float>(a, s)
                               : (a.dtype == DSPARK_BF16 ? forward<__nv_bfloat16>(a, s) : forward<__half>(a, s));
}

cudaError_t launch_token_logprobs_backward(const LogprobArgs& a, cudaStream_t s) {
  return a.dtype == DSPARK_F32 ? backward<float>(a, s)
                               : (a.dtype == DSPARK_BF16 ? backward<__nv_bfloat16>(a, s) : backward<__half>(a, s));
}

}  // namespace dspark
