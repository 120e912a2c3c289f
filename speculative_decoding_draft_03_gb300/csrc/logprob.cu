// logprob.cu — log probabilities of given tokens, with entropy and the best alternatives,
// and their gradient.
//
// Forward.  One pass over a row, by a thread-block cluster whose CTAs take contiguous slices
// and leave what they found in the first one's shared memory (no scratch, no second launch);
// the first one joins it, selects, and writes the outputs.  A thread keeps
// base-2 softmax statistics about a running reference, r ~ max of x c (c = log2(e) / T):
//   s = sum 2^u, w = sum 2^u u, u = x c - r;  entropy = (log2 s - w / s) ln 2,
// and with m the logit that the reference came from (r is m c rounded), S = log2 s - (m c - r):
//   lse = m / T + S ln 2,  ln p_v = (x_v - m) / T - S ln 2.
// The best K ids come from the same pass.  Each 1 KB segment of the row leaves its
// largest key in shared memory; the K best elements lie in the K segments with the largest
// maxima (an element of any other segment has K larger ones before it; among equal maxima the
// earlier segments), so only those few segments are read again, from the L2 cache.
// What bounds it: the copy rate of the device memory, and the selection at the end of each row,
// some 7000 cycles of one CTA while the others of its SM stream.  Measured: 1536 rows of 129280
// bf16, 30% of them skipped (278 MB): 48.0 us (87% of the copy rate), with the best 5 ids 56
// us, with 20 61 us; 256 rows of 151936 fp32, 30% skipped (109 MB), with the best 20: 30 us (2.4
// slices an SM, so that some SMs take three: 22 us without ids; and the selections of all rows
// come together at the end).
//
// Backward.  Elementwise, one read and one write of the row: 1024 rows of 151936 bf16, 10% of them
// skipped (591 MB), in 95 us (93% of the copy rate); 300 rows of 50257 fp32 (115 MB) in 20.6 us (83%).
#include <cooperative_groups.h>

#include <type_traits>

#include "serving.cuh"

namespace dspark {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A normaliser below this one is known well enough for the gradient: to 2^-19 for fp32, and to 2^-17
// where the gradient is rounded to 16 bits (2^-11 at best).
template <typename T>
constexpr float kLargeLse = sizeof(T) == 4 ? 64.f : 256.f;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 2;              // 16-byte pieces of a segment per lane: segments of 1 KB
constexpr int kSegPieces = 32 * kPer;
constexpr int kSteps = 4;            // segments in flight per warp
constexpr int kRing = kPer * kSteps * kThreads * 16;  // bytes
constexpr int kLongSlice = 128;       // segments
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i + 1 < N; i += 2) m = max3(m, x[i], x[i + 1]);
  return fmaxf(m, x[N - 1]);
}
// Order-preserving code of a number (-0 as +0); elements outside the row have code 0, below
// -inf's.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// ------------------------------------------------------------------- statistics of a row

// Softmax statistics about the reference r (in base 2), which is m c rounded for a logit m of the
// row.  r is held at kLowRef or above: a thread that saw only masked ids has sums of 0 about it.
constexpr float kLowRef = -1e30f, kHighRef = 1e30f;
struct __align__(16) Stats2 {
  float r, s, w, m;
};
__device__ __forceinline__ Stats2 join(Stats2 a, Stats2 b) {
  const float r = fmaxf(a.r, b.r), da = fmaxf(a.r - r, -200.f), db = fmaxf(b.r - r, -200.f), fa = ex2(da), fb = ex2(db);
  return {r, a.s * fa + b.s * fb, fmaf(da, a.s, a.w) * fa + fmaf(db, b.s, b.w) * fb, a.r >= b.r ? a.m : b.m};
}
// (the same in every lane)
__device__ __forceinline__ Stats2 warp_join(Stats2 a) {
  const float r = value_of(__reduce_max_sync(~0u, key_of(a.r))), d = fmaxf(a.r - r, -200.f), f = ex2(d);
  float s = a.s * f, w = fmaf(d, a.s, a.w) * f;
#pragma unroll
  for (int i = 16; i; i >>= 1) {
    s += __shfl_xor_sync(~0u, s, i);
    w += __shfl_xor_sync(~0u, w, i);
  }
  return {r, s, w, __shfl_sync(~0u, a.m, __ffs(__ballot_sync(~0u, a.r == r)) - 1)};
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

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
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
  int2 near[kCand];
  int n_segs, n_near, n_cand;
  Best warp_best[kWarps];
  alignas(16) uint32_t floor_buf[32];
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

// A key that at least K of the block's per-thread values reach: the K-th largest of each warp's
// few best (the block's K-th largest itself unless one warp holds more than that of them).  One
// barrier; `buf` is free again after the caller's next barrier.
constexpr int kWarpBest = 32 / kWarps;
__device__ __forceinline__ uint32_t kth_floor(uint32_t v, int K, uint32_t* buf) {
  static_assert(kWarpBest * kWarps == 32 && kMaxTopK <= 32, "one value per lane");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // half as many values again as K are enough to place it well
  const int take = min(kWarpBest, (K + K / 2 + kWarps - 1) / kWarps);
  uint32_t mine = 0;
  for (int i = 0; i < take; ++i) {
    const uint32_t m = __reduce_max_sync(~0u, v);
    if (lane == i) mine = m;
    const uint32_t at = __ballot_sync(~0u, v == m);
    if (lane == __ffs(at) - 1) v = 0;
  }
  if (lane < kWarpBest) buf[kWarpBest * warp + lane] = mine;
  __syncthreads();
  const uint32_t x = buf[lane];
  int above = 0;  // values larger than this one
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const uint4 w = *reinterpret_cast<const uint4*>(buf + j);
    above += (w.x > x) + (w.y > x) + (w.z > x) + (w.w > x);
  }
  return __reduce_min_sync(~0u, above < K ? x : ~0u);
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

// The K <= V best elements of the row, into sh.result (a row with a NaN may leave fewer: the rest
// have key 0).  seg_key: the n segments' largest keys; ring: kRing bytes.  Its loops stay rolled:
// this code runs once per row, and its instructions come from far (with the elements in unrolled
// registers 4096 rows of 32000 bf16 with 5 ids took 102 us, so they take 69).
template <typename T>
__device__ void row_best(const Row<T>& row, int n, const uint32_t* seg_key, int K, unsigned char* ring, TopShared& sh) {
  constexpr int VE = Piece<T>::n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int turn = 0;
  if (threadIdx.x < kMaxTopK) sh.result[threadIdx.x] = {0u, 0x7FFFFFFF};
  if (threadIdx.x == 0) sh.n_near = sh.n_cand = 0, sh.n_segs = n <= kSegs ? n : 0;

  // 1. the segments worth another look
  uint32_t floor_key = kLowestKey;
  if (n <= kSegs) {
    if (threadIdx.x < n) sh.segs[threadIdx.x] = threadIdx.x;
  } else {
    // the thread's best segment; neighbouring segments (where likely ids gather) go to different
    // warps
    uint32_t top = 0;
    for (int i = lane * kWarps + warp; i < n; i += kThreads) top = max(top, seg_key[i]);
    floor_key = max(kth_floor(top, K, sh.floor_buf), kLowestKey);
    auto gather = [&]() {
      for (int i = threadIdx.x; i < n; i += kThreads)
        if (seg_key[i] >= floor_key) {
          const int k = atomicAdd(&sh.n_segs, 1);
          if (k < kSegs) sh.segs[k] = i;
        }
      __syncthreads();
    };
    gather();
    int n_at = sh.n_segs;
    if (n_at > kSegs) {
      auto at_least = [&](uint32_t k) {
        int c = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) c += seg_key[i] >= k;
        return block_sum(c, sh.count, turn);
      };
      floor_key = bisect(floor_key, 0xFFFFFFFFu, K, kSegs, n_at, at_least);
      __syncthreads();
      if (threadIdx.x == 0) sh.n_segs = 0;
      __syncthreads();
      if (n_at <= kSegs) {
        gather();
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
    }
  }
  __syncthreads();

  // 2. their elements, into the ring; a thread reads what it copied
  static_assert(kSegs * kSegPieces * 16 <= kRing, "the ring holds them");
  const int segs = sh.n_segs;
  auto pieces = [&](auto f) {
#pragma unroll 1
    for (int k = warp; k < kPer * segs; k += kWarps)
      f(sh.segs[k / kPer] * kSegPieces + k % kPer * 32 + lane, (k * 32 + lane) * 16);
  };
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  pieces([&](int piece, int at) {
    if (row.whole(piece)) {
      copy16(ring_at + at, row.at + row.first(piece));
    } else {  // -inf outside the row
      float x[VE];
      row.load(piece, x);
      sts16(ring_at + at, Piece<T>::pack(x));
    }
  });
  copy_commit();
  copy_wait<0>();
  // f(key, id) of every element of this thread
  auto each = [&](auto f) {
    pieces([&](int piece, int at) {
      float x[VE];
      Piece<T>::unpack(lds16(ring_at + at), x);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const int id = row.first(piece) + i;
        if (id >= 0 && id < row.V) f(key_of(x[i]), id);
      }
    });
  };

  // 3. those at or above the threshold (the segments': an element below it is not among the best)
  auto clear = [&]() {
    if (threadIdx.x == 0) sh.n_near = sh.n_cand = 0;
  };
  auto collect = [&]() {  // their number; kCand + 1: more than are held
    const float floor = value_of(floor_key);
    pieces([&](int piece, int at) {
      float x[VE];
      Piece<T>::unpack(lds16(ring_at + at), x);
      if (max_of(x) >= floor) {
        const int k = atomicAdd(&sh.n_near, 1);
        if (k < kCand) sh.near[k] = make_int2(at, row.first(piece));
      }
    });
    __syncthreads();
    const int near = sh.n_near;  // pieces that hold some: now a thread per element
    for (int t = threadIdx.x; t < min(near, kCand) * VE; t += kThreads) {
      const int2 p = sh.near[t / VE];
      const float x = Piece<T>::value(reinterpret_cast<const T*>(ring + p.x)[t % VE]);
      const int id = p.y + t % VE;
      if (x >= floor && id >= 0 && id < row.V) {
        const int k = atomicAdd(&sh.n_cand, 1);
        if (k < kCand) sh.cand[k] = {key_of(x), id};
      }
    }
    __syncthreads();
    return near <= kCand ? min(sh.n_cand, kCand + 1) : kCand + 1;
  };
  auto closer = [&]() {
    float best = -INFINITY;
    pieces([&](int, int at) {
      float x[VE];
      Piece<T>::unpack(lds16(ring_at + at), x);
      best = fmaxf(best, max_of(x));
    });
    floor_key = max(floor_key, kth_floor(key_of(best), K, sh.floor_buf));
  };
  int n_el = kCand + 1;
#pragma unroll 1
  for (int i = n > kSegs ? 0 : 1; i < 2 && n_el > kCand; ++i) {
    if (i == 1) {  // no threshold so far, or the best lie together
      closer();
      clear();
      __syncthreads();
    }
    n_el = collect();
  }
  if (n_el > kCand) {  // too many: a higher threshold, if ties leave one
    auto at_least = [&](uint32_t k) {
      int c = 0;
      each([&](uint32_t key, int) { c += key >= k; });
      return block_sum(c, sh.count, turn);
    };
    floor_key = bisect(floor_key, 0xFFFFFFFFu, K, kCand, n_el, at_least);
    __syncthreads();
    clear();
    __syncthreads();
    if (n_el <= kCand)
      each([&](uint32_t key, int id) {
        if (key >= floor_key) sh.cand[atomicAdd(&sh.n_cand, 1)] = {key, id};
      });
    __syncthreads();
  }
  if (n_el <= kCand) {
    // 4. each candidate's place is the number of those before it
    for (int k = threadIdx.x; k < n_el; k += kThreads) {
      const Best mine = sh.cand[k];
      int place = 0;
#pragma unroll 4
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
    each([&](uint32_t key, int id) {
      const Best e = {key, id};
      if (before(last, e) && before(e, b)) b = e;
    });
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

// Packed pairs, each half rounded like its scalar operation.
__device__ __forceinline__ void fma_pair(float& a, float& b, float x0, float x1, float y0, float y1, float z0, float z1) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(a), "=f"(b)
      : "f"(x0), "f"(x1), "f"(y0), "f"(y1), "f"(z0), "f"(z1));
}

// A thread's statistics take in one piece, whose logits are `most` at most.  The reference moves
// only when that passes it by kSlack: any reference is right, but log2 s and w / s, whose
// difference is the entropy, are as large as the lag: with 16 the entropy was off by 7e-6 where this
// leaves 1e-6.  (1536 rows of 129280 bf16: 63.3 us so, 62.4 with 16, 64.9 with 0.)
constexpr float kSlack = 4.f;
struct Running {
  float r, s0, s1, w0, w1, m;  // sums over even and odd elements
};
template <int N>
__device__ __forceinline__ void take(Running& st, const float (&x)[N], float most, float c) {
  const float top = most * c;
  if (top > st.r + kSlack) {
    const float d = st.r - top, f = ex2(d), dc = fmaxf(d, -200.f);
    st.w0 = fmaf(dc, st.s0, st.w0) * f;
    st.w1 = fmaf(dc, st.s1, st.w1) * f;
    st.s0 *= f;
    st.s1 *= f;
    st.r = top;
    st.m = most;
  }
  float u[N], p[N];
#pragma unroll
  for (int i = 0; i < N; i += 2) fma_pair(u[i], u[i + 1], x[i], x[i + 1], c, c, -st.r, -st.r);
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = ex2(u[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = fmaxf(u[i], -200.f);  // masked ids: 0 x -inf does not arise
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    add2f(st.s0, st.s1, p[i], p[i + 1]);
    fma_pair(st.w0, st.w1, p[i], p[i + 1], u[i], u[i + 1], st.w0, st.w1);
  }
}

// One cluster per row.  A thread copies the pieces that it will read into a ring of its own,
// kSteps ahead (the ring holds what registers cannot: 32 KB per CTA in flight, no barriers).
// Dynamic shared memory: the ring, and a key per segment of the row (top_k > 0).  64 registers,
// four CTAs per SM (80 and three: 4096 rows of 32000 bf16 83 us instead of 73).
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(LogprobArgs a, int slice) {
  constexpr int VE = Piece<T>::n;
  extern __shared__ __align__(16) unsigned char dynamic[];
  uint32_t* seg_key = reinterpret_cast<uint32_t*>(dynamic + kRing);
  __shared__ Stats2 part[8 * kWarps];
  __shared__ Softmax slow_part[kWarps];
  __shared__ TopShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int n = blockIdx.x / ctas, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // running: may be written to
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
  const int segs = (row.pieces + kSegPieces - 1) / kSegPieces, seg0 = min(rank * slice, segs), seg1 = min(seg0 + slice, segs);

  // segments [full0, full1) lie wholly in the row; the others (its ends) are read directly
  const int full0 = row.shift ? 1 : 0, full1 = (a.V + row.shift) / (VE * kSegPieces);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(dynamic) + threadIdx.x * 16;
  const char* from = reinterpret_cast<const char*>(row.at - row.shift) + lane * 16;
  int ahead = seg0 + warp;  // the next segment to copy
  uint32_t put = 0, get = 0;
  auto issue = [&]() {
    if (ahead < seg1 && ahead >= full0 && ahead < full1) {
      const char* src = from + (size_t)ahead * (kSegPieces * 16);
#pragma unroll
      for (int u = 0; u < kPer; ++u) copy16(ring + put + u * (kThreads * 16), src + u * 512);
    }
    ahead += kWarps;
    put = put + kPer * kThreads * 16 == kRing ? 0 : put + kPer * kThreads * 16;
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kSteps - 1; ++i) issue();
  if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  uint32_t* const to_key = cluster.map_shared_rank(seg_key, 0);
  Running run = {kLowRef, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int g = seg0 + warp; g < seg1; g += kWarps) {
    issue();
    copy_wait<kSteps - 1>();
    float most = -INFINITY;
    if (g >= full0 && g < full1) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        float x[VE];
        Piece<T>::unpack(lds16(ring + get + u * (kThreads * 16)), x);
        const float m = max_of(x);
        take(run, x, m, c);
        most = fmaxf(most, m);
      }
    } else {
      for (int u = 0; u < kPer; ++u) {
        const int piece = g * kSegPieces + u * 32 + lane;
        if (piece >= row.pieces) break;
        float x[VE];
        row.load(piece, x);
        const float m = max_of(x);
        take(run, x, m, c);
        most = fmaxf(most, m);
      }
      __syncwarp();
    }
    get = get + kPer * kThreads * 16 == kRing ? 0 : get + kPer * kThreads * 16;
    if (TOP) {
      const uint32_t k = __reduce_max_sync(~0u, key_of(most));
      if (lane == 0) to_key[g] = k;
    }
  }
  Stats2 st = {run.r, run.s0 + run.s1, run.w0 + run.w1, run.m};
  st = warp_join(st);
  if (lane == 0) *cluster.map_shared_rank(part + rank * kWarps + warp, 0) = st;
  if (ctas > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  st = {kLowRef, 0.f, 0.f, 0.f};
  for (int w = lane; w < ctas * kWarps; w += 32) st = join(st, part[w]);
  st = warp_join(st);
  if (TOP) row_best(row, segs, seg_key, a.top_k, dynamic, sh);

  // ln p of a logit about m, or from the careful statistics
  float l2 = log2f(st.s);
  const float x_tok = Piece<T>::value(row.at[tok]);
  const bool plain = st.s > 0.f && st.r < kHighRef && st.r > kLowRef;  // (false where s is NaN)
  if (plain) {
    const float u_m = fmaf(st.m, c, -st.r);
    const bool one = st.s == ex2(u_m) && st.w == st.s * u_m;  // m has all the weight: nothing else was added
    const float ln_s = one ? 0.f : (l2 - u_m) * kLn2;
    auto logprob = [&](float x) { return fminf(fmaf(x - st.m, a.inv_temp, -ln_s), 0.f); };
    if (threadIdx.x == 0) {
      a.logprob_out[n] = logprob(x_tok);
      a.entropy_out[n] = one ? 0.f : fmaxf((l2 - st.w / st.s) * kLn2, 0.f);
      a.lse_out[n] = fmaf(st.m, a.inv_temp, ln_s);
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

// Written once: first to leave the cache (1024 rows of 151936 bf16: 97 us, with plain stores 100).
__device__ __forceinline__ void store_stream16(void* p, uint4 v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

constexpr int kBackPieces = 4;  // 16-byte pieces per thread

// grid: (pieces of a row / (256 x kBackPieces), rows).
template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_backward_kernel(LogprobArgs a) {
  constexpr int VE = Piece<T>::n;
  __shared__ float2 part[kWarps];
  griddep_wait();
  griddep_allow_next();
  const int n = blockIdx.y, tok = a.tokens[n];
  const Row<T> row(a.logits, n * a.row_stride, a.V);
  const Row<T> out(a.grad_out, n * a.grad_stride, a.V);
  T* to = const_cast<T*>(out.at);
  const float lse = a.lse[n], H = a.entropy[n];
  bool none = tok < 0 || tok >= a.V;
  const float gl = a.grad_logprob[n], ge = a.grad_entropy ? a.grad_entropy[n] : 0.f;
  // ln p = (x - at) / T - log_sum.  A large lse has too few digits left behind the point (masks of
  // the type's lowest value in the whole row: none): maximum and sum are taken again, by one CTA
  // that then writes the whole row (which may lie in the logits' place).  So they are for an
  // infinite one: the lowest value over T < 1 passes fp32's range, but only a row of -inf has nothing
  // left.  (1024 rows of 151936 bf16: 199 us if all are taken again, 16 rows 55 us: one CTA's
  // chain of loads.)
  float at = 0.f, log_sum = lse;
  const bool apart = !none && fabsf(lse) > kLargeLse<T>;
  if (apart) {
    if (blockIdx.x != 0) return;
    const float c = a.inv_temp * kLog2e;
    float m = -INFINITY, s = 0.f;
    auto rebase = [&](float to) {  // (m = -inf: s is 0)
      if (to > m) s *= ex2((m - to) * c), m = to;
    };
    for (int piece = threadIdx.x; piece < row.pieces; piece += kThreads) {
      float x[VE];
      row.load(piece, x);
      rebase(max_of(x));
      if (m > -INFINITY)
#pragma unroll
        for (int i = 0; i < VE; ++i) s += ex2((x[i] - m) * c);
    }
    float most = value_of(__reduce_max_sync(~0u, key_of(m)));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5].x = most;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) most = fmaxf(most, part[w].x);
    rebase(most);
#pragma unroll
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(~0u, s, i);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5].y = s;
    __syncthreads();
    s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += part[w].y;
    none = most == -INFINITY;
    at = most;
    log_sum = log2f(s) * kLn2;
  }
  const float A = fmaf(ge, H, gl);
  auto gradient = [&](float x, int v, auto again) {
    // ln p held above -300, where p is 0 whatever the mask's value: 0 x -inf does not arise
    const float lp = fmaxf(again ? (x - at) * a.inv_temp - log_sum : fmaf(x, a.inv_temp, -log_sum), -300.f);
    const float p = again ? exp2f(lp * kLog2e) : ex2(lp * kLog2e);  // (exp2f: small ones too, which low temperatures make)
    const float d = -p * fmaf(ge, lp, A) * a.inv_temp;
    return none ? 0.f : (v == tok ? fmaf(gl, a.inv_temp, d) : d);
  };
  auto write = [&](int block, auto again) {
    if (row.shift == out.shift) {
      const int piece0 = block * (kThreads * kBackPieces) + threadIdx.x;
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
        for (int i = 0; i < VE; ++i) x[i] = gradient(x[i], e + i, again);
        if (row.whole(piece)) {
          store_stream16(to + e, Piece<T>::pack(x));
        } else {
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (e + i >= 0 && e + i < a.V) to[e + i] = Piece<T>::rounded(x[i]);
        }
      }
    } else {
      const int e0 = block * (kThreads * kBackPieces * VE) - row.shift;
      for (int v = max(e0, 0) + threadIdx.x; v < min(e0 + kThreads * kBackPieces * VE, a.V); v += kThreads)
        to[v] = Piece<T>::rounded(gradient(none ? 0.f : Piece<T>::value(row.at[v]), v, again));
    }
  };
  if (apart)
    for (int block = 0; block < gridDim.x; ++block) write(block, std::true_type());
  else
    write(blockIdx.x, std::false_type());
}

constexpr size_t kMaxSmem = kRing + sizeof(uint32_t) * (kMaxLogprobV / 4 / kSegPieces + 2);

template <typename T>
cudaError_t forward(const LogprobArgs& a, cudaStream_t s) {
  const int pieces = (a.V + 2 * Piece<T>::n - 2) / Piece<T>::n, segs = (pieces + kSegPieces - 1) / kSegPieces;  // at most, any shift
  // CTAs per row: enough rows keep every SM busy by themselves; few are split over a cluster
  // while a slice keeps its threads in work, to two CTAs per SM where slices are long (64 rows of
  // 151936 bf16, 5 ids, by 4 CTAs each: 9.4 us, by 8 11.5; 256 rows of 151936 fp32, 20 ids, by 2:
  // 30 us, by 1 37)
  int ctas = 1;
  while (ctas < 8 && segs > ctas * 2 * kWarps &&
         (long long)a.N * ctas < (segs > ctas * kLongSlice ? 2ll : 1ll) * sm_count())
    ctas *= 2;
  const int slice = (segs + ctas - 1) / ctas;
  const size_t smem = kRing + (a.top_k > 0 ? sizeof(uint32_t) * segs : 0);
  auto* kernel = a.top_k > 0 ? logprob_kernel<T, true> : logprob_kernel<T, false>;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = allow_smem(kernel, kMaxSmem, done[a.top_k > 0]);
  if (e != cudaSuccess) return e;
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
