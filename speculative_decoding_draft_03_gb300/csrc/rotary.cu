// rotary.cu — rotary positions: pairs of a head's elements turned by an angle that grows with the
// token's position; by itself, and on the way of keys and queries into a paged cache's step.
//
// The angle of pair i at position p is p f_i.  Held in radians in 32 bits it would be off by 2^-24 of
// itself, some 0.01 at position 200,000; here f_i is a 64-bit fraction of a turn ("rate"), so p f_i
// modulo one turn is one wrapping integer product, exact at every position, and its upper 32 bits go
// to sincospif.  Nothing is read from a table in memory.
//   * A CTA takes a few tokens.  Its threads first compute the tokens' cosines and sines, once for all
//     heads, into shared memory; then each takes 16-byte pieces: in the half layout the same piece of
//     both halves, in the interleaved one a piece of neighbouring pairs.
//   * The rotation is two products and a sum in fp32; one rounding to the stored type.
// What bounds it: device memory (each element is read and written once).
#include <algorithm>

#include "serving.cuh"

namespace dspark {
namespace {

enum { kBadPage = 71, kBadQueries = 72 };
constexpr int kThreads = 256;

template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);  // elements of a 16-byte piece

template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static __device__ __forceinline__ void unpack(uint4 r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void one(float* p, float x) { *p = x; }
};
template <>
struct Piece<__nv_bfloat16> {
  static __device__ __forceinline__ void unpack(uint4 r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
};
template <>
struct Piece<__half> {
  static __device__ __forceinline__ void unpack(uint4 r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __half2float(__ushort_as_half((unsigned short)w[i]));
      x[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float one(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ void one(__half* p, float x) { *p = __float2half_rn(x); }
};

// x / scale as e4m3, rounded to nearest even and held within +-448.
__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint16_t p[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = __fdiv_rn(x[4 * h + 2 * i], scale), b = __fdiv_rn(x[4 * h + 2 * i + 1], scale);
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p[i]) : "f"(b), "f"(a));
    }
    w[h] = p[0] | ((uint32_t)p[1] << 16);
  }
  return make_uint2(w[0], w[1]);
}

// The cosine and sine, times the magnitude, of a position's turn; `back` turns the other way.
__device__ __forceinline__ float2 turn_of(int position, int64_t rate, float magnitude, bool back) {
  const uint64_t turns = (uint64_t)(int64_t)position * (uint64_t)rate;  // in 2^-64, modulo 1
  const int top = (int)(uint32_t)((turns + 0x80000000ull) >> 32);
  float s, c;
  sincospif((float)top * 0x1p-31f, &s, &c);  // half turns in [-1, 1]
  return make_float2(c * magnitude, (back ? -s : s) * magnitude);
}

// Where pair i's factors stand among a token's in shared memory: neighbouring pieces' pairs with the
// same place in their piece side by side, so that the threads' reads touch every bank once.
template <int PAIRS>
__device__ __forceinline__ int place_of(int i, int pieces) {
  return PAIRS == 1 ? i : (i % PAIRS) * pieces + i / PAIRS;
}

// One row's rotating piece u of `pieces`: read, turned, and handed on.
template <typename T, bool INTER>
struct Turned {
  static constexpr int E = kPiece<T>, PAIRS = INTER ? E / 2 : E;
  uint4 a, b;
  __device__ __forceinline__ void load(const T* row, int u, int half) {
    a = load_once16(row + u * E);
    if (!INTER) b = load_once16(row + half + u * E);
  }
  // the piece (INTER), or the pieces of both halves, after the turn
  __device__ __forceinline__ void turn(const float2* f, int u, int pieces, float (&x)[E], float (&y)[E]) const {
    Piece<T>::unpack(a, x);
    if (INTER) {
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        const float2 t = f[j * pieces + u];
        const float p = x[2 * j], q = x[2 * j + 1];
        x[2 * j] = p * t.x - q * t.y;
        x[2 * j + 1] = q * t.x + p * t.y;
      }
    } else {
      Piece<T>::unpack(b, y);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        const float2 t = f[j * pieces + u];
        const float p = x[j], q = y[j];
        x[j] = p * t.x - q * t.y;
        y[j] = q * t.x + p * t.y;
      }
    }
  }
};

template <typename T, bool INTER, bool WIDE>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, int tokens) {
  extern __shared__ float2 factors[];  // [tokens][pairs]
  griddep_wait();
  griddep_allow_next();
  constexpr int E = WIDE ? kPiece<T> : 1, PAIRS = WIDE ? (INTER ? E / 2 : E) : 1;
  const int pairs = a.rot / 2, pieces = pairs / PAIRS;  // rotating pieces of a row
  const int t0 = blockIdx.x * tokens, n = min(tokens, a.T - t0);
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    factors[t * pairs + place_of<PAIRS>(p, pieces)] = turn_of(a.positions[t0 + t], a.rates[p], a.magnitude, a.inverse);
  }
  __syncthreads();
  const T* x = static_cast<const T*>(a.x);
  T* out = static_cast<T*>(a.out);
  const bool in_place = a.x == a.out;
  const int rest = in_place ? 0 : (a.D - a.rot) / E, per_row = pieces + rest, per_token = a.H * per_row;
  for (int i = threadIdx.x; i < n * per_token; i += kThreads) {
    const int t = i / per_token, k = i - t * per_token, h = k / per_row, u = k - h * per_row;
    const T* from = x + (int64_t)(t0 + t) * a.x_token + (int64_t)h * a.x_head;
    T* to = out + (int64_t)(t0 + t) * a.out_token + (int64_t)h * a.out_head;
    const float2* f = factors + t * pairs;
    if constexpr (WIDE) {
      if (u >= pieces) {
        const int d = a.rot + (u - pieces) * E;
        store16(to + d, load_once16(from + d));
        continue;
      }
      Turned<T, INTER> p;
      float lo[E], hi[E];
      p.load(from, u, pairs);
      p.turn(f, u, pieces, lo, hi);
      store16(to + u * E, Piece<T>::pack(lo));
      if (!INTER) store16(to + pairs + u * E, Piece<T>::pack(hi));
    } else {
      if (u >= pieces) {
        const int d = a.rot + u - pieces;
        to[d] = from[d];
        continue;
      }
      const int i0 = INTER ? 2 * u : u, i1 = INTER ? 2 * u + 1 : u + pairs;
      const float2 c = f[u];
      const float p = Piece<T>::one(from + i0), q = Piece<T>::one(from + i1);
      Piece<T>::one(to + i0, p * c.x - q * c.y);
      Piece<T>::one(to + i1, q * c.x + p * c.y);
    }
  }
}

// ------------------------------------------------------------------------------ append

// Where a token's keys and values go: its slot's place, or -1 where nothing is stored.
struct Place {
  int64_t at;    // element of head 0 in the pools
  int position;  // -1: the token is of no slot, or of one without room
};

__device__ __forceinline__ Place place_token(const AppendArgs& a, int t) {
  Place p{-1, -1};
  const int r = upper_bound(a.q_start, a.R + 1, t) - 1;
  if (r < 0 || r >= a.R || (a.granted != nullptr && a.granted[r] == 0)) return p;
  const int begin = a.q_start[r], n = a.q_start[r + 1] - begin, i = t - begin;
  const long long pos = (long long)a.seq_len[r] - n + i;
  if (i < 0 || i >= n || pos < 0 || pos >= (long long)a.max_pages * a.page_size) {
    report_bad_input(a.status, kBadQueries);
    return p;
  }
  const int nth = (int)pos / a.page_size, page = a.page_table[r * a.table_stride + nth];
  if (page < 0 || page >= a.num_pages) {
    report_bad_input(a.status, kBadPage);
    return p;
  }
  p.position = (int)pos;
  p.at = page * a.page_stride + ((int)pos - nth * a.page_size) * a.token_stride;
  return p;
}

constexpr int kMaxTokens = 16;  // of a CTA

template <typename T, bool INTER, bool QUANT>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, int tokens) {
  extern __shared__ float2 factors[];  // [tokens][pairs]
  __shared__ Place places[kMaxTokens];
  griddep_wait();
  griddep_allow_next();
  constexpr int E = kPiece<T>, PAIRS = INTER ? E / 2 : E;
  const int pairs = a.rot / 2, pieces = pairs / PAIRS, rest = (a.D - a.rot) / E, turning = pieces + rest, whole = a.D / E;
  const int t0 = blockIdx.x * tokens, n = min(tokens, a.T - t0);
  if (threadIdx.x < n) places[threadIdx.x] = place_token(a, t0 + threadIdx.x);
  __syncthreads();
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    factors[t * pairs + place_of<PAIRS>(p, pieces)] = turn_of(places[t].position, a.rates[p], a.magnitude, false);
  }
  __syncthreads();
  const int of_q = a.Hq * turning, of_k = of_q + a.Hkv * turning, per_token = of_k + a.Hkv * whole;
  for (int i = threadIdx.x; i < n * per_token; i += kThreads) {
    const int t = i / per_token;
    int k = i - t * per_token;
    if (places[t].position < 0) continue;
    const float2* f = factors + t * pairs;
    const bool is_q = k < of_q, is_v = k >= of_k;
    if (!is_q) k -= is_v ? of_k : of_q;
    const int per_row = is_v ? whole : turning, h = k / per_row, u = k - h * per_row;
    const T* from = static_cast<const T*>(is_q ? a.q : (is_v ? a.v : a.k)) +
                    (int64_t)(t0 + t) * (is_q ? a.q_token : a.in_token) + (int64_t)h * (is_q ? a.q_head : a.in_head);
    const float scale = QUANT && !is_q ? (is_v ? a.v_scale : a.k_scale)[h] : 1.f;
    const int64_t at = is_q ? (int64_t)(t0 + t) * a.q_out_token + (int64_t)h * a.q_out_head
                            : places[t].at + (int64_t)h * a.head_stride;
    void* to = is_q ? a.q_out : (is_v ? a.v_pool : a.k_pool);
    float lo[E], hi[E];
    auto put = [&](int d, const float(&x)[E]) {
      if (QUANT && !is_q) {
        if constexpr (QUANT) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(to) + at + d) = to_e4m3(x, scale);
      } else {
        store16(static_cast<T*>(to) + at + d, Piece<T>::pack(x));
      }
    };
    if (is_v || u >= pieces) {  // stored as it is
      const int d = is_v ? u * E : a.rot + (u - pieces) * E;
      const uint4 raw = load_once16(from + d);
      if (QUANT && !is_q) {
        Piece<T>::unpack(raw, lo);
        put(d, lo);
      } else {
        store16(static_cast<T*>(to) + at + d, raw);
      }
      continue;
    }
    Turned<T, INTER> p;
    p.load(from, u, pairs);
    p.turn(f, u, pieces, lo, hi);
    put(u * E, lo);
    if (!INTER) put(pairs + u * E, hi);
  }
}

template <typename T, bool INTER>
cudaError_t launch(const RotaryArgs& a, cudaStream_t s) {
  constexpr int E = kPiece<T>;
  const int64_t stride = a.x_token | a.x_head | a.out_token | a.out_head;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0 && stride % E == 0 &&
                    a.D % E == 0 && a.rot % (INTER ? E : 2 * E) == 0;
  const int tokens = std::max(1, std::min(4, a.T / (4 * sm_count())));
  const dim3 grid((unsigned)((a.T + tokens - 1) / tokens));
  const size_t smem = (size_t)tokens * (a.rot / 2) * sizeof(float2);
  return wide ? launch_chained(rotary_kernel<T, INTER, true>, grid, dim3(kThreads), smem, s, 1, a, tokens)
              : launch_chained(rotary_kernel<T, INTER, false>, grid, dim3(kThreads), smem, s, 1, a, tokens);
}

template <typename T, bool INTER>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  const int tokens = std::max(1, std::min(4, a.T / (4 * sm_count())));
  const dim3 grid((unsigned)((a.T + tokens - 1) / tokens));
  const size_t smem = (size_t)tokens * (a.rot / 2) * sizeof(float2);
  return a.dtype_kv == DSPARK_E4M3 ? launch_chained(append_kernel<T, INTER, true>, grid, dim3(kThreads), smem, s, 1, a, tokens)
                                   : launch_chained(append_kernel<T, INTER, false>, grid, dim3(kThreads), smem, s, 1, a, tokens);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case DSPARK_F32: return a.interleaved ? launch<float, true>(a, s) : launch<float, false>(a, s);
    case DSPARK_BF16: return a.interleaved ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
    default: return a.interleaved ? launch<__half, true>(a, s) : launch<__half, false>(a, s);
  }
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  if (a.dtype_in == DSPARK_BF16) return a.interleaved ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
  return a.interleaved ? launch<__half, true>(a, s) : launch<__half, false>(a, s);
}

}  // namespace dspark
