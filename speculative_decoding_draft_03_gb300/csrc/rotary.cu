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
// What bounds it: device memory, each element being read and written once, where a token's rows give every thread of
// a CTA a piece.  8192 tokens of 40 heads of 128 in bf16: 28.6 us, 86 % of the copy rate; 16 prompts (9.5 K tokens)
// appended to an e4m3 cache: 39.7 us, 79 %; one token of each of 32 requests: 2.5 us, the launch.  With few heads most
// of a CTA's threads stand idle: 40000 tokens of 5 heads of 128 take 26.5 us (57 %), of 2 heads 21.3 (29 %), of 1 head of
// 64 14.1 (11 %).  Rows that are no whole pieces go an element at a time, by instructions: 8192 tokens of 40 heads of
// 80, 20 or 40 of them turned, 98 to 104 us (15 %).
#include <algorithm>

#include "serving.cuh"

namespace dspark {
namespace {

enum { kBadPage = 71, kBadQueries = 72 };
constexpr int kTokens = 4;  // of a CTA, at most

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

// x / scale, correctly rounded from the rounded reciprocal by one residual (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor").  `lift` brings a scale below 2^-100 or above
// 2^100, and x with it, nearer to 1, so that the reciprocal and the residual are normal numbers; what overflows
// stays infinite, and an infinite scale leaves 0 of what is finite (its residual is taken with 0 in its place).
// (16 prompts appended to an e4m3 cache: 49 us with __fdiv_rn for scales out of range beside it, 40 so.)
struct Divisor {
  float scale, inverse, lift;
};
__device__ __forceinline__ Divisor divisor(float s) {
  const float size = fabsf(s), lift = size < 0x1p-100f ? 0x1p64f : (size > 0x1p100f ? 0x1p-64f : 1.f);
  return {size < INFINITY ? s * lift : (size == INFINITY ? 0.f : s), __frcp_rn(s * lift), lift};
}
__device__ __forceinline__ float divided(float x, const Divisor& by) {
  // (the residual by its negative: so a -0 stays one)
  const float y = x * by.lift, q = y * by.inverse, r = fmaf(-fmaf(q, by.scale, -y), by.inverse, q);
  return fabsf(q) < INFINITY ? r : q;
}
// x / scale as e4m3, rounded to nearest even and held within +-448: two of them, and eight.
__device__ __forceinline__ uint16_t to_e4m3(float x0, float x1, const Divisor& by) {
  uint16_t p;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(divided(x1, by)), "f"(divided(x0, by)));
  return p;
}
__device__ __forceinline__ uint2 to_e4m3(float (&x)[8], const Divisor& by) {
  uint16_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = to_e4m3(x[2 * i], x[2 * i + 1], by);
  return make_uint2(p[0] | ((uint32_t)p[1] << 16), p[2] | ((uint32_t)p[3] << 16));
}

// The cosine and sine, times the magnitude, of a position's turn; `back` turns the other way.  The turn goes through
// one fp32 number, which near half a turn is off by 2^-25 half turns, as much as the result's own rounding to fp32
// (rms error of fp32 results 3.8e-8, 3.0e-8 with exact angles): the 64-bit product's further digits are dropped.
__device__ __forceinline__ float2 turn_of(int position, int64_t rate, float magnitude, bool back) {
  const uint64_t turns = (uint64_t)(int64_t)position * (uint64_t)rate;  // in 2^-64, modulo 1
  const int top = (int)(uint32_t)((turns + 0x80000000ull) >> 32);
  float s, c;
  sincospif((float)top * 0x1p-31f, &s, &c);  // half turns in [-1, 1]
  return make_float2(c * magnitude, (back ? -s : s) * magnitude);
}

// A pair turned, in place: the same roundings in every kernel here.
__device__ __forceinline__ void turn_pair(float& p, float& q, float2 t) {
  const float p0 = p;
  p = fmaf(p0, t.x, -(q * t.y));
  q = fmaf(p0, t.y, q * t.x);
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
      for (int j = 0; j < PAIRS; ++j) turn_pair(x[2 * j], x[2 * j + 1], f[j * pieces + u]);
    } else {
      Piece<T>::unpack(b, y);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) turn_pair(x[j], y[j], f[j * pieces + u]);
    }
  }
};

template <typename T, bool INTER, bool WIDE, int kThreads>
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
  // a place of a token's rows a thread, for all the CTA's tokens: their loads are on their way together
  for (int k = threadIdx.x; k < per_token; k += kThreads) {
    const int h = k / per_row, u = k - h * per_row;
    const T* from = x + (int64_t)t0 * a.x_token + (int64_t)h * a.x_head;
    T* to = out + (int64_t)t0 * a.out_token + (int64_t)h * a.out_head;
    if constexpr (WIDE) {
      if (u >= pieces) {
        const int d = a.rot + (u - pieces) * E;
        uint4 v[kTokens];
#pragma unroll
        for (int t = 0; t < kTokens; ++t)
          if (t < n) v[t] = load_once16(from + t * a.x_token + d);
#pragma unroll
        for (int t = 0; t < kTokens; ++t)
          if (t < n) store16(to + t * a.out_token + d, v[t]);
        continue;
      }
      Turned<T, INTER> p[kTokens];
#pragma unroll
      for (int t = 0; t < kTokens; ++t)
        if (t < n) p[t].load(from + t * a.x_token, u, pairs);
#pragma unroll
      for (int t = 0; t < kTokens; ++t) {
        if (t >= n) break;
        float lo[E], hi[E];
        p[t].turn(factors + t * pairs, u, pieces, lo, hi);
        store16(to + t * a.out_token + u * E, Piece<T>::pack(lo));
        if (!INTER) store16(to + t * a.out_token + pairs + u * E, Piece<T>::pack(hi));
      }
    } else {
      for (int t = 0; t < n; ++t, from += a.x_token, to += a.out_token) {
        if (u >= pieces) {
          const int d = a.rot + u - pieces;
          to[d] = from[d];
          continue;
        }
        const int i0 = INTER ? 2 * u : u, i1 = INTER ? 2 * u + 1 : u + pairs;
        float p = Piece<T>::one(from + i0), q = Piece<T>::one(from + i1);
        turn_pair(p, q, factors[t * pairs + u]);
        Piece<T>::one(to + i0, p);
        Piece<T>::one(to + i1, q);
      }
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

template <typename T, bool INTER, bool QUANT, int kThreads, int kTokens>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, int tokens) {
  extern __shared__ float2 factors[];  // [tokens][pairs]
  __shared__ Place places[kTokens];
  griddep_wait();
  griddep_allow_next();
  constexpr int E = kPiece<T>, PAIRS = INTER ? E / 2 : E;
  const int pairs = a.rot / 2, pieces = pairs / PAIRS, rest = (a.D - a.rot) / E, turning = pieces + rest, whole = a.D / E;
  const int t0 = blockIdx.x * tokens, n = min(tokens, a.T - t0);
  const int of_q = a.Hq * turning, of_k = of_q + a.Hkv * turning, per_token = of_k + a.Hkv * whole;
  // a place of a token's rows: of its queries, keys or values
  struct Unit {
    bool is_q, is_v, turns;
    int h, u, d;
  };
  auto unit = [&](int k) {
    Unit x;
    x.is_q = k < of_q, x.is_v = k >= of_k;
    k -= x.is_q ? 0 : (x.is_v ? of_k : of_q);
    const int per_row = x.is_v ? whole : turning;
    x.h = k / per_row, x.u = k - x.h * per_row;
    x.turns = !x.is_v && x.u < pieces;
    x.d = x.turns || x.is_v ? x.u * E : a.rot + (x.u - pieces) * E;
    return x;
  };
  // the CTA's tokens' loads are on their way together, the first while the tokens' places are looked up
  Turned<T, INTER> p[kTokens];
  auto load = [&](const Unit& x) {
    const int64_t step = x.is_q ? a.q_token : a.in_token;
    const T* from = static_cast<const T*>(x.is_q ? a.q : (x.is_v ? a.v : a.k)) + t0 * step +
                    (int64_t)x.h * (x.is_q ? a.q_head : a.in_head) + x.d;
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      if (t >= n) break;
      p[t].a = load_once16(from + t * step);
      if (!INTER && x.turns) p[t].b = load_once16(from + t * step + pairs);
    }
  };
  if (threadIdx.x < per_token) load(unit(threadIdx.x));
  if (threadIdx.x < n) places[threadIdx.x] = place_token(a, t0 + threadIdx.x);
  __syncthreads();
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    factors[t * pairs + place_of<PAIRS>(j, pieces)] = turn_of(places[t].position, a.rates[j], a.magnitude, false);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < per_token; k += kThreads) {
    const Unit x = unit(k);
    if (k >= kThreads) load(x);
    void* to = x.is_q ? a.q_out : (x.is_v ? a.v_pool : a.k_pool);
    const bool quant = QUANT && !x.is_q;
    const Divisor scale = divisor(quant ? (x.is_v ? a.v_scale : a.k_scale)[x.h] : 1.f);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      if (t >= n || places[t].position < 0) continue;
      const int64_t at =
          (x.is_q ? (t0 + t) * a.q_out_token + (int64_t)x.h * a.q_out_head : places[t].at + (int64_t)x.h * a.head_stride) + x.d;
      auto put = [&](int64_t where, float(&y)[E]) {
        if constexpr (QUANT) {
          if (quant) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(to) + where) = to_e4m3(y, scale);
            return;
          }
        }
        store16(static_cast<T*>(to) + where, Piece<T>::pack(y));
      };
      float lo[E], hi[E];
      if (x.turns) {
        p[t].turn(factors + t * pairs, x.u, pieces, lo, hi);
        put(at, lo);
        if (!INTER) put(at + pairs, hi);
      } else if (quant) {
        Piece<T>::unpack(p[t].a, lo);
        put(at, lo);
      } else {  // stored as it is
        store16(static_cast<T*>(to) + at, p[t].a);
      }
    }
  }
}

// The same where the turned part is not whole pieces: a pair of a token's elements a thread (of the part that turns
// its pairs, else neighbours), a token a CTA.  What bounds it: instructions, some 40 a pair.  (9.5 K tokens of 48 heads
// of 80, 40 of them turned: 95 us, all 80 by pieces 29; with four pairs' loads together 97.)
constexpr int kPairThreads = 256;
template <typename T, bool INTER, bool QUANT>
__global__ void __launch_bounds__(kPairThreads) append_pairs_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float2 factors[];  // [pairs]
  __shared__ Place place;
  griddep_wait();
  griddep_allow_next();
  const int pairs = a.rot / 2, half = a.D / 2, t = blockIdx.x;
  if (threadIdx.x == 0) place = place_token(a, t);
  __syncthreads();
  if (place.position < 0) return;
  for (int i = threadIdx.x; i < pairs; i += kPairThreads) factors[i] = turn_of(place.position, a.rates[i], a.magnitude, false);
  __syncthreads();
  const int of_q = a.Hq * half, of_k = of_q + a.Hkv * half, all = of_k + a.Hkv * half;
  for (int k = threadIdx.x; k < all; k += kPairThreads) {
    const bool is_q = k < of_q, is_v = k >= of_k;
    const int in = k - (is_q ? 0 : (is_v ? of_k : of_q)), h = in / half, u = in - h * half;
    const bool turns = !is_v && u < pairs;
    const int i0 = turns && !INTER ? u : 2 * u, i1 = turns && !INTER ? u + pairs : 2 * u + 1;
    const T* from = static_cast<const T*>(is_q ? a.q : (is_v ? a.v : a.k)) + t * (is_q ? a.q_token : a.in_token) +
                    h * (is_q ? a.q_head : a.in_head);
    const int64_t at = is_q ? t * a.q_out_token + h * a.q_out_head : place.at + h * a.head_stride;
    void* to = is_q ? a.q_out : (is_v ? a.v_pool : a.k_pool);
    const T x = from[i0], y = from[i1];
    float p = Piece<T>::one(&x), q = Piece<T>::one(&y);
    if (turns) turn_pair(p, q, factors[u]);
    if constexpr (QUANT) {
      if (!is_q) {
        const uint16_t two = to_e4m3(p, q, divisor((is_v ? a.v_scale : a.k_scale)[h]));
        uint8_t* row = static_cast<uint8_t*>(to) + at;
        row[i0] = (uint8_t)two, row[i1] = (uint8_t)(two >> 8);
        continue;
      }
    }
    T* row = static_cast<T*>(to) + at;
    if (turns) Piece<T>::one(row + i0, p), Piece<T>::one(row + i1, q);
    else row[i0] = x, row[i1] = y;  // as they are
  }
}

template <typename T, bool INTER>
cudaError_t launch(const RotaryArgs& a, cudaStream_t s) {
  constexpr int E = kPiece<T>;
  const int64_t stride = a.x_token | a.x_head | a.out_token | a.out_head;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0 && stride % E == 0 &&
                    a.D % E == 0 && a.rot % (INTER ? E : 2 * E) == 0;
  // (8192 tokens of 40 heads in bf16: 28.8 us with 128 threads, 29.5 with 256; 4096 of 32 in fp32, forward and
  // back: 51.5 and 51.2)
  constexpr int kThreads = sizeof(T) == 4 ? 256 : 128;
  // (40 heads of 128 in bf16, one token a CTA and two: 304 tokens 3.3 us and 3.5, 608 4.9 and 4.4, 1216 8.9 and 6.5)
  const int tokens = std::max(1, std::min(kTokens, a.T / (4 * sm_count())));
  const dim3 grid((unsigned)(((int64_t)a.T + tokens - 1) / tokens));
  const size_t smem = (size_t)tokens * (a.rot / 2) * sizeof(float2);
  if (tokens == 1)  // (few tokens: what counts is one's time)
    return wide ? launch_chained(rotary_kernel<T, INTER, true, 256>, grid, dim3(256), smem, s, 1, a, tokens)
                : launch_chained(rotary_kernel<T, INTER, false, 256>, grid, dim3(256), smem, s, 1, a, tokens);
  return wide ? launch_chained(rotary_kernel<T, INTER, true, kThreads>, grid, dim3(kThreads), smem, s, 1, a, tokens)
              : launch_chained(rotary_kernel<T, INTER, false, kThreads>, grid, dim3(kThreads), smem, s, 1, a, tokens);
}

template <typename T, bool INTER, bool QUANT>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  // (16 prompts of up to 1024 tokens, e4m3: 128 threads and two tokens 40 us, 256 and four 47;
  // the verified block of 32 requests: 512 threads 3.8 us, 256 4.2, 128 5.2.  The two forms, 48 heads of 128: 608
  // tokens 4.9 and 7.3 us, 900 7.6 and 7.9, 1216 9.1 and 9.4, 1500 11.5 and 11.1, 2000 14.2 and 12.5; into an e4m3
  // cache 7.1 and 7.4, 8.2 and 8.2, 10.7 and 9.2, 13.3 and 12.2, 16.7 and 12.9)
  const size_t one = (size_t)(a.rot / 2) * sizeof(float2);
  if (a.rot % (INTER ? kPiece<T> : 2 * kPiece<T>) != 0)
    return launch_chained(append_pairs_kernel<T, INTER, QUANT>, dim3((unsigned)a.T), dim3(kPairThreads), one, s, 1, a);
  if (a.T >= 8 * sm_count())
    return launch_chained(append_kernel<T, INTER, QUANT, 128, 2>, dim3((unsigned)(((int64_t)a.T + 1) / 2)), dim3(128), 2 * one, s, 1, a, 2);
  return launch_chained(append_kernel<T, INTER, QUANT, 512, 1>, dim3((unsigned)a.T), dim3(512), one, s, 1, a, 1);
}
template <typename T, bool INTER>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  return a.dtype_kv == DSPARK_E4M3 ? launch_append<T, INTER, true>(a, s) : launch_append<T, INTER, false>(a, s);
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
