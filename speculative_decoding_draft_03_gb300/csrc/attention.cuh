// attention.cuh — what the kernels of attention over a paged cache share: the requests, how
// their work is dealt out, and the joining of parts.
#pragma once

#include "serving.cuh"

namespace dspark {
namespace attention {

enum { kBadPage = 51, kBadRequest = 52 };
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
// Transposes an 8 x 8 matrix of 16-bit elements spread over the warp (row g in lanes 4 g ..).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The 16-bit type of the products: bf16, or fp16 (which also holds every e4m3 value exactly).
template <bool BF>
struct Half16;
template <>
struct Half16<true> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ float lo(uint32_t x) { return __uint_as_float(x << 16); }
  static __device__ __forceinline__ float hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
  static constexpr uint32_t kExp = 0x7F80u;  // exponent bits: all set for NaN and infinities
  static constexpr float kLift = 0.f;
};
template <>
struct Half16<false> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ float lo(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)x)); }
  static __device__ __forceinline__ float hi(uint32_t x) {
    return __half2float(__ushort_as_half((unsigned short)(x >> 16)));
  }
  static constexpr uint32_t kExp = 0x7C00u;
  // Weights are rounded as multiples of 2^-kLift of the largest: fp16 loses digits below 2^-14 and
  // everything below 2^-25, which the normaliser would still count.  What a context of L tokens loses
  // is then at most L 2^-32 of its sum.  (A larger lift would pass fp16's range where scores are so
  // large that their difference with the reference rounds up.)
  static constexpr float kLift = 7.f;
};
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}

// ------------------------------------------------------------------------------- the plan

struct Request {
  int len, nq, q0, first;  // first: where its units begin, a multiple of TK at or before what it sees
  int chunks, blocks;      // units of a (head, ROWS query rows) item, and such items per head
};

// chunks = 0: nothing to do (no queries, or invalid: reported).
template <int TK, int ROWS>
__device__ __forceinline__ Request request(const AttentionArgs& a, int r, bool report) {
  Request k;
  k.q0 = a.q_start[r];
  const int q1 = a.q_start[r + 1];
  k.nq = q1 - k.q0;
  k.len = a.seq_len[r];
  k.first = 0;
  k.chunks = 0;
  k.blocks = 1;
  if (k.q0 < 0 || q1 > a.T || q1 < k.q0 || k.nq > a.max_q || k.len < 0 || k.len > a.max_pages * a.page_size) {
    if (report) report_bad_input(a.status, kBadRequest);
    return k;
  }
  if (k.nq == 0) return k;
  if (a.granted != nullptr && a.granted[r] == 0) k.len = 0;  // its queries see nothing
  if (a.window > 0) k.first = max(0, k.len - k.nq - a.window + 1) / TK * TK;
  k.chunks = max(1, (k.len - k.first + TK - 1) / TK);
  k.blocks = (k.nq * a.G - 1) / ROWS + 1;  // (a call's rows may reach 2^31 - 1: none may be added to them)
  return k;
}

// Does a query of request k see the position, or a later one?  (The first unit may begin before all
// that they see.)
__device__ __forceinline__ bool seen(const AttentionArgs& a, const Request& k, int pos) {
  return a.window == 0 || pos > k.len - k.nq - a.window;
}

// A share that a worker leaves to the joining kernel: the item's place and its units.
struct Share {
  int r, item, q0, nq;   // item: cache head * row blocks + row block; r < 0: none
  long long begin, end;  // the item's units
};

struct Scratch {
  Share* share;   // [workers] the item that starts in a worker's range and goes past it
  float2* stats;  // [workers][2][rows] (maximum in base 2, sum)
  float* out;     // [workers][2][rows][D]
  long long* per; // [1] units per worker
};

// The smallest share of a worker.  (With 1 four requests of up to 200 tokens take 7.9 us, with 2
// 9.6 us, with 4 12.0 us: the joining of more parts costs less than their spread gives.)
constexpr int kMinUnits = 1;

// Where a worker stands: unit `chunk` of an item of request r.
struct Cursor {
  Request k;
  int r, item, items, chunk;
};
template <int TK, int ROWS>
__device__ __forceinline__ void open(const AttentionArgs& a, Cursor& c) {
  c.k = request<TK, ROWS>(a, c.r, false);
  c.items = a.Hkv * c.k.blocks;
}
template <int TK, int ROWS>
__device__ __forceinline__ void advance(const AttentionArgs& a, Cursor& c) {
  if (++c.chunk < c.k.chunks) return;
  c.chunk = 0;
  if (++c.item < c.items) return;
  c.item = 0;
  do {
    ++c.r;
    if (c.r >= a.R) return;
    open<TK, ROWS>(a, c);
  } while (c.k.chunks == 0);
}
template <int TK, int ROWS>
__device__ __forceinline__ Cursor stand(const AttentionArgs& a, int r, long long off) {
  Cursor c;
  c.r = r;
  open<TK, ROWS>(a, c);
  c.item = (int)(off / c.k.chunks);
  c.chunk = (int)(off % c.k.chunks);
  return c;
}

// Deals the units out: every CTA sums the requests' units (a slice per thread), `per` units go to
// each of `workers` workers, of which this CTA holds MINE from `first` on; their starts (request
// and unit within it) are left in start_r and start_off.
struct Deal {
  long long per, total;
};
template <int TK, int ROWS, int MINE, int THREADS>
__device__ __forceinline__ Deal deal(const AttentionArgs& a, long long first, long long workers, long long* scan,
                                     int* start_r, long long* start_off) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slice = (a.R + THREADS - 1) / THREADS, r_lo = min((int)threadIdx.x * slice, a.R), r_hi = min(r_lo + slice, a.R);
  long long mine = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    const Request k = request<TK, ROWS>(a, r, blockIdx.x == 0);
    mine += (long long)a.Hkv * k.blocks * k.chunks;
  }
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  Deal deal;
  deal.total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) upto += scan[w];
    deal.total += scan[w];
  }
  deal.per = max((long long)kMinUnits, (deal.total + workers - 1) / workers);
  for (int w = 0; w < MINE; ++w) {
    const long long u = (first + w) * deal.per;
    if (u >= upto - mine && u < upto) {
      long long off = u - (upto - mine);
      int r = r_lo;
      for (;; ++r) {
        const Request k = request<TK, ROWS>(a, r, false);
        const long long n = (long long)a.Hkv * k.blocks * k.chunks;
        if (off < n) break;
        off -= n;
      }
      start_r[w] = r;
      start_off[w] = off;
    }
  }
  __syncthreads();
  return deal;
}

// Joins the parts of the item that starts in worker blockIdx.x's range and goes past it: four
// of its rows per CTA (blockIdx.y), the parts dealt to groups of threads.
constexpr int kJoinRows = 4, kJoinThreads = 256;
template <bool BFQ, int DP, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttentionArgs a, Scratch scr) {
  constexpr int kQuads = DP / 4;                                      // threads of a row
  constexpr int kGroups = kJoinThreads / (kJoinRows * kQuads) > 0 ? kJoinThreads / (kJoinRows * kQuads) : 1;
  constexpr int kSpan = kGroups * kJoinRows * kQuads / kJoinThreads;  // rows' quads per thread (DP = 256: 1)
  static_assert(kSpan == 1, "one quad of one row per thread");
  __shared__ float2 half[kJoinThreads / 32];
  __shared__ float4 sums[kJoinThreads];
  griddep_wait();
  const Share k = scr.share[blockIdx.x];
  if (k.r < 0) return;
  const int G = a.G, rb = (k.nq * G - 1) / ROWS + 1, h = k.item / rb, row0 = (k.item - h * rb) * ROWS;
  const int rows = min(ROWS, k.nq * G - row0), first = blockIdx.y * kJoinRows;
  if (first >= rows) return;
  const int w0 = blockIdx.x, parts = (int)((k.end - 1) / *scr.per) - w0 + 1;  // part p: worker w0 + p
  // the statistics of a row by 64 threads: maximum and sum
  const int tid = threadIdx.x, lane = tid & 31, mine = tid >> 6;
  auto stat = [&](int p, int row) { return scr.stats[((size_t)(w0 + p) * 2 + (p == 0)) * ROWS + row]; };
  float m = -INFINITY, l = 0.f;
  if (first + mine < rows) {
    for (int p = tid & 63; p < parts; p += 64) {
      const float2 st = stat(p, first + mine);
      const float now = fmaxf(m, st.x);
      if (now > -INFINITY) l = l * ex2(m - now) + st.y * ex2(st.x - now);
      else l += st.y;
      m = now;
    }
  }
  auto merge = [&](float m2, float l2) {
    const float now = fmaxf(m, m2), ref = now == -INFINITY ? 0.f : now;
    l = l * ex2(m - ref) + l2 * ex2(m2 - ref);
    m = now;
  };
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float m2 = __shfl_xor_sync(~0u, m, d), l2 = __shfl_xor_sync(~0u, l, d);
    merge(m2, l2);
  }
  if (lane == 0) half[tid >> 5] = make_float2(m, l);
  __syncthreads();

  const int group = tid / (kJoinRows * kQuads), row = tid / kQuads % kJoinRows, d = tid % kQuads * 4;
  const bool there = first + row < rows;
  m = half[2 * row].x, l = half[2 * row].y;
  merge(half[2 * row + 1].x, half[2 * row + 1].y);
  const float ref = m == -INFINITY ? 0.f : m;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (there) {
#pragma unroll 4
    for (int p = group; p < parts; p += kGroups) {
      const float f = ex2(stat(p, first + row).x - ref);
      const float4 v =
          *reinterpret_cast<const float4*>(scr.out + (((size_t)(w0 + p) * 2 + (p == 0)) * ROWS + first + row) * DP + d);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
  }
  if (kGroups > 1) {
    sums[tid] = o;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      const float4 v = sums[tid + g * kJoinRows * kQuads];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
  }
  if (!there) return;
  const float vs = a.v_scale != nullptr ? a.v_scale[h] : 1.f;
  const int rr = row0 + first + row, i = rr / G;
  const size_t at = (size_t)(k.q0 + i) * a.Hq + h * G + rr - i * G;
  const float f = l == 0.f ? 0.f : vs / l;
  if (d < a.D)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * a.D + d) =
        make_uint2(Half16<BFQ>::pack(o.x * f, o.y * f), Half16<BFQ>::pack(o.z * f, o.w * f));
  if (d == 0 && a.lse_out != nullptr) a.lse_out[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The scratch behind the workspace's status block, for `workers` workers with items of `rows`
// query rows of D elements.
inline size_t share_bytes(int workers) { return align256(sizeof(Share) * (size_t)workers); }
inline size_t stats_bytes(int workers, int rows) { return align256(sizeof(float2) * (size_t)workers * 2 * rows); }
inline size_t scratch_bytes(int workers, int rows, int D) {
  return 256 + share_bytes(workers) + stats_bytes(workers, rows) + sizeof(float) * (size_t)workers * 2 * rows * D;
}
inline Scratch scratch_at(void* p, int workers, int rows) {
  unsigned char* at = static_cast<unsigned char*>(p);
  Scratch s;
  s.per = reinterpret_cast<long long*>(at);
  s.share = reinterpret_cast<Share*>(at + 256);
  s.stats = reinterpret_cast<float2*>(at + 256 + share_bytes(workers));
  s.out = reinterpret_cast<float*>(at + 256 + share_bytes(workers) + stats_bytes(workers, rows));
  return s;
}
template <bool BFQ, int DP, int ROWS>
cudaError_t launch_join(const AttentionArgs& a, const Scratch& scr, int workers, cudaStream_t s) {
  const int rows = ROWS < a.max_q * a.G ? ROWS : a.max_q * a.G;  // of an item, at most
  return launch_chained(join_kernel<BFQ, DP, ROWS>, dim3(workers, (rows + kJoinRows - 1) / kJoinRows), dim3(kJoinThreads), 0,
                        s, 1, a, scr);
}

constexpr int kMaxSms = 160;  // of the largest GB300 part; the scratch is sized without a device

}  // namespace attention
}  // namespace dspark
