// paged_attention.cu — attention of each request's last tokens over its paged key-value cache.
//
// A pass reads every seen key and value once and does little arithmetic on it (with G query
// heads per cache head and nq queries, nq G / 1 multiply-adds per element read), so what counts
// is that all SMs stream the cache all the time, whatever the lengths:
//   * The work is cut into units of TK tokens of one (request, cache head, 16 query rows) and
//     the units, in order, are dealt out evenly to the warps of the grid.  A warp works on its
//     own: its own ring of asynchronous copies, its own running maximum, sum and output; no
//     barrier between warps.  The cut follows from the lengths on the device (every CTA sums
//     them), so the launch does not depend on them and can be captured.
//   * Query rows (the G heads of a cache head, times the queries) are the 16 rows of the
//     tensor-core product; both products run as m16n8k16 on 16-bit operands with fp32 sums.
//     The weights go from the first product's result registers to the second's operands.
//   * A (request, head, rows) item that several warps share leaves partial outputs, which a
//     second kernel joins in a fixed order; an item of one warp is written at once.
// Element order inside a product is free as long as both operands agree, and is chosen so that
// a thread reads 16 contiguous bytes of a key row (d = 32 b + 8 t ..) and the query fragments
// are 16 contiguous bytes of a query row.
#include <algorithm>

#include "serving.cuh"

namespace dspark {
namespace {

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
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
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
};
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}

// ------------------------------------------------------------------------------- the plan

struct Request {
  int len, nq, q0, first;  // first: the first position that any of its queries sees
  int chunks, blocks;      // units of a (head, 16 query rows) item, and such items per head
};

constexpr int kRows = 16;

// chunks = 0: nothing to do (no queries, or invalid: reported).
template <int TK>
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
  if (a.window > 0) k.first = max(0, k.len - k.nq - a.window + 1);
  k.chunks = max(1, (k.len - k.first + TK - 1) / TK);
  k.blocks = (k.nq * a.G + kRows - 1) / kRows;
  return k;
}

// A share that a worker leaves to the joining kernel: the item's place and its units.
struct Share {
  int r, item, q0, nq;   // item: cache head * row blocks + row block; r < 0: none
  long long begin, end;  // the item's units
};

struct Scratch {
  Share* share;   // [workers] the item that starts in a worker's range and goes past it
  float2* stats;  // [workers][2][16] (maximum in base 2, sum)
  float* out;     // [workers][2][16][D]
  long long* per; // [1] units per worker
};

// The smallest share of a worker: below it the joining costs more than the spread gives.
constexpr int kMinUnits = 2;

// --------------------------------------------------------------------------- the main kernel

template <bool BF, bool Q8, int DP, int TK, int WARPS, int STAGES>
struct Cfg {
  static constexpr int kBytes = Q8 ? 1 : 2;
  static constexpr int row = DP * kBytes;          // bytes of a row in shared memory
  static constexpr int tile = TK * row;            // keys, or values, of a unit
  static constexpr int stage = 2 * tile;
  static constexpr int smem = WARPS * STAGES * stage;
  static constexpr int chunks = row / 16;          // 16-byte pieces of a row
};

// Where piece c of token row i lies: pieces are swapped within groups of eight so that the
// reads below (16 bytes per thread for keys, transposing loads for values) touch every bank
// once.
template <bool Q8>
__device__ __forceinline__ int key_piece(int i, int c) {
  return Q8 ? c ^ ((i & 3) << 1) : c ^ ((i & 1) << 2);
}
template <bool Q8>
__device__ __forceinline__ int value_piece(int i, int c) {
  return Q8 ? c ^ (((i >> 1) & 3) << 1) : c ^ (i & 7);
}
// Rows of 64 bytes hold four pieces only.
template <int CHUNKS>
__device__ __forceinline__ int held(int piece) {
  return CHUNKS >= 8 ? piece : piece & (CHUNKS - 1);
}

template <bool BFQ, bool Q8, int DP, int TK, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32) attention_kernel(const __grid_constant__ AttentionArgs a, Scratch scr) {
  using C = Cfg<BFQ, Q8, DP, TK, WARPS, STAGES>;
  using H = Half16<BFQ && !Q8>;  // type of the products
  constexpr int NT = TK / 8;     // key tiles of 8 tokens
  constexpr int DT = DP / 8;     // output tiles of 8 columns
  constexpr int DB = DP / 32;    // blocks of 32 elements of a row
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long scan[WARPS], start_off[WARPS];
  __shared__ int start_r[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int G = a.G;
  const long long worker = (long long)blockIdx.x * WARPS + warp, workers = (long long)gridDim.x * WARPS;

  griddep_wait();
  griddep_allow_next();

  // ---- which units: every CTA sums the requests' units (a slice per thread)
  const int slice = (a.R + WARPS * 32 - 1) / (WARPS * 32), r_lo = min((int)threadIdx.x * slice, a.R),
            r_hi = min(r_lo + slice, a.R);
  long long mine = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    const Request k = request<TK>(a, r, blockIdx.x == 0);
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
  long long total = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) upto += scan[w];
    total += scan[w];
  }
  const long long per = max((long long)kMinUnits, (total + workers - 1) / workers);
  for (int w = 0; w < WARPS; ++w) {
    const long long u = ((long long)blockIdx.x * WARPS + w) * per;
    if (u >= upto - mine && u < upto) {
      long long off = u - (upto - mine);
      int r = r_lo;
      for (;; ++r) {
        const Request k = request<TK>(a, r, false);
        const long long n = (long long)a.Hkv * k.blocks * k.chunks;
        if (off < n) break;
        off -= n;
      }
      start_r[w] = r;
      start_off[w] = off;
    }
  }
  __syncthreads();
  if (lane == 0) {
    scr.share[worker].r = -1;
    if (worker == 0) *scr.per = per;
  }
  const long long u_begin = worker * per, u_end = min(total, u_begin + per);
  if (u_begin >= u_end) return;
  __syncwarp();

  // ---- the copying side: one unit after the other into a ring of stages
  const unsigned char* k_pool = static_cast<const unsigned char*>(a.k_pool);
  const unsigned char* v_pool = static_cast<const unsigned char*>(a.v_pool);
  const uint32_t ring = smem_addr(smem) + warp * STAGES * C::stage;
  struct Cursor {
    Request k;
    int r, item, items, chunk;
  };
  auto open = [&](Cursor& c) {
    c.k = request<TK>(a, c.r, false);
    c.items = a.Hkv * c.k.blocks;
  };
  auto advance = [&](Cursor& c) {
    if (++c.chunk < c.k.chunks) return;
    c.chunk = 0;
    if (++c.item < c.items) return;
    c.item = 0;
    do {
      ++c.r;
      if (c.r >= a.R) return;
      open(c);
    } while (c.k.chunks == 0);
  };
  Cursor use;
  use.r = start_r[warp];
  open(use);
  use.item = (int)(start_off[warp] / use.k.chunks);
  use.chunk = (int)(start_off[warp] % use.k.chunks);
  Cursor get = use;

  // This lane's token of the unit at `get`: its page, one unit ahead of the copies.
  int page = 0, pos = 0;
  auto look_up = [&]() {
    pos = get.k.first + get.chunk * TK + (lane % TK);
    page = -1;
    if (get.r < a.R && pos < get.k.len) page = a.page_table[get.r * a.table_stride + pos / a.page_size];
  };
  look_up();
  long long left = u_end - u_begin;  // units still to be copied
  int put = 0;                       // next stage
  auto issue = [&]() {
    if (left > 0) {
      --left;
      int64_t from = -1;  // in 16-byte pieces; -1: nothing there, zeros instead
      if (pos < get.k.len) {
        if (page >= 0 && page < a.num_pages) {
          const int h = get.k.blocks == 1 ? get.item : get.item / get.k.blocks;
          from = ((int64_t)page * a.page_stride + (int64_t)h * a.head_stride + (int64_t)(pos % a.page_size) * a.token_stride) *
                 C::kBytes / 16;
        } else {
          report_bad_input(a.status, kBadPage);
        }
      }
      const uint32_t at = ring + put * C::stage;
      constexpr int kPer = C::chunks < 32 ? 32 / C::chunks : 1;  // rows copied at a time
      const int c = lane % C::chunks;
      const bool inside = c * 16 < a.D * C::kBytes;
#pragma unroll 4
      for (int i0 = 0; i0 < TK; i0 += kPer) {
        const int i = i0 + lane / C::chunks;
        const int64_t f = __shfl_sync(~0u, from, i);
        const bool take = f >= 0 && inside;
        const size_t off = take ? (size_t)(f + c) * 16 : 0;
        copy16(at + i * C::row + held<C::chunks>(key_piece<Q8>(i, c)) * 16, k_pool + off, take);
        copy16(at + C::tile + i * C::row + held<C::chunks>(value_piece<Q8>(i, c)) * 16, v_pool + off, take);
      }
      put = put + 1 == STAGES ? 0 : put + 1;
      if (left > 0) {
        advance(get);
        look_up();
      }
    }
    copy_commit();
  };
  for (int s = 0; s < STAGES - 1; ++s) issue();

  // ---- the computing side
  float o[DT][4], m[2], l[2];
  uint32_t qf[DB][2][4];  // query fragments: 32-element block, half of it
  int last[2], low[2];    // the positions that this thread's rows see: low..last
  float c_row[2];         // scores in base 2: scale log2(e) (k_scale) (2^e of a scaled fp16 query row)
  int stage = 0;
  bool fresh = true;  // the next unit opens an item
  long long item_begin = u_begin - use.chunk;
  for (long long u = u_begin; u < u_end; ++u) {
    const int h = use.k.blocks == 1 ? use.item : use.item / use.k.blocks;
    const int row0 = (use.item - h * use.k.blocks) * kRows;
    if (fresh) {
      fresh = false;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
      const float c = a.scale * kLog2e * (Q8 ? a.k_scale[h] : 1.f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = row0 + g + 8 * j, i = row / G;
        const bool there = row < use.k.nq * G;
        last[j] = there ? use.k.len - use.k.nq + i : -1;
        low[j] = a.window > 0 ? max(0, last[j] - a.window + 1) : 0;
        c_row[j] = c;
        const int64_t at = (int64_t)(use.k.q0 + i) * a.q_stride_token + (int64_t)(h * G + row - i * G) * a.q_stride_head;
        uint4 raw[DB];
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          raw[b] = make_uint4(0, 0, 0, 0);
          if (there && 32 * b + 8 * t4 < a.D)
            raw[b] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + 32 * b + 8 * t4);
        }
        if (Q8 && BFQ) {
          // bf16 queries over an e4m3 cache: fp16 operands, the row scaled by a power of two to
          // a maximum in [1, 2) so that it fits fp16's range; what falls below 2^-24 of the
          // row's maximum is lost, far under the sums' rounding
          float top = 0.f;
#pragma unroll
          for (int b = 0; b < DB; ++b) {
            const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = fmaxf(top, fmaxf(fabsf(Half16<true>::lo(w[e])), fabsf(Half16<true>::hi(w[e]))));
          }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          int e2 = 0;
          if (top > 0.f && top < INFINITY) e2 = min(max(ilogbf(top), -126), 126);
          const float down = ldexpf(1.f, -e2);
          c_row[j] = c * ldexpf(1.f, e2);
#pragma unroll
          for (int b = 0; b < DB; ++b) {
            uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = Half16<false>::pack(Half16<true>::lo(w[e]) * down, Half16<true>::hi(w[e]) * down);
            raw[b] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          qf[b][0][j] = raw[b].x;
          qf[b][0][j + 2] = raw[b].y;
          qf[b][1][j] = raw[b].z;
          qf[b][1][j + 2] = raw[b].w;
        }
      }
    }

    issue();
    copy_wait<STAGES - 1>();
    __syncwarp();
    const uint32_t keys = ring + stage * C::stage, values = keys + C::tile;

    // scores
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int b = 0; b < DB; ++b) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int i = 8 * j + g;
        uint32_t x, y, z, w;
        if (Q8) {
          const int piece = held<C::chunks>(key_piece<Q8>(i, 2 * b + (t4 >> 1)));
          const uint2 v = lds8(keys + i * C::row + piece * 16 + (t4 & 1) * 8);
          x = e4m3_to_half2(v.x);
          y = e4m3_to_half2(v.x >> 16);
          z = e4m3_to_half2(v.y);
          w = e4m3_to_half2(v.y >> 16);
        } else {
          const uint4 v = lds16(keys + i * C::row + held<C::chunks>(key_piece<Q8>(i, 4 * b + t4)) * 16);
          x = v.x, y = v.y, z = v.z, w = v.w;
        }
        H::mma(s[j], qf[b][0], x, y);
        H::mma(s[j], qf[b][1], z, w);
      }
    }

    // mask and softmax about the running maximum
    const int p0 = use.k.first + use.chunk * TK;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = p0 + 8 * j + 2 * t4 + (e & 1), row = e >> 1;
        const bool seen = p >= low[row] && p <= last[row];
        s[j][e] = seen ? s[j][e] * c_row[row] : -INFINITY;
        top[row] = fmaxf(top[row], s[j][e]);
      }
#pragma unroll
    for (int row = 0; row < 2; ++row) {
      top[row] = fmaxf(top[row], __shfl_xor_sync(~0u, top[row], 1));
      top[row] = fmaxf(top[row], __shfl_xor_sync(~0u, top[row], 2));
    }
    const bool grows = top[0] > m[0] || top[1] > m[1];
    if (__any_sync(~0u, grows)) {
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        const float now = fmaxf(m[row], top[row]);
        const float f = m[row] == -INFINITY ? 0.f : ex2(m[row] - now);
        m[row] = now;
        l[row] *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          o[i][2 * row] *= f;
          o[i][2 * row + 1] *= f;
        }
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][e] = ex2(s[j][e] - ref[e >> 1]);
        l[e >> 1] += s[j][e];
      }

    // Rows that see different positions share this unit's values: a value that is not finite
    // must not reach the rows that do not see it (0 x NaN).  Such a token is added on its own
    // to the rows that see it, and its row is cleared for the product.
    if (use.k.nq > 1 && (p0 + TK > use.k.len - use.k.nq + 1 || (a.window > 0 && p0 < use.k.len - a.window))) {
      uint32_t odd = 0;  // bit i: token i holds a value that is not finite
      for (int i = 0; i < TK; ++i) {
        bool found = false;
        for (int c = lane; c < C::row / 4; c += 32) {
          uint32_t w;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(values + i * C::row + c * 4));
          if (Q8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) found |= ((w >> (8 * e)) & 0x7F) == 0x7F;
          } else {
            found |= (w & H::kExp) == H::kExp || ((w >> 16) & H::kExp) == H::kExp;
          }
        }
        if (__any_sync(~0u, found)) odd |= 1u << i;
      }
      while (odd) {
        const int i = __ffs(odd) - 1;
        odd &= odd - 1;
        float w[2];
        // weight of (row g, token i): held by lane 4 g + (i % 8) / 2
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j == i / 8)
#pragma unroll
            for (int row = 0; row < 2; ++row) {
              const float even = __shfl_sync(~0u, s[j][2 * row], (lane & 28) + (i % 8) / 2);
              const float oddv = __shfl_sync(~0u, s[j][2 * row + 1], (lane & 28) + (i % 8) / 2);
              w[row] = i & 1 ? oddv : even;
            }
#pragma unroll
        for (int n = 0; n < DT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = Q8 ? (2 * t4 + (e & 1)) * (DP / 8) + n : 8 * n + 2 * t4 + (e & 1), row = e >> 1;
            const int byte = d * C::kBytes;
            const uint32_t at = values + i * C::row + held<C::chunks>(value_piece<Q8>(i, byte / 16)) * 16 + byte % 16;
            float v;
            if (Q8) {
              uint16_t x;
              asm volatile("{.reg .b32 t; ld.shared.u8 t, [%1]; cvt.u16.u32 %0, t;}" : "=h"(x) : "r"(at));
              v = Half16<false>::lo(e4m3_to_half2(x));
            } else {
              uint16_t x;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at));
              v = H::lo(x);
            }
            const int p = p0 + i;
            if (p >= low[row] && p <= last[row]) o[n][e] = fmaf(w[row], v, o[n][e]);
          }
        __syncwarp();
        for (int c = lane; c < C::chunks; c += 32) sts16(values + i * C::row + c * 16, make_uint4(0, 0, 0, 0));
        __syncwarp();
      }
    }

    // output += weights x values
#pragma unroll
    for (int k = 0; k < TK / 16; ++k) {
      const uint32_t p[4] = {H::pack(s[2 * k][0], s[2 * k][1]), H::pack(s[2 * k][2], s[2 * k][3]),
                             H::pack(s[2 * k + 1][0], s[2 * k + 1][1]), H::pack(s[2 * k + 1][2], s[2 * k + 1][3])};
      if (!Q8) {
        // matrices (tokens 0-7 | 8-15) x (columns 0-7 | 8-15) of 16 columns
        const int i = 16 * k + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int n = 0; n < DT; n += 2) {
          uint32_t v[4];
          ldmatrix_t(v, values + i * C::row + held<C::chunks>(value_piece<Q8>(i, n + (lane >> 4))) * 16);
          H::mma(o[n], p, v[0], v[1]);
          H::mma(o[n + 1], p, v[2], v[3]);
        }
      } else {
        // column n of output tile i is element n DP/8 + i: a thread reads DP/8 contiguous bytes
        // of four token rows and pairs them up
        constexpr int kRun = DP / 8;  // bytes
        constexpr int kStep = kRun < 16 ? kRun : 16;
#pragma unroll
        for (int d0 = 0; d0 < kRun; d0 += kStep) {
          uint32_t w[4][kStep / 4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = 16 * k + 8 * (q >> 1) + 2 * t4 + (q & 1);
            const int byte = g * kRun + d0;
            const uint32_t at = values + i * C::row + held<C::chunks>(value_piece<Q8>(i, byte / 16)) * 16 + byte % 16;
            if (kStep == 16) {
              const uint4 v = lds16(at);
              w[q][0] = v.x, w[q][1] = v.y, w[q][2 % (kStep / 4)] = v.z, w[q][3 % (kStep / 4)] = v.w;
            } else {
              const uint2 v = lds8(at);
              w[q][0] = v.x, w[q][1 % (kStep / 4)] = v.y;
            }
          }
#pragma unroll
          for (int e = 0; e < kStep / 4; ++e) {
            // bytes of the two tokens side by side: (r0[0] r1[0] r0[1] r1[1]), (r0[2] ...)
            const uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5140), a1 = __byte_perm(w[0][e], w[1][e], 0x7362);
            const uint32_t b0 = __byte_perm(w[2][e], w[3][e], 0x5140), b1 = __byte_perm(w[2][e], w[3][e], 0x7362);
            const int n = d0 + 4 * e;
            H::mma(o[n], p, e4m3_to_half2(a0), e4m3_to_half2(b0));
            H::mma(o[n + 1], p, e4m3_to_half2(a0 >> 16), e4m3_to_half2(b0 >> 16));
            H::mma(o[n + 2], p, e4m3_to_half2(a1), e4m3_to_half2(b1));
            H::mma(o[n + 3], p, e4m3_to_half2(a1 >> 16), e4m3_to_half2(b1 >> 16));
          }
        }
      }
    }
    __syncwarp();  // the stage may be filled again
    stage = stage + 1 == STAGES ? 0 : stage + 1;

    // ---- the item, or this worker's part of it, ends
    if (use.chunk + 1 == use.k.chunks || u + 1 == u_end) {
      const long long item_end = item_begin + use.k.chunks;
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        l[row] += __shfl_xor_sync(~0u, l[row], 1);
        l[row] += __shfl_xor_sync(~0u, l[row], 2);
      }
      if (item_begin >= u_begin && item_end <= u_end) {
        const float vs = Q8 ? a.v_scale[h] : 1.f;
#pragma unroll
        for (int row = 0; row < 2; ++row) {
          const int rr = row0 + g + 8 * row;
          if (rr >= use.k.nq * G) continue;
          const int i = rr / G;
          const size_t at = (size_t)(use.k.q0 + i) * a.Hq + h * G + rr - i * G;
          const float f = l[row] == 0.f ? 0.f : vs / l[row];
          uint16_t* out = static_cast<uint16_t*>(a.out) + at * a.D;
          if (!Q8) {
#pragma unroll
            for (int n = 0; n < DT; ++n)
              if (8 * n < a.D)
                *reinterpret_cast<uint32_t*>(out + 8 * n + 2 * t4) =
                    Half16<BFQ>::pack(o[n][2 * row] * f, o[n][2 * row + 1] * f);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int n = 0; n < DT; n += 2) {
                const int d = (2 * t4 + e) * (DP / 8) + n;
                if (d < a.D)
                  *reinterpret_cast<uint32_t*>(out + d) =
                      Half16<BFQ>::pack(o[n][2 * row + e] * f, o[n + 1][2 * row + e] * f);
              }
          }
          if (t4 == 0 && a.lse_out != nullptr) a.lse_out[at] = l[row] == 0.f ? -INFINITY : (m[row] + log2f(l[row])) * kLn2;
        }
      } else {
        // the worker's part 0 began before its range, part 1 begins in it
        const int part = item_begin >= u_begin;
        const size_t base = (size_t)(worker * 2 + part) * kRows;
#pragma unroll
        for (int row = 0; row < 2; ++row) {
          if (t4 == 0) scr.stats[base + g + 8 * row] = make_float2(m[row], l[row]);
          float* out = scr.out + (base + g + 8 * row) * DP;
#pragma unroll
          for (int n = 0; n < DT; ++n) {
            if (!Q8) {
              *reinterpret_cast<float2*>(out + 8 * n + 2 * t4) = make_float2(o[n][2 * row], o[n][2 * row + 1]);
            } else {
              out[(2 * t4) * (DP / 8) + n] = o[n][2 * row];
              out[(2 * t4 + 1) * (DP / 8) + n] = o[n][2 * row + 1];
            }
          }
        }
        if (part == 1 && lane == 0)
          scr.share[worker] = Share{use.r, use.item, use.k.q0, use.k.nq, item_begin, item_end};
      }
      fresh = true;
      item_begin = item_end;
    }
    advance(use);
  }
}

// Joins the parts of the item that starts in worker blockIdx.x's range and goes past it: four
// of its rows per CTA (blockIdx.y), the parts dealt to groups of threads.
constexpr int kJoinRows = 4, kJoinThreads = 256;
template <bool BFQ, int DP>
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
  const int G = a.G, rb = (k.nq * G + kRows - 1) / kRows, h = k.item / rb, row0 = (k.item - h * rb) * kRows;
  const int rows = min(kRows, k.nq * G - row0), first = blockIdx.y * kJoinRows;
  if (first >= rows) return;
  const int w0 = blockIdx.x, parts = (int)((k.end - 1) / *scr.per) - w0 + 1;  // part p: worker w0 + p
  // the statistics of a row by 64 threads: maximum and sum
  const int tid = threadIdx.x, lane = tid & 31, mine = tid >> 6;
  auto stat = [&](int p, int row) { return scr.stats[((size_t)(w0 + p) * 2 + (p == 0)) * kRows + row]; };
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
          *reinterpret_cast<const float4*>(scr.out + (((size_t)(w0 + p) * 2 + (p == 0)) * kRows + first + row) * DP + d);
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

// Warps per SM and ring stages: together about 190 KB of copies in flight per SM.
template <bool Q8, int DP>
struct Shape {
  static constexpr int TK = !Q8 && DP >= 128 ? 16 : 32;
  static constexpr int warps = 4;
  static constexpr int stages = 3;
  static constexpr int ctas = DP == 256 ? 1 : 2;  // per SM
};

constexpr int kMaxSms = 160;     // of the largest GB300 part; the scratch is sized without a device
constexpr int kMaxWorkers = kMaxSms * 2 * 4;

int padded(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }

template <bool BFQ, bool Q8, int DP>
cudaError_t launch(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  using S = Shape<Q8, DP>;
  using C = Cfg<BFQ, Q8, DP, S::TK, S::warps, S::stages>;
  auto* kernel = attention_kernel<BFQ, Q8, DP, S::TK, S::warps, S::stages>;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(kernel, C::smem, done);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count(), kMaxSms) * S::ctas, workers = grid * S::warps;
  unsigned char* at = static_cast<unsigned char*>(scratch);
  Scratch scr;
  scr.per = reinterpret_cast<long long*>(at);
  scr.share = reinterpret_cast<Share*>(at + 256);
  scr.stats = reinterpret_cast<float2*>(at + 256 + align256(sizeof(Share) * (size_t)kMaxWorkers));
  scr.out = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(scr.stats) +
                                     align256(sizeof(float2) * (size_t)kMaxWorkers * 2 * kRows));
  e = launch_chained(kernel, dim3(grid), dim3(S::warps * 32), C::smem, s, 1, a, scr);
  if (e != cudaSuccess) return e;
  const int rows = std::min(kRows, a.max_q * a.G);  // of an item, at most
  return launch_chained(join_kernel<BFQ, DP>, dim3(workers, (rows + kJoinRows - 1) / kJoinRows), dim3(kJoinThreads), 0, s, 1,
                        a, scr);
}

template <bool BFQ, bool Q8>
cudaError_t launch(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  switch (padded(a.D)) {
    case 64: return launch<BFQ, Q8, 64>(a, scratch, s);
    case 128: return launch<BFQ, Q8, 128>(a, scratch, s);
    default: return launch<BFQ, Q8, 256>(a, scratch, s);
  }
}

}  // namespace

size_t paged_attention_scratch(int, int, int, int, int D, int) {
  return 256 + align256(sizeof(Share) * (size_t)kMaxWorkers) + align256(sizeof(float2) * (size_t)kMaxWorkers * 2 * kRows) +
         sizeof(float) * (size_t)kMaxWorkers * 2 * kRows * padded(D);
}

cudaError_t launch_paged_attention(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  const bool q8 = a.dtype_kv == DSPARK_E4M3;
  if (a.dtype_q == DSPARK_BF16) return q8 ? launch<true, true>(a, scratch, s) : launch<true, false>(a, scratch, s);
  return q8 ? launch<false, true>(a, scratch, s) : launch<false, false>(a, scratch, s);
}

}  // namespace dspark
