// paged_attention.cu — attention of each request's last tokens over its paged key-value cache.
//
// A pass reads every seen key and value once and does little arithmetic on it (with G query
// heads per cache head and nq queries, 2 nq G multiply-adds per element pair read), so what
// counts is that all SMs stream the cache all the time, whatever the lengths:
//   * The work is cut into units of TK tokens of one (request, cache head, block of query rows)
//     and the units, in order, are dealt out evenly to the warps of the grid.  A warp works on
//     its own: its own ring of asynchronous copies, its own running maximum, sum and output; no
//     barrier between warps.  The cut follows from the lengths on the device (every CTA sums
//     them), so the launch does not depend on them and can be captured.
//   * Both products run as m16n8k16 on 16-bit operands with fp32 sums, with the tokens (then the
//     value columns) as the 16 rows and eight query rows (the G heads of a cache head, times the
//     queries) as the 8 columns: one new token's few rows waste little, and NB groups of eight
//     share every key and value read from shared memory.
//   * A (request, head, rows) item that several warps share leaves partial outputs, which a
//     second kernel joins in a fixed order; an item of one warp is written at once.
// Element order inside a product is free as long as both operands agree, and is chosen so that
// a thread reads 16 contiguous bytes of a key row at a time and the query fragments are 16
// contiguous bytes of a query row.
// What bounds it: with a 16-bit cache the device memory (32 requests of 1 K to 8 K tokens, 8 heads
// of 128 elements, one new token: 692 MB in 113 us, 6.1 TB/s, 4 us of it joining); with an e4m3
// cache the warps' chains of conversions and products (two contexts of 115 K tokens: 517 MB in 99
// us, of which the main kernel takes 87).
#include <algorithm>

#include "attention.cuh"
#include "attention_wide.h"

namespace dspark {
namespace {

using namespace attention;

// --------------------------------------------------------------------------- the main kernel

// Shared memory of a warp: a ring of units, each the keys, then the values, as panels of 128
// bytes of every token's row ([panel][TK][128]), whose 16-byte pieces are swapped by the row's
// number: the reads below (16 bytes per thread, transposing loads) touch every bank once.
template <bool Q8, int DP, int NB, int TK, int WARPS, int STAGES>
struct Cfg {
  static constexpr int kBytes = Q8 ? 1 : 2;
  static constexpr int row = DP * kBytes;
  static_assert(row % 128 == 0, "whole panels");
  static constexpr int panels = row / 128;
  static constexpr int panel = TK * 128;
  static constexpr int tile = TK * row;  // keys, or values, of a unit
  static constexpr int stage = 2 * tile;
  static constexpr int chunks = row / 16;  // 16-byte pieces of a row
  static constexpr bool q_smem = NB * DP > 256;  // the queries' fragments do not fit into registers
  static constexpr int q_bytes = q_smem ? NB * 8 * DP * 2 : 0;
  static constexpr int per_warp = STAGES * stage + q_bytes;
  static constexpr int smem = WARPS * per_warp;
};
template <int PANEL>
__device__ __forceinline__ uint32_t piece_at(int i, int c) {
  return (uint32_t)((c >> 3) * PANEL + i * 128 + (((c & 7) ^ (i & 7)) << 4));
}
// Which element of a value row is row r (0..15) of output tile n: with 16-bit values tile n holds
// 16 n .., with 8-bit ones (a thread reads piece g of a panel) rows g and g + 8 are neighbours.
template <bool Q8>
__device__ __forceinline__ int element(int n, int r) {
  return Q8 ? n / 8 * 128 + 16 * (r & 7) + 2 * (n % 8) + (r >> 3) : 16 * n + r;
}

template <bool BFQ, bool Q8, int DP, int NB, int TK, int WARPS, int STAGES, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS) attention_kernel(const __grid_constant__ AttentionArgs a, Scratch scr) {
  using C = Cfg<Q8, DP, NB, TK, WARPS, STAGES>;
  using H = Half16<BFQ && !Q8>;  // type of the products
  constexpr int ROWS = 8 * NB;
  constexpr int MT = TK / 16;    // token tiles of 16
  constexpr int DT = DP / 16;    // output tiles of 16 elements
  constexpr int KS = DP / 16;    // steps of 16 elements of a row
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long scan[WARPS], start_off[WARPS];
  __shared__ int start_r[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int G = a.G;
  const long long worker = (long long)blockIdx.x * WARPS + warp, workers = (long long)gridDim.x * WARPS;

  griddep_wait();
  griddep_allow_next();

  const Deal d = deal<TK, ROWS, WARPS, WARPS * 32>(a, (long long)blockIdx.x * WARPS, workers, scan, start_r, start_off);
  if (lane == 0) {
    scr.share[worker].r = -1;
    if (worker == 0) *scr.per = d.per;
  }
  const long long u_begin = worker * d.per, u_end = min(d.total, u_begin + d.per);
  if (u_begin >= u_end) return;
  __syncwarp();

  // ---- the copying side: one unit after the other into a ring of stages
  const unsigned char* k_pool = static_cast<const unsigned char*>(a.k_pool);
  const unsigned char* v_pool = static_cast<const unsigned char*>(a.v_pool);
  const uint32_t ring = smem_addr(smem) + warp * C::per_warp, q_at = ring + STAGES * C::stage;
  Cursor use = stand<TK, ROWS>(a, start_r[warp], start_off[warp]), get = use;

  // This lane's token of the unit at `get`: its page, looked up one unit ahead of the copies.
  int page = 0, pos = 0, slot = 0;
  auto look_up = [&]() {
    pos = get.k.first + get.chunk * TK + lane % TK;
    page = -1;
    const int nth = pos / a.page_size;
    slot = pos - nth * a.page_size;
    if (pos < get.k.len) page = a.page_table[get.r * a.table_stride + nth];
  };
  look_up();
  long long left = u_end - u_begin;  // units still to be copied
  int put = 0;                       // next stage
  auto issue = [&]() {
    if (left > 0) {
      --left;
      const int h = get.k.blocks == 1 ? get.item : get.item / get.k.blocks;
      const uint32_t at = ring + put * C::stage;
      const bool there = pos < get.k.len && page >= 0 && page < a.num_pages;
      if (pos < get.k.len && !there && seen(a, get.k, pos)) report_bad_input(a.status, kBadPage);
      int64_t from = -1;  // in 16-byte pieces; -1: nothing there, zeros instead
      if (there)
        from = ((int64_t)page * a.page_stride + (int64_t)h * a.head_stride + (int64_t)slot * a.token_stride) * C::kBytes / 16;
      constexpr int kPer = C::chunks < 32 ? 32 / C::chunks : 1;  // rows copied at a time
      const int c = lane % C::chunks;
      const bool inside = c * 16 < a.D * C::kBytes;
#pragma unroll 4
      for (int i0 = 0; i0 < TK; i0 += kPer) {
        const int i = i0 + lane / C::chunks;
        const int64_t f = __shfl_sync(~0u, from, i);
        const bool take = f >= 0 && inside;
        const size_t off = take ? (size_t)(f + c) * 16 : 0;
        copy16(at + piece_at<C::panel>(i, c), k_pool + off, take);
        copy16(at + C::tile + piece_at<C::panel>(i, c), v_pool + off, take);
      }
      put = put + 1 == STAGES ? 0 : put + 1;
      if (left > 0) {
        advance<TK, ROWS>(a, get);
        look_up();
      }
    }
    copy_commit();
  };
  for (int s = 0; s < STAGES - 1; ++s) issue();

  // ---- the computing side.  This thread's query rows are 8 nb + 2 t4 and the next, nb < NB.
  float o[DT][NB][4], m[NB][2], l[NB][2];
  uint32_t qf[C::q_smem ? 1 : NB][C::q_smem ? 1 : KS][2];  // query fragments
  float c_row[Q8 && BFQ ? NB : 1][2];  // scores in base 2: scale log2(e) (k_scale) (2^e of a scaled fp16 query row)
  int stage = 0;
  bool fresh = true;  // the next unit opens an item
  long long item_begin = u_begin - use.chunk;
  for (long long u = u_begin; u < u_end; ++u) {
    const int h = use.k.blocks == 1 ? use.item : use.item / use.k.blocks;
    const int row0 = (use.item - h * use.k.blocks) * ROWS;
    if (fresh) {
      fresh = false;
#pragma unroll
      for (int n = 0; n < DT; ++n)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) o[n][nb][0] = o[n][nb][1] = o[n][nb][2] = o[n][nb][3] = 0.f;
      const float c = a.scale * kLog2e * (Q8 ? a.k_scale[h] : 1.f);
      c_row[0][0] = c_row[0][1] = c;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
        // The order of a row's elements in the steps follows the keys' reads: with 16-bit keys a
        // thread takes pieces 2 t, 2 t + 1 of 8 elements of each panel, with 8-bit keys those of 16.
        const int row = row0 + 8 * nb + g, i = row / G;
        const bool there = row < use.k.nq * G;
        const int64_t at = (int64_t)(use.k.q0 + i) * a.q_stride_token + (int64_t)(h * G + row - i * G) * a.q_stride_head;
        uint4 raw[KS / 2];
#pragma unroll
        for (int b = 0; b < KS / 2; ++b) {
          const int d = Q8 ? b / 4 * 128 + 32 * t4 + b % 4 * 8 : b / 2 * 64 + 16 * t4 + b % 2 * 8;
          raw[b] = make_uint4(0, 0, 0, 0);
          if (there && d < a.D) raw[b] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + d);
        }
        if (Q8 && BFQ) {
          // bf16 queries over an e4m3 cache: fp16 operands, the row scaled by a power of two to
          // a maximum in [1, 2) so that it fits fp16's range; what falls below 2^-24 of the
          // row's maximum is lost, far under the sums' rounding
          float top = 0.f;
#pragma unroll
          for (int b = 0; b < KS / 2; ++b) {
            const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = fmaxf(top, fmaxf(fabsf(Half16<true>::lo(w[e])), fabsf(Half16<true>::hi(w[e]))));
          }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          int e2 = 0;
          if (top > 0.f && top < INFINITY) e2 = min(max(ilogbf(top), -126), 126);
          const float down = ldexpf(1.f, -e2), up = c * ldexpf(1.f, e2);
          c_row[Q8 && BFQ ? nb : 0][0] = __shfl_sync(~0u, up, 8 * t4);  // of row 2 t4, held by lanes 4 (2 t4) ..
          c_row[Q8 && BFQ ? nb : 0][1] = __shfl_sync(~0u, up, 8 * t4 + 4);
#pragma unroll
          for (int b = 0; b < KS / 2; ++b) {
            uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = Half16<false>::pack(Half16<true>::lo(w[e]) * down, Half16<true>::hi(w[e]) * down);
            raw[b] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
#pragma unroll
        for (int b = 0; b < KS / 2; ++b) {
          if (C::q_smem) {  // this thread reads back what it wrote
            sts16(q_at + ((nb * (KS / 2) + b) * 32 + lane) * 16, raw[b]);
          } else {
            qf[C::q_smem ? 0 : nb][C::q_smem ? 0 : 2 * b][0] = raw[b].x;
            qf[C::q_smem ? 0 : nb][C::q_smem ? 0 : 2 * b][1] = raw[b].y;
            qf[C::q_smem ? 0 : nb][C::q_smem ? 0 : 2 * b + 1][0] = raw[b].z;
            qf[C::q_smem ? 0 : nb][C::q_smem ? 0 : 2 * b + 1][1] = raw[b].w;
          }
        }
      }
    }

    issue();
    copy_wait<STAGES - 1>();
    __syncwarp();
    const uint32_t keys = ring + stage * C::stage, values = keys + C::tile;

    // scores: s[mt][nb] = 16 tokens x 8 rows (tokens g, g + 8; rows 2 t4, 2 t4 + 1)
    float s[MT][NB][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) s[i][nb][0] = s[i][nb][1] = s[i][nb][2] = s[i][nb][3] = 0.f;
#pragma unroll
    for (int b = 0; b < C::chunks / 4; ++b) {  // pieces 2 t, 2 t + 1 of each panel
      const int c = b / 2 * 8 + 2 * t4 + b % 2;
      constexpr int kSteps = Q8 ? 4 : 2;  // steps that a piece feeds
      uint32_t q[NB][kSteps][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (C::q_smem) {
#pragma unroll
          for (int e = 0; e < kSteps / 2; ++e) {
            const uint4 v = lds16(q_at + ((nb * (KS / 2) + b * (kSteps / 2) + e) * 32 + lane) * 16);
            q[nb][2 * e][0] = v.x, q[nb][2 * e][1] = v.y, q[nb][2 * e + 1][0] = v.z, q[nb][2 * e + 1][1] = v.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kSteps; ++e)
#pragma unroll
            for (int z = 0; z < 2; ++z)
              q[nb][e][z] = qf[C::q_smem ? 0 : nb][C::q_smem ? 0 : kSteps * b + e][z];
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint4 lo = lds16(keys + piece_at<C::panel>(16 * i + g, c));
        const uint4 hi = lds16(keys + piece_at<C::panel>(16 * i + 8 + g, c));
        const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, y[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int e = 0; e < kSteps; ++e) {
          uint32_t k[4];
          if (Q8) {
            k[0] = e4m3_to_half2(x[e]), k[2] = e4m3_to_half2(x[e] >> 16);
            k[1] = e4m3_to_half2(y[e]), k[3] = e4m3_to_half2(y[e] >> 16);
          } else {
            k[0] = x[2 * e % 4], k[2] = x[(2 * e + 1) % 4], k[1] = y[2 * e % 4], k[3] = y[(2 * e + 1) % 4];
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) H::mma(s[i][nb], k, q[nb][e][0], q[nb][e][1]);
        }
      }
    }

    // mask and softmax about the running maximum less kLift
    const int p0 = use.k.first + use.chunk * TK;
    // a unit that not every query sees whole
    const bool edge = p0 + TK > use.k.len - use.k.nq + 1 || (a.window > 0 && p0 < use.k.len - a.window);
    float top[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float c = c_row[Q8 && BFQ ? nb : 0][z];
        top[nb][z] = -INFINITY;
        int last = 0x7FFFFFFF, low = 0;
        if (edge) {
          const int row = row0 + 8 * nb + 2 * t4 + z;
          last = row < use.k.nq * G ? use.k.len - use.k.nq + row / G : -1;
          if (a.window > 0) low = last - a.window + 1;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = z; e < 4; e += 2) {
            const int p = p0 + 16 * i + g + 8 * (e >> 1);
            s[i][nb][e] = p >= low && p <= last ? s[i][nb][e] * c : -INFINITY;
            top[nb][z] = fmaxf(top[nb][z], s[i][nb][e]);
          }
      }
    bool grows = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top[nb][z] = fmaxf(top[nb][z], __shfl_xor_sync(~0u, top[nb][z], d));
        top[nb][z] -= H::kLift;
        grows |= top[nb][z] > m[nb][z];
      }
    if (__any_sync(~0u, grows)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float now = fmaxf(m[nb][z], top[nb][z]);
          const float f = m[nb][z] == -INFINITY ? 0.f : ex2(m[nb][z] - now);
          m[nb][z] = now;
          l[nb][z] *= f;
#pragma unroll
          for (int n = 0; n < DT; ++n) {
            o[n][nb][z] *= f;
            o[n][nb][z + 2] *= f;
          }
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float ref = m[nb][z] == -INFINITY ? 0.f : m[nb][z];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = z; e < 4; e += 2) {
            s[i][nb][e] = ex2(s[i][nb][e] - ref);
            l[nb][z] += s[i][nb][e];
          }
      }

    // Rows that see different positions share this unit's values: one that is not finite must not
    // reach the rows that do not see it (0 x NaN).  Such a token is added on its own to the rows
    // that see it, and its row is cleared for the product.
    if (edge && (use.k.nq > 1 || a.window > 0)) {
      uint32_t odd = 0;  // bit i: token i holds a value that is not finite
      for (int i = 0; i < TK; ++i) {
        bool found = false;
        for (int c = lane; c < C::chunks; c += 32) {
          const uint4 v = lds16(values + piece_at<C::panel>(i, c));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (Q8) {
#pragma unroll
              for (int b = 0; b < 4; ++b) found |= ((w[e] >> (8 * b)) & 0x7F) == 0x7F;
            } else {
              found |= (w[e] & H::kExp) == H::kExp || ((w[e] >> 16) & H::kExp) == H::kExp;
            }
          }
        }
        if (__any_sync(~0u, found)) odd |= 1u << i;
      }
      while (odd) {
        const int at = __ffs(odd) - 1, p = p0 + at;
        odd &= odd - 1;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            // weight of (token, row 2 t4 + z): held by lane 4 (token % 8) + t4
            float w = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
              if (i == at / 16) {
                const float first = __shfl_sync(~0u, s[i][nb][z], (at % 8) * 4 + t4);
                const float second = __shfl_sync(~0u, s[i][nb][z + 2], (at % 8) * 4 + t4);
                w = at % 16 < 8 ? first : second;
              }
            const int row = row0 + 8 * nb + 2 * t4 + z;
            const int last = row < use.k.nq * G ? use.k.len - use.k.nq + row / G : -1;
            const bool sees = p <= last && (a.window == 0 || p > last - a.window);
#pragma unroll
            for (int n = 0; n < DT; ++n)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const int byte = element<Q8>(n, g + 8 * half) * C::kBytes;
                const uint32_t from = values + piece_at<C::panel>(at, byte / 16) + byte % 16;
                uint32_t x;
                if (Q8) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(from));
                else asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(from));
                const float v = Q8 ? Half16<false>::lo(e4m3_to_half2(x)) : H::lo(x);
                if (sees) o[n][nb][z + 2 * half] = fmaf(w, v, o[n][nb][z + 2 * half]);
              }
          }
        __syncwarp();
        for (int c = lane; c < C::chunks; c += 32) sts16(values + piece_at<C::panel>(at, c), make_uint4(0, 0, 0, 0));
        __syncwarp();
      }
    }

    // output (elements x rows) += values x weights.  The weights are rounded to the values' 16 bits,
    // as the instruction wants both operands; the normaliser adds them unrounded.  Each is off by
    // half a step (2^-8 relative at most for bf16, 2^-11 for fp16), independently: the outputs' error goes from
    // the 1.7e-3 of their own rounding to bf16 to 2.0e-3 (fp16: 2.1e-4 to 2.9e-4; relative, rms).
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      uint32_t p[NB][2];  // weights, transposed: tokens 2 t4 .. (and 8 on), row g
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        p[nb][0] = transpose8(H::pack(s[k][nb][0], s[k][nb][1]));
        p[nb][1] = transpose8(H::pack(s[k][nb][2], s[k][nb][3]));
      }
      if (!Q8) {
        // matrices (tokens 0-7 | 8-15) x (elements 0-7 | 8-15) of a tile of 16 elements
        const int i = 16 * k + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
        for (int n = 0; n < DT; ++n) {
          uint32_t v[4];
          ldmatrix_t(v, values + piece_at<C::panel>(i, 2 * n + ((lane >> 3) & 1)));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) H::mma(o[n][nb], v, p[nb][0], p[nb][1]);
        }
      } else {
        // a thread reads piece g of four token rows of each panel and pairs the bytes up
#pragma unroll
        for (int b = 0; b < C::panels; ++b) {
          uint32_t w[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 v = lds16(values + piece_at<C::panel>(16 * k + 8 * (q >> 1) + 2 * t4 + (q & 1), 8 * b + g));
            w[q][0] = v.x, w[q][1] = v.y, w[q][2] = v.z, w[q][3] = v.w;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // bytes 2 e, 2 e + 1 of the two tokens side by side: (r0[0] r1[0] r0[1] r1[1])
            const uint32_t which = e & 1 ? 0x7362 : 0x5140;
            const uint32_t x = __byte_perm(w[0][e / 2], w[1][e / 2], which), y = __byte_perm(w[2][e / 2], w[3][e / 2], which);
            const uint32_t v[4] = {e4m3_to_half2(x), e4m3_to_half2(x >> 16), e4m3_to_half2(y), e4m3_to_half2(y >> 16)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) H::mma(o[8 * b + e][nb], v, p[nb][0], p[nb][1]);
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
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nb][z] += __shfl_xor_sync(~0u, l[nb][z], d);
      const bool whole = item_begin >= u_begin && item_end <= u_end;
      // the worker's part 0 began before its range, part 1 begins in it
      const int part = item_begin >= u_begin;
      const size_t base = (size_t)(worker * 2 + part) * ROWS;
      const float vs = Q8 ? a.v_scale[h] : 1.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int r2 = 8 * nb + 2 * t4;  // this thread's rows r2, r2 + 1
        if (whole) {
          const float f0 = l[nb][0] == 0.f ? 0.f : vs / l[nb][0], f1 = l[nb][1] == 0.f ? 0.f : vs / l[nb][1];
          if (!Q8) {
            // packed by rows, then transposed: row g, elements 2 t4 ..
            const int rr = row0 + 8 * nb + g, i = rr / G;
            uint16_t* out = static_cast<uint16_t*>(a.out) + ((size_t)(use.k.q0 + i) * a.Hq + h * G + rr - i * G) * a.D;
#pragma unroll
            for (int n = 0; n < DT; ++n) {
              const uint32_t x = transpose8(Half16<BFQ>::pack(o[n][nb][0] * f0, o[n][nb][1] * f1));
              const uint32_t y = transpose8(Half16<BFQ>::pack(o[n][nb][2] * f0, o[n][nb][3] * f1));
              if (rr < use.k.nq * G && 16 * n < a.D) {
                *reinterpret_cast<uint32_t*>(out + 16 * n + 2 * t4) = x;
                *reinterpret_cast<uint32_t*>(out + 16 * n + 8 + 2 * t4) = y;
              }
            }
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int rr = row0 + r2 + z, i = rr / G;
            if (rr >= use.k.nq * G) continue;
            const size_t at = (size_t)(use.k.q0 + i) * a.Hq + h * G + rr - i * G;
            if (Q8) {
              uint16_t* out = static_cast<uint16_t*>(a.out) + at * a.D;
              const float f = z ? f1 : f0;
#pragma unroll
              for (int n = 0; n < DT; ++n) {
                const int d = element<Q8>(n, g);  // and the next one
                if (d < a.D)
                  *reinterpret_cast<uint32_t*>(out + d) = Half16<BFQ>::pack(o[n][nb][z] * f, o[n][nb][z + 2] * f);
              }
            }
            if (g == 0 && a.lse_out != nullptr)
              a.lse_out[at] = l[nb][z] == 0.f ? -INFINITY : (m[nb][z] + log2f(l[nb][z])) * kLn2;
          }
        } else {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (g == 0) scr.stats[base + r2 + z] = make_float2(m[nb][z], l[nb][z]);
            float* out = scr.out + (base + r2 + z) * DP;
#pragma unroll
            for (int n = 0; n < DT; ++n) {
              if (Q8) {
                *reinterpret_cast<float2*>(out + element<Q8>(n, g)) = make_float2(o[n][nb][z], o[n][nb][z + 2]);
              } else {
                out[element<Q8>(n, g)] = o[n][nb][z];
                out[element<Q8>(n, g + 8)] = o[n][nb][z + 2];
              }
            }
          }
        }
      }
      if (!whole && part == 1 && lane == 0)
        scr.share[worker] = Share{use.r, use.item, use.k.q0, use.k.nq, item_begin, item_end};
      fresh = true;
      item_begin = item_end;
    }
    advance<TK, ROWS>(a, use);
  }
}

// Tokens per unit, warps, ring stages and CTAs per SM: 130 to 200 KB of ring per SM, and as many
// warps as the registers of the outputs (DP NB / 8 per thread) leave.
template <bool Q8, int DP, int NB>
struct Shape {
  static constexpr int TK = !Q8 && DP >= 128 ? 16 : 32;
  static constexpr int warps = 4;
  static constexpr int stages = NB == 4 ? 2 : 3;
  static constexpr int ctas = DP == 256 ? 1 : 2;  // per SM
};

constexpr int kMaxWorkers = kMaxSms * 2 * 4;

// Query rows of a cache head (at most, over the requests) above which the other kernel is faster:
// 32 requests of 1 K to 8 K tokens, 16-bit cache: 12 rows 110 us here and 110 there, 16 rows 104 and
// 102, 20 rows 145 and 112; e4m3 cache: 12 rows 79 and 98, 16 rows 86 and 106, 20 rows 164 and 113.
// Rows of 64 elements: 16 rows 85 and 83, 24 rows 113 and 85, 64 rows 171 and 104.  200 requests of 50
// to 600 tokens: 16 rows 85 and 118, 24 rows 136 and 121, 64 rows 201 and 158; with 64 elements 24 rows
// 100 and 125, 32 rows 110 and 109; with an e4m3 cache 32 rows 195 and 177, 64 rows 274 and 307.  (The
// lengths are on the device, so the rule cannot ask for them.)
constexpr int kWideRows = 16;

int padded(int D, bool q8) { return D <= 64 && !q8 ? 64 : (D <= 128 ? 128 : 256); }  // (8-bit panels hold 128 elements)
// Groups of eight query rows per item: what the call's largest block needs, up to 32 rows (their
// outputs fill the registers; 16 with rows of 256 elements).
int groups(int D, int max_q, int G) {
  const int rows = max_q * G;
  return rows <= 8 ? 1 : (rows <= 16 || D > 128 ? 2 : 4);
}

template <bool BFQ, bool Q8, int DP, int NB>
cudaError_t launch(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  using S = Shape<Q8, DP, NB>;
  using C = Cfg<Q8, DP, NB, S::TK, S::warps, S::stages>;
  static_assert(S::ctas * S::warps <= kMaxWorkers / kMaxSms, "scratch");
  auto* kernel = attention_kernel<BFQ, Q8, DP, NB, S::TK, S::warps, S::stages, S::ctas>;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(kernel, C::smem, done);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count(), kMaxSms) * S::ctas, workers = grid * S::warps;
  const Scratch scr = scratch_at(scratch, kMaxWorkers, 8 * NB);
  e = launch_chained(kernel, dim3(grid), dim3(S::warps * 32), C::smem, s, 1, a, scr);
  return e != cudaSuccess ? e : launch_join<BFQ, DP, 8 * NB>(a, scr, workers, s);
}

template <bool BFQ, bool Q8, int DP>
cudaError_t launch(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  const int n = groups(a.D, a.max_q, a.G);
  if (n == 1) return launch<BFQ, Q8, DP, 1>(a, scratch, s);
  if constexpr (DP <= 128)
    if (n == 4) return launch<BFQ, Q8, DP, 4>(a, scratch, s);
  return launch<BFQ, Q8, DP, 2>(a, scratch, s);
}

template <bool BFQ, bool Q8>
cudaError_t launch(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  const int D = padded(a.D, Q8);
  if constexpr (!Q8)
    if (D == 64) return launch<BFQ, Q8, 64>(a, scratch, s);
  return D == 128 ? launch<BFQ, Q8, 128>(a, scratch, s) : launch<BFQ, Q8, 256>(a, scratch, s);
}

}  // namespace

size_t paged_attention_scratch(int, int, int Hq, int Hkv, int D, int max_q) {
  return std::max(scratch_bytes(kMaxWorkers, 8 * groups(D, max_q, Hq / Hkv), padded(D, true)),
                  attention_wide_scratch(Hq, Hkv, D, max_q));
}

size_t attention_rows_scratch(int Hq, int Hkv, int D) {
  return scratch_bytes(kMaxWorkers, 8 * groups(D, kMaxQueries, Hq / Hkv), padded(D, true));
}

cudaError_t launch_paged_attention(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  cudaError_t e;
  if (a.max_q * a.G > kWideRows && launch_attention_wide(a, scratch, s, e)) return e;
  return launch_attention_rows(a, scratch, s);
}

cudaError_t launch_attention_rows(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  const bool q8 = a.dtype_kv == DSPARK_E4M3;
  if (a.dtype_q == DSPARK_BF16) return q8 ? launch<true, true>(a, scratch, s) : launch<true, false>(a, scratch, s);
  return q8 ? launch<false, true>(a, scratch, s) : launch<false, false>(a, scratch, s);
}

}  // namespace dspark
