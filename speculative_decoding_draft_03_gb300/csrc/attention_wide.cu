// attention_wide.cu — attention of larger blocks of queries over a paged cache, on the
// 5th-generation tensor cores.
//
// With many query rows per cache head (G heads times the verified block's queries) the products
// outgrow the register-operand instructions; here both run as tcgen05.mma with the tokens, then
// the value elements, as the 128 rows and the query rows as the N columns:
//   S [128 tokens x N]   = K [128 tokens x D] . Q^T    (both K-major)
//   O [128 elements x N] += V^T [elements x 128 tokens] . P   (both MN-major)
// so that keys and values are used as they lie in the pages (panels of 128-byte rows, 128-byte
// swizzle, by tensor copies), each weight is written once as part of a 16-byte piece of its
// token's row, and the output leaves with its elements in neighbouring lanes.
//   * One persistent CTA per SM: warps 0 and 2 copy, warp 1 issues the products, the other 8 or 16
//     do the softmax: a thread owns one token (its TMEM lane) and 16 or 32 of the columns.  S is
//     double buffered; the copies run up to three tiles ahead of the products.
//   * An e4m3 cache is copied as it is; four more warps turn each tile into fp16 (which holds every
//     e4m3 value) for the products.  bf16 query rows are scaled by powers of two into fp16's range.
//   * The softmax reference of a column moves only when a score passes the one that set it by
//     2^kSlack (any reference is right; the weights stay below 2^(kSlack + kLift), inside fp16's
//     range): a vote per tile replaces the maximum over the tokens, and the output is rescaled in
//     TMEM only then.
//   * The work is dealt out in tiles of 128 tokens as for the other kernel, a CTA per worker.
// What bounds it: to 32 columns the device memory (the verified block of 32 requests of 1 K to 8 K
// tokens: 640 MB in 113 us, 5.7 TB/s; items' starts and ends cost the rest); from 64 on the chain
// of a tile from its scores over the weights to its product (64 rows: 133 us, 128 rows: 196 us or
// 236 TFLOP/s: no weight is stored before the last tile's product has ended), and the item's drain
// where contexts are short (200 requests of 50 to 600 tokens, 64 rows: 149 us); with an e4m3 cache
// the chain of copy, conversion and product (32 rows: 112 us, some 3000 cycles a tile, of which its
// 210 KB of shared-memory traffic are 1640; the keys' converted tile is single buffered, and the same
// warps convert keys and values in turn).
// Every mbarrier wait is bounded; a wait that gives up reports DSPARK_TIMEOUT and the CTA winds
// down (the softmax warps leave together, by a vote).
#include <algorithm>

#include "attention_tc.cuh"
#include "attention_wide.h"

namespace dspark {
namespace {

using namespace attention;

// Softmax warps: four lane quarters times the column groups, of 16 or 32 columns.  (With the four
// converting warps of an e4m3 cache 16 of them would leave 80 registers a thread.)
constexpr int softmax_warps(bool q8, int N) { return q8 || N == 32 ? 8 : 16; }
constexpr int kConvertWarps = 4;

// Barriers of the softmax warps.
template <int THREADS>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(THREADS)
      : "memory");
  return r != 0;
}
// ------------------------------------------------------------------------- shared memory

template <bool Q8, int DP, int N>
struct Plan {
  static constexpr int first_softmax = Q8 ? 3 + kConvertWarps : 3;  // warp
  static constexpr int softmax = 32 * softmax_warps(Q8, N), threads = 32 * first_softmax + softmax;
  static constexpr int groups = softmax_warps(Q8, N) / 4, columns = N / groups;  // column groups
  static constexpr int panels = DP / 64;             // of 16-bit elements
  static constexpr int tile = panels * kTile * 128;  // keys, or values, of a tile, as the products read them
  static constexpr int copied = Q8 ? kTile * 128 : tile;  // ... and as they are copied
  static constexpr int copy_panels = Q8 ? 1 : panels;
  static constexpr int k_stages = DP == 64 ? 4 : 3, v_stages = DP == 64 ? 4 : (N == 128 ? 2 : 3);
  static constexpr int tmem_cols = N == 32 ? 128 : (N == 64 ? 256 : 512);  // S twice, O: 3 N, a power of two
  // offsets, on 1 KB boundaries where products or copies read or write
  static constexpr int q = 0;                                        // [panels][N][128]
  static constexpr int p = q + panels * N * 128;                     // [(N + 63) / 64][128 tokens][128]
  static constexpr int k = p + (N + 63) / 64 * kTile * 128;          // [k_stages][copied]
  static constexpr int v = k + k_stages * copied;                    // [v_stages][copied]
  static constexpr int k16 = v + v_stages * copied;                  // e4m3: [tile] keys, then [2][tile] values, as fp16
  static constexpr int v16 = k16 + (Q8 ? tile : 0);
  static constexpr int reference = v16 + (Q8 ? 2 * tile : 0);        // [N] float
  static constexpr int factor = reference + 4 * N;                   // [N] float: rescaling, or one token's weights
  static constexpr int sums = p;                                     // [4][N] float, while the weights are not in use
  static constexpr int last = factor + 4 * N;                        // [N] int: the last position a column sees
  static constexpr int place = last + 4 * N;                         // [N] int: its row of the output, or -1
  static constexpr int up = place + 4 * N;                           // [N] float: scores in base 2 per product
  static constexpr int odd = up + (Q8 ? 4 * N : 0);                  // [128] bytes: tokens to be added on their own
  static constexpr int bars = odd + 128;
  static constexpr int n_bars = 2 * (k_stages + v_stages) + 8 + (Q8 ? 6 : 0);
  static constexpr int start_off = bars + 8 * n_bars;                // long long
  static constexpr int scan = start_off + 8;                         // [threads / 32] long long
  static constexpr int start_r = scan + 8 * (threads / 32);          // int
  static constexpr int tmem = start_r + 4, abort_flag = tmem + 4;
  static constexpr int total = abort_flag + 4;
  static_assert(total <= 232448, "227 KB");
};

template <bool BFQ, bool Q8, int DP, int N>
__global__ void __launch_bounds__(Plan<Q8, DP, N>::threads, 1)
    attention_wide_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Maps maps, int box, Scratch scr) {
  using L = Plan<Q8, DP, N>;
  using H = Half16<BFQ && !Q8>;  // type of the products
  constexpr int C = L::columns;  // per softmax thread
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return base + L::bars + 8 * i; };
  const int k_full = 0, k_empty = L::k_stages, v_full = 2 * L::k_stages, v_empty = v_full + L::v_stages,
            s_full = v_empty + L::v_stages, s_free = s_full + 2, p_ready = s_free + 2, o_done = p_ready + 1,
            q_ready = o_done + 1, drained = q_ready + 1,
            k16_full = drained + 1, k16_empty = k16_full + 1, v16_full = k16_empty + 1, v16_empty = v16_full + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::abort_flag);
  const long long worker = blockIdx.x, workers = gridDim.x;
  const int G = a.G;

  if (tid == 0) {
    constexpr int readers = Q8 ? kConvertWarps : 1;  // of a copied tile
    for (int i = 0; i < L::k_stages; ++i) mbar_init(bar(k_full + i), 1), mbar_init(bar(k_empty + i), readers);
    for (int i = 0; i < L::v_stages; ++i) mbar_init(bar(v_full + i), 1), mbar_init(bar(v_empty + i), readers);
    if (Q8) {
      mbar_init(bar(k16_full), kConvertWarps);
      mbar_init(bar(k16_empty), 1);
      for (int i = 0; i < 2; ++i) mbar_init(bar(v16_full + i), kConvertWarps), mbar_init(bar(v16_empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(bar(s_full + i), 1), mbar_init(bar(s_free + i), L::softmax / 32);
    mbar_init(bar(p_ready), L::softmax / 32);
    mbar_init(bar(o_done), 1);
    mbar_init(bar(q_ready), L::softmax / 32);
    mbar_init(bar(drained), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 128) smem[L::odd + tid] = 0;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + L::tmem), "r"(L::tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  griddep_wait();
  griddep_allow_next();
  const Deal d = deal<kTile, N, 1, L::threads>(a, worker, workers, reinterpret_cast<long long*>(smem + L::scan),
                                             reinterpret_cast<int*>(smem + L::start_r),
                                             reinterpret_cast<long long*>(smem + L::start_off));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::tmem), o_cols = tmem + 2 * N;
  if (tid == 0) {
    scr.share[worker].r = -1;
    if (worker == 0) *scr.per = d.per;
  }
  const long long u_begin = worker * d.per, u_end = min(d.total, u_begin + d.per);
  const bool aligned = (base & 1023u) == 0;  // (as the swizzle wants; so it is without static shared memory)
  if (!aligned && tid == 0) report_bad_input(a.status, 612);
  const bool work = aligned && u_begin < u_end;
  Cursor use = {};
  if (work)
    use = stand<kTile, N>(a, *reinterpret_cast<int*>(smem + L::start_r), *reinterpret_cast<long long*>(smem + L::start_off));
  const int tiles = work ? (int)(u_end - u_begin) : 0;

  if (warp == 0 || warp == 2) {
    // ---- copies, of keys (warp 0) and of values (warp 2: issuing a tile's boxes takes a warp
    // most of a tile's time): a lane per box of a tile, its page looked up one tile ahead
    const bool keys = warp == 0;
    const int stages = keys ? L::k_stages : L::v_stages, full = keys ? k_full : v_full, empty = keys ? k_empty : v_empty;
    const uint32_t ring = base + (keys ? L::k : L::v);
    const CUtensorMap* map = keys ? &maps.k : &maps.v;
    const int boxes = kTile / box;
    int page = -1, slot = 0;
    bool inside = false;
    auto look_up = [&]() {
      const int pos = use.k.first + use.chunk * kTile + lane * box, nth = pos / a.page_size;
      slot = pos - nth * a.page_size;
      inside = lane < boxes && pos < use.k.len && seen(a, use.k, pos + box - 1);
      page = inside ? a.page_table[use.r * a.table_stride + nth] : -1;
    };
    if (tiles > 0) look_up();
    int filled = 0, stage = 0, phase = 1;  // (the first round finds every stage empty)
    for (int i = 0; i < tiles; ++i) {
      const int h = use.k.blocks == 1 ? use.item : use.item / use.k.blocks;
      const bool there = page >= 0 && page < a.num_pages;
      if (inside && !there) report_bad_input(a.status, kBadPage);
      const int from = there ? page : a.num_pages;  // past the pool: zeros
      if (i >= stages && !mbar_wait(bar(empty + stage), phase, abort_flag, a.status, 601)) break;
      if (lane == 0) mbar_expect(bar(full + stage), L::copied);
      __syncwarp();
      if (lane < boxes)
#pragma unroll
        for (int n = 0; n < L::copy_panels; ++n)
          tma_box(ring + stage * L::copied + n * (kTile * 128) + lane * box * 128, map, bar(full + stage), 64 * n, slot, h, from);
      filled = i + 1;
      if (++stage == stages) stage = 0, phase ^= 1;
      if (i + 1 < tiles) {
        advance<kTile, N>(a, use);
        look_up();
      }
    }
    // every copy lands before the CTA ends (at once, unless a role gave up)
    for (int i = max(0, filled - stages); i < filled; ++i) mbar_drain(bar(full + i % stages), (i / stages) & 1);
  } else if (warp == 1) {
    // ---- products
    if (lane == 0) {
      constexpr uint32_t s_desc = idesc<BFQ && !Q8>(N, false, false), o_desc = idesc<BFQ && !Q8>(N, true, true);
      // descriptors of the first step; the others lie a constant further (in units of 16 bytes)
      const uint64_t k_first = sw128(base + (Q8 ? L::k16 : L::k), 16, 1024), q_first = sw128(base + L::q, 16, 1024);
      // (rows of 64 elements: the upper half of the product repeats the lower)
      const uint64_t v_first = sw128(base + (Q8 ? L::v16 : L::v), L::panels > 1 ? kTile * 128 : 0, 1024),
                     p_first = sw128(base + L::p, kTile * 128, 1024);
      auto scores = [&](int i) {
        const int ks = Q8 ? 0 : i % L::k_stages;
        if (!(Q8 ? mbar_wait(bar(k16_full), i & 1, abort_flag, a.status, 603)
                 : mbar_wait(bar(k_full + ks), (i / L::k_stages) & 1, abort_flag, a.status, 603)))
          return false;
        if (i >= 2 && !mbar_wait(bar(s_free + (i & 1)), (i / 2 - 1) & 1, abort_flag, a.status, 604)) return false;
        fence_after();
        const uint64_t keys = k_first + (uint32_t)(ks * (L::tile / 16));
        const uint32_t to = tmem + (i & 1) * N;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
          mma(to, keys + (kk / 4 * (kTile * 8) + kk % 4 * 2), q_first + (kk / 4 * (N * 8) + kk % 4 * 2), s_desc, kk > 0);
        commit(bar(s_full + (i & 1)));
        commit(bar(Q8 ? k16_empty : k_empty + ks));
        return true;
      };
      int i = 0, items = 0;
      bool ok = true;
      while (ok && i < tiles) {
        const int n = min(use.k.chunks - use.chunk, tiles - i);  // tiles of this item
        ok = mbar_wait(bar(q_ready), items & 1, abort_flag, a.status, 605) && scores(i);
        for (int t = 0; ok && t < n; ++t, ++i) {
          if (t + 1 < n && !scores(i + 1)) ok = false;
          const int vs = Q8 ? i & 1 : i % L::v_stages;
          ok = ok && mbar_wait(bar((Q8 ? v16_full : v_full) + vs), (Q8 ? i / 2 : i / L::v_stages) & 1, abort_flag, a.status, 606) &&
               mbar_wait(bar(p_ready), i & 1, abort_flag, a.status, 607);
          if (!ok) break;
          fence_after();
          const uint64_t values = v_first + (uint32_t)(vs * (L::tile / 16));
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) mma(o_cols, values + kk * 128, p_first + kk * 128, o_desc, 1);
          commit(bar(o_done));
          commit(bar((Q8 ? v16_empty : v_empty) + vs));
        }
        ++items;
        use.chunk = use.k.chunks - 1;
        if (i < tiles) advance<kTile, N>(a, use);
      }
      // every product is done before the CTA gives its tensor memory back
      commit(bar(drained));
      mbar_drain(bar(drained), 0);
    }
    __syncwarp();
  } else if (Q8 && warp < L::first_softmax) {
    // ---- e4m3 to fp16: a thread per token, 16 elements (one piece) into two pieces at a time
    const int token = tid - 96;
    auto convert = [&](uint32_t from, uint32_t to) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 x = lds16(from + token * 128 + ((c ^ (token & 7)) << 4));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[2 * e] = e4m3_to_half2(w[e]), h[2 * e + 1] = e4m3_to_half2(w[e] >> 16);
        const uint32_t row = to + (c >> 2) * (kTile * 128) + token * 128;
        const int piece = 2 * c & 7;
        sts16(row + ((piece ^ (token & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
        sts16(row + (((piece + 1) ^ (token & 7)) << 4), make_uint4(h[4], h[5], h[6], h[7]));
      }
      fence_smem();
      __syncwarp();
    };
    for (int i = 0; i < tiles; ++i) {
      const int ks = i % L::k_stages, vs = i % L::v_stages;
      if (!mbar_wait(bar(k_full + ks), (i / L::k_stages) & 1, abort_flag, a.status, 613)) break;
      if (i >= 1 && !mbar_wait(bar(k16_empty), (i - 1) & 1, abort_flag, a.status, 614)) break;
      convert(base + L::k + ks * L::copied, base + L::k16);
      if (lane == 0) mbar_arrive(bar(k_empty + ks)), mbar_arrive(bar(k16_full));
      if (!mbar_wait(bar(v_full + vs), (i / L::v_stages) & 1, abort_flag, a.status, 615)) break;
      if (i >= 2 && !mbar_wait(bar(v16_empty + (i & 1)), (i / 2 - 1) & 1, abort_flag, a.status, 616)) break;
      convert(base + L::v + vs * L::copied, base + L::v16 + (i & 1) * L::tile);
      if (lane == 0) mbar_arrive(bar(v_empty + vs)), mbar_arrive(bar(v16_full + (i & 1)));
    }
    __syncwarp();
  } else {
    // ---- softmax
    const int st = tid - 32 * L::first_softmax, quarter = warp & 3, group = (warp - L::first_softmax) >> 2, token = quarter * 32 + lane, c0 = group * C;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    float* reference = reinterpret_cast<float*>(smem + L::reference);
    float* factor = reinterpret_cast<float*>(smem + L::factor);
    float* sums = reinterpret_cast<float*>(smem + L::sums);
    int* last = reinterpret_cast<int*>(smem + L::last);
    int* place = reinterpret_cast<int*>(smem + L::place);
    volatile unsigned char* odd = smem + L::odd;
    float* up = reinterpret_cast<float*>(smem + L::up);
    // The query rows of an item, 16-byte pieces per thread; they are asked for while the item before
    // is drained (short contexts change items every few tiles), but with 128 columns, whose warps
    // have no registers left (64 query rows: 130 us so, 134 us without; 128 rows: 204 and 194).
    constexpr int kQ = N * (DP / 8) / L::softmax;
    static_assert(kQ * L::softmax == N * (DP / 8), "whole pieces");
    constexpr bool kAhead = N <= 64;
    const float per_g = 1.f / (float)G;
    auto query_of = [&](int row) { return (int)(((float)row + 0.5f) * per_g); };  // row / G, exact below 2^20
    uint4 ahead[kQ];
    auto fetch_q = [&]() {
      const int h = use.k.blocks == 1 ? use.item : use.item / use.k.blocks, row0 = (use.item - h * use.k.blocks) * N;
#pragma unroll
      for (int j = 0; j < kQ; ++j) {
        const int e = st + j * L::softmax, c = e % (DP / 8), rr = row0 + e / (DP / 8), q = query_of(rr);
        ahead[j] = make_uint4(0, 0, 0, 0);
        if (rr < use.k.nq * G && c * 8 < a.D)
          ahead[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                     (int64_t)(use.k.q0 + q) * a.q_stride_token +
                                                     (int64_t)(h * G + rr - q * G) * a.q_stride_head + c * 8);
      }
    };
    float l[C];
    bool ok = true;
    int i = 0;
    long long item_begin = u_begin - use.chunk;
    if (kAhead && tiles > 0) fetch_q();
    while (i < tiles) {
      const int n = min(use.k.chunks - use.chunk, tiles - i);
      const int h = use.k.blocks == 1 ? use.item : use.item / use.k.blocks, row0 = (use.item - h * use.k.blocks) * N;
      const float c2 = a.scale * kLog2e * (Q8 ? a.k_scale[h] : 1.f);  // scores in base 2 per product (e4m3: `up`)
      softmax_sync<L::softmax>();  // the previous item's tables are no longer read
      if (!kAhead) fetch_q();
#pragma unroll
      for (int j = 0; j < kQ; ++j) {
        const int e = st + j * L::softmax, row = e / (DP / 8), c = e % (DP / 8);
        uint4 x = ahead[j];
        if (Q8) {
          // fp16 operands; a bf16 row is scaled by a power of two to a maximum in [1, 2) (what falls
          // below 2^-24 of it is lost, far under the sums' rounding).  16 lanes hold a row.
          static_assert(!Q8 || DP == 128, "a row per half warp");
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
          int e2 = 0;
          if (BFQ) {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              top = max3(top, fabsf(Half16<true>::lo(w[k])), fabsf(Half16<true>::hi(w[k])));
#pragma unroll
            for (int s = 8; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, s));
            if (top > 0.f && top < INFINITY) e2 = min(max(ilogbf(top), -126), 126);
            const float down = ldexpf(1.f, -e2);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = Half16<false>::pack(Half16<true>::lo(w[k]) * down, Half16<true>::hi(w[k]) * down);
          }
          if (c == 0) up[row] = c2 * ldexpf(1.f, e2);
          x = make_uint4(w[0], w[1], w[2], w[3]);
        }
        sts16(base + L::q + (c >> 3) * (N * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4), x);
      }
      fence_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(q_ready));  // the first scores are computed meanwhile
      if (st < N) {
        const int rr = row0 + st, q = query_of(rr);
        const bool there = rr < use.k.nq * G;
        reference[st] = kUnset;
        last[st] = there ? use.k.len - use.k.nq + q : -1;
        place[st] = there ? (use.k.q0 + q) * a.Hq + h * G + rr - q * G : -1;
      }
      {
        float zero[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) zero[e] = 0.f;
#pragma unroll
        for (int c = 0; c < C; c += 16) tmem_store(o_cols + lanes + c0 + c, zero);
        tmem_store_wait();
      }
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] = 0.f;
      fence_before();
      softmax_sync<L::softmax>();

      for (int t = 0; t < n; ++t, ++i) {
        ok = ok && mbar_wait(bar(s_full + (i & 1)), (i >> 1) & 1, abort_flag, a.status, 608);
        fence_after();
        const int p0 = use.k.first + (use.chunk + t) * kTile, pos = p0 + token;
        const bool edge = p0 + kTile > use.k.len - use.k.nq + 1 || (a.window > 0 && p0 < use.k.len - a.window);
        // 16 columns of this token's scores (products), those that a column does not see -inf.  A
        // warp with 16 columns holds them; one with 32 reads them again at each use, its registers
        // being full of sums (128 query rows: 211 us so, 282 us with 32 held; 64 query rows, whose
        // warps have 16: 156 us so, 141 us held; both before the items overlapped).
        constexpr bool kHeld = C == 16;
        float x[16];
        auto release = [&]() {  // S may be written again
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(s_free + (i & 1)));
        };
        auto fetch = [&](int c) {
          tmem_load(tmem + (i & 1) * N + lanes + c0 + c, x);
          if (kHeld) release();
          if (edge) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int to = last[c0 + c + e];
              if (pos > to || (a.window > 0 && pos <= to - a.window)) x[e] = -INFINITY;
            }
          }
        };
        auto refetch = [&](int c) {
          if (!kHeld) fetch(c);
        };
        auto scale_of = [&](int c) {
          return Q8 ? *reinterpret_cast<const float4*>(up + c0 + c) : make_float4(c2, c2, c2, c2);
        };
        // scores to weights about the references (a masked score has weight 0 whatever the scale's sign)
        auto weigh = [&](int c) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 r = *reinterpret_cast<const float4*>(reference + c0 + c + e), k = scale_of(c + e);
            const float rr[4] = {r.x, r.y, r.z, r.w}, kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[e + j] = edge && x[e + j] == -INFINITY ? 0.f : ex2(fmaf(x[e + j], kk[j], -rr[j]));
          }
        };
        auto add = [&](int c) {
#pragma unroll
          for (int e = 0; e < 16; ++e) l[c + e] += x[e];
        };

        // does a score pass its reference?
        float most = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; c += 16) {
          fetch(c);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 r = *reinterpret_cast<const float4*>(reference + c0 + c + e), k = scale_of(c + e);
            const float u0 = fmaf(x[e], k.x, -r.x), u1 = fmaf(x[e + 1], k.y, -r.y), u2 = fmaf(x[e + 2], k.z, -r.z),
                        u3 = fmaf(x[e + 3], k.w, -r.w);
            most = max3(most, edge && x[e] == -INFINITY ? -INFINITY : u0, edge && x[e + 1] == -INFINITY ? -INFINITY : u1);
            most = max3(most, edge && x[e + 2] == -INFINITY ? -INFINITY : u2, edge && x[e + 3] == -INFINITY ? -INFINITY : u3);
          }
        }
        bool waited = false;  // for the previous tile's product into O
        auto wait_o = [&]() {
          if (!waited && i > 0) ok = mbar_wait(bar(o_done), (i - 1) & 1, abort_flag, a.status, 609) && ok;
          waited = true;
        };
        if (softmax_any<L::softmax>(most > kSlack + H::kLift || !ok)) {
          if (softmax_any<L::softmax>(!ok)) goto done;
          wait_o();
          softmax_sync<L::softmax>();
          // new references: the columns' maxima, over lanes, then over the four quarters
#pragma unroll
          for (int c = 0; c < C; c += 16) {
            refetch(c);
            float mine = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float v = warp_max(edge && x[e] == -INFINITY ? -INFINITY : x[e] * (Q8 ? up[c0 + c + e] : c2));
              if (lane == e) mine = v;
            }
            if (lane < 16) sums[quarter * N + c0 + c + lane] = mine;
          }
          softmax_sync<L::softmax>();
          if (st < N) {
            const float was = reference[st];
            const float now = fmaxf(
                was, fmaxf(fmaxf(sums[st], sums[N + st]), fmaxf(sums[2 * N + st], sums[3 * N + st])) - H::kLift);
            reference[st] = now;
            factor[st] = ex2(was - now);
          }
          softmax_sync<L::softmax>();
          if (t > 0) {  // (an item's first tile finds its outputs and sums empty)
            fence_after();
#pragma unroll
            for (int c = 0; c < C; c += 16) {
              float o[16];
              tmem_load(o_cols + lanes + c0 + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float f = factor[c0 + c + e];
                o[e] *= f;
                l[c + e] *= f;
              }
              tmem_store(o_cols + lanes + c0 + c, o);
            }
            tmem_store_wait();
          }
        }
        if (kHeld) {
          weigh(0);
          add(0);
          wait_o();
        }
        if (edge) {
          wait_o();
          // Tokens that no column sees hold anything (the rest of a page): their values are
          // cleared.  One that only some columns see must not reach the others if it is not
          // finite (0 x NaN): it is added on its own, and cleared for the product.
          const int vs = Q8 ? i & 1 : i % L::v_stages;
          ok = mbar_wait(bar((Q8 ? v16_full : v_full) + vs), (Q8 ? i / 2 : i / L::v_stages) & 1, abort_flag, a.status, 610) && ok;
          const uint32_t values = base + (Q8 ? L::v16 : L::v) + vs * L::tile;
          constexpr int kPieces = L::panels * 8 / L::groups;  // this thread's part of the token's row
          auto part_of_row = [&](int c) {
            const int piece = group * kPieces + c;
            return values + (piece >> 3) * (kTile * 128) + token * 128 + (((piece & 7) ^ (token & 7)) << 4);
          };
          const int seen_from = a.window > 0 ? max(0, use.k.len - use.k.nq - a.window + 1) : 0;
          const bool unseen = pos >= use.k.len || pos < seen_from;
          const bool partly = !unseen && (pos > use.k.len - use.k.nq || (a.window > 0 && pos < use.k.len - a.window));
          bool strange = false;
          if (partly) {
            for (int c = 0; c < kPieces; ++c) {
              const uint4 v = lds16(part_of_row(c));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) strange |= (w[e] & H::kExp) == H::kExp || ((w[e] >> 16) & H::kExp) == H::kExp;
            }
          }
          if (strange) odd[token] = 1;
          if (softmax_any<L::softmax>(strange)) {
            for (int k = 0; k < kTile; ++k) {
              if (!odd[k]) continue;
#pragma unroll
              for (int c = 0; c < C; c += 16) {
                if (!kHeld) {
                  fetch(c);
                  weigh(c);
                }
                if (token == k) {
#pragma unroll
                  for (int e = 0; e < 16; ++e) factor[c0 + c + e] = x[e];
                }
              }
              softmax_sync<L::softmax>();
              fence_after();
              // this thread: element `token` of the value, its group of the columns
              float v = 0.f;
              if (token < DP) {
                const uint32_t at = values + (token >> 6) * (kTile * 128) + k * 128 + ((((token & 63) >> 3) ^ (k & 7)) << 4) +
                                    (token & 7) * 2;
                uint32_t w;
                asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w) : "r"(at));
                v = H::lo(w);
              }
#pragma unroll
              for (int c = 0; c < C; c += 16) {
                float o[16];
                tmem_load(o_cols + lanes + c0 + c, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const int to = last[c0 + c + e], p = p0 + k;
                  if (p <= to && (a.window == 0 || p > to - a.window)) o[e] = fmaf(factor[c0 + c + e], v, o[e]);
                }
                tmem_store(o_cols + lanes + c0 + c, o);
              }
              tmem_store_wait();
              softmax_sync<L::softmax>();
            }
          }
          const bool clear = unseen || odd[token];
          softmax_sync<L::softmax>();
          odd[token] = 0;
          if (clear)
            for (int c = 0; c < kPieces; ++c) sts16(part_of_row(c), make_uint4(0, 0, 0, 0));
        }
        // the weights: C 16-bit values of the token's row (rounded as the instruction wants both
        // operands; the normaliser adds them unrounded)
#pragma unroll
        for (int c = 0; c < C; c += 16) {
          if (!kHeld) {
            fetch(c);
            weigh(c);
            add(c);
          }
          wait_o();  // the previous weights have been used
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            const int piece = (c0 + c + e) / 8;
            sts16(base + L::p + (piece >> 3) * (kTile * 128) + token * 128 + (((piece & 7) ^ (token & 7)) << 4),
                  make_uint4(H::pack(x[e], x[e + 1]), H::pack(x[e + 2], x[e + 3]), H::pack(x[e + 4], x[e + 5]),
                             H::pack(x[e + 6], x[e + 7])));
          }
        }
        if (!kHeld) release();
        fence_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(p_ready));
      }

      // ---- the item, or this worker's part of it, ends
      const long long item_end = item_begin + use.k.chunks;
      const Share ended{use.r, use.item, use.k.q0, use.k.nq, item_begin, item_end};
      use.chunk = use.k.chunks - 1;
      if (i < tiles) {
        advance<kTile, N>(a, use);
        if (kAhead) fetch_q();
      }
      ok = mbar_wait(bar(o_done), (i - 1) & 1, abort_flag, a.status, 611) && ok;
      fence_after();
      if (softmax_any<L::softmax>(!ok)) goto done;
      // the columns' sums over the warp, 16 at a time: each step halves the columns a lane holds
#pragma unroll
      for (int c = 0; c < C; c += 16) {
#pragma unroll
        for (int w = 8; w; w >>= 1) {
          const bool upper = lane & (2 * w);
#pragma unroll
          for (int e = 0; e < w; ++e) {
            const float keep = upper ? l[c + e + w] : l[c + e], give = upper ? l[c + e] : l[c + e + w];
            l[c + e] = keep + __shfl_xor_sync(~0u, give, 2 * w);
          }
        }
        l[c] += __shfl_xor_sync(~0u, l[c], 1);
        if ((lane & 1) == 0) sums[quarter * N + c0 + c + (lane >> 1)] = l[c];
      }
      softmax_sync<L::softmax>();
      const bool whole = item_begin >= u_begin && item_end <= u_end;
      const int part = item_begin >= u_begin;  // part 0 began before the worker's range
      const size_t rows = (size_t)(worker * 2 + part) * N;
      if (st < N) {
        const float sum = (sums[st] + sums[N + st]) + (sums[2 * N + st] + sums[3 * N + st]);
        if (whole) {
          factor[st] = sum == 0.f ? 0.f : (Q8 ? a.v_scale[h] : 1.f) / sum;
          if (place[st] >= 0 && a.lse_out != nullptr)
            a.lse_out[place[st]] = sum == 0.f ? -INFINITY : (reference[st] + log2f(sum)) * kLn2;
        } else {
          scr.stats[rows + st] = make_float2(sum == 0.f ? -INFINITY : reference[st], sum);
        }
      }
      softmax_sync<L::softmax>();
#pragma unroll
      for (int c = 0; c < C; c += 16) {
        float o[16];
        tmem_load(o_cols + lanes + c0 + c, o);
        if (token >= DP) continue;
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 16; ++e) scr.out[(rows + c0 + c + e) * DP + token] = o[e];
          continue;
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(factor + c0 + c + e);
          const int4 p = *reinterpret_cast<const int4*>(place + c0 + c + e);
          const float ff[4] = {f.x, f.y, f.z, f.w};
          const int pp[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (pp[k] >= 0 && token < a.D)
              static_cast<uint16_t*>(a.out)[(size_t)pp[k] * a.D + token] =
                  (uint16_t)Half16<BFQ>::pack(ff[k] == 0.f ? 0.f : o[e + k] * ff[k], 0.f);
        }
      }
      fence_before();
      if (!whole && part == 1 && st == 0) scr.share[worker] = ended;
      item_begin = item_end;
    }
  done:;
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::tmem_cols) : "memory");
  }
}

// ------------------------------------------------------------------------------ host side

// Columns of an item: what the call's largest block needs, up to 128 (64 over an e4m3 cache, whose
// converted tiles take the shared memory).
int columns(int max_q, int G, bool q8) {
  const int rows = max_q * G;
  return rows <= 32 ? 32 : (rows <= 64 || q8 ? 64 : 128);
}

template <bool BFQ, bool Q8, int DP, int N>
cudaError_t launch(const AttentionArgs& a, const Maps& maps, int box, void* scratch, cudaStream_t s) {
  using L = Plan<Q8, DP, N>;
  auto* kernel = attention_wide_kernel<BFQ, Q8, DP, N>;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(kernel, L::total, done);
  if (e != cudaSuccess) return e;
  const int workers = std::min(sm_count(), kMaxSms);
  const Scratch scr = scratch_at(scratch, kMaxSms, N);
  e = launch_chained(kernel, dim3(workers), dim3(L::threads), L::total, s, 1, a, maps, box, scr);
  return e != cudaSuccess ? e : launch_join<BFQ, DP, N>(a, scr, workers, s);
}

template <bool BFQ>
cudaError_t launch(const AttentionArgs& a, const Maps& maps, int box, void* scratch, cudaStream_t s) {
  const bool q8 = a.dtype_kv == DSPARK_E4M3;
  const int n = columns(a.max_q, a.G, q8);
  if (q8)
    return n == 32 ? launch<BFQ, true, 128, 32>(a, maps, box, scratch, s) : launch<BFQ, true, 128, 64>(a, maps, box, scratch, s);
  if (a.D <= 64)
    return n == 32 ? launch<BFQ, false, 64, 32>(a, maps, box, scratch, s)
                   : (n == 64 ? launch<BFQ, false, 64, 64>(a, maps, box, scratch, s)
                              : launch<BFQ, false, 64, 128>(a, maps, box, scratch, s));
  return n == 32 ? launch<BFQ, false, 128, 32>(a, maps, box, scratch, s)
                 : (n == 64 ? launch<BFQ, false, 128, 64>(a, maps, box, scratch, s)
                            : launch<BFQ, false, 128, 128>(a, maps, box, scratch, s));
}

}  // namespace

size_t attention_wide_scratch(int Hq, int Hkv, int D, int max_q) {
  return D > 128 ? 0 : attention::scratch_bytes(kMaxSms, columns(max_q, Hq / Hkv, false), 128);
}

bool launch_attention_wide(const AttentionArgs& a, void* scratch, cudaStream_t s, cudaError_t& e) {
  if (a.D > 128) return false;
  const int box = box_tokens(a.page_size);
  Maps maps;
  if (box == 0 || !encode_pool(&maps.k, a, a.k_pool, box) || !encode_pool(&maps.v, a, a.v_pool, box)) return false;
  e = a.dtype_q == DSPARK_BF16 ? launch<true>(a, maps, box, scratch, s) : launch<false>(a, maps, box, scratch, s);
  return true;
}

}  // namespace dspark
