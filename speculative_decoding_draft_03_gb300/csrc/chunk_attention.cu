// chunk_attention.cu — attention of long blocks of queries (a chunk of a prompt) over a paged cache, on
// the 5th-generation tensor cores.
//
// A block of n queries does 4 D G n flops per seen key, so from some hundred queries on the products
// bound it, not the cache.  Here the query rows are the 128 rows of the products and the tokens their
// columns:
//   S [128 rows x 128 tokens] = Q . K^T      (both K-major, in shared memory)
//   O [128 rows x D]         += P . V        (P from tensor memory, where it takes S's place; V MN-major)
//   * Rows are a request's queries, token by token with the G heads of a cache head side by side, so that
//     heads share every key and value and a block's diagonal is narrow.  An item is 256 rows: two row
//     tiles A and B that share the copied keys and values, one in its softmax while the other's products
//     run.
//   * A softmax thread owns a row: maximum, sum and reference stay in its registers and no thread waits
//     for another.  The reference moves only when a score passes it by 2^kSlack (any reference is right;
//     the weights stay inside their type's range); only then is O rescaled, by the warp that needs it.
//   * One persistent CTA per SM.  Warps 0 and 2 copy keys and values by page boxes (tensor copies), warp
//     1 issues the products, eight warps (two groups) do the softmax.  Values of tiles at the diagonal, at
//     a window's edge or at the context's end pass warp 3 first, which clears what no row of the item
//     sees, and what only some see if it is not finite (0 x NaN); the rows that see such a token add it
//     on their own.
//   * An e4m3 cache is copied as it is; four more warps turn each tile into fp16 (which holds every e4m3
//     value), and look at the values as warp 3 does otherwise.  bf16 query rows are scaled by powers of
//     two into fp16's range.
//   * An item's last scores free its queries' place: the next item's come while those are weighed, and its
//     first product is issued behind the last one's weights (with the queries loaded after the last weights, a
//     row a lane, 64 blocks of 512 queries took 370 us for 290 so).
//   * The work is dealt out in tiles of 128 tokens that an item sees, evenly over the CTAs; items that
//     several share are joined by a second kernel, in a fixed order.
// What bounds it: the products of a tile of both row tiles (D = 128) keep the tensor cores busy for 2050
// clocks; a tile takes about 3100, the chain of one row tile: 1600 from telling the weights to seeing the next
// scores (two waits, two matrices' products in turn with the other's), 1500 of softmax.  8192 causal queries, 32
// heads over 8 of 128: 409 us, 1343 TFLOP/s (up to 430 from run to run: it tells where the code comes to lie); 2048
// at 32768 tokens: 716 to 737 us, 1490 to 1440 TFLOP/s; over e4m3 the conversion comes on top (8192 causal: 489 us).
// Short items cost something beside their tiles: 64 prompts of 512, 273 us for the 99 that their bytes take.
// Every mbarrier wait is bounded; a wait that gives up reports DSPARK_TIMEOUT and the CTA winds down.
#include <algorithm>

#include "attention_tc.cuh"

namespace dspark {
namespace {

using namespace attention;

constexpr int kRowsOf = 128;           // a row tile
constexpr int kItem = 2 * kRowsOf;     // an item
constexpr int kGroupThreads = 128;     // of a softmax group
constexpr uint32_t kAbs = 0x7FFF7FFFu;  // of two 16-bit floats
constexpr uint32_t kEnds = 1, kTwo = 2, kEdge = 4;  // of a tile: its item ends, has both row tiles; see at_edge

// ---------------------------------------------------------------------------- wrappers

// mbar_wait, out of line where the phase is still open: the roles' loops share the instruction cache, and a
// dozen copies of it cost more than the calls (512 queries at 65536 tokens of an e4m3 cache took 470 us so, 580
// inlined).  Suspended for 2 us at a time, though hardly a wait is as long: the flag is looked at in between, and the
// warp that issues the products, which goes on over its tiles once a wait has given up, is through with a tile in
// some 10 us (with 262 us at a time, in a millisecond; leaving its loop cost 2 % where nothing gives up).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, DeviceStatus* st, int where) {
  const long long t0 = clock64();
  while (!mbar_sleep<1 << 11>(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort_flag = 1;
      report_timeout(st, where);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, DeviceStatus* st, int where) {
  return mbar_test(bar, parity) || wait_on(bar, parity, abort_flag, st, where);
}
// A row of fp16 queries with its signs turned, or of NaN.  (Out of line: hardly ever called.)
__device__ __noinline__ void odd_scale(uint32_t at, int swizzle, int pieces, bool turn) {
  const uint32_t f = turn ? 0x80008000u : 0u, n = turn ? 0u : 0x7FFF7FFFu;
  for (int c = 0; c < pieces; ++c) {
    const uint32_t p = at + (c >> 3) * (kTile * 128) + (((c & 7) ^ swizzle) << 4);
    const uint4 v = lds16(p);
    sts16(p, make_uint4((v.x ^ f) | n, (v.y ^ f) | n, (v.z ^ f) | n, (v.w ^ f) | n));
  }
}
// Products and commits by one elected lane of a warp.  Matrices in shared memory go by their descriptors' lower
// halves (the upper ones: rows of 128 bytes in groups of eight, swizzled).  All products of a matrix in one
// statement: 16 columns of both operands each, one election.
constexpr uint32_t kUpper = (1024u >> 4) | 1u << 14 | 2u << 29;
#define BEGIN_PRODUCTS                                                                                  \
  "{\n\t.reg .pred p, q;\n\t.reg .b32 m, n;\n\t.reg .b64 x, y;\n\telect.sync _|q, 0xffffffff;\n\t" \
  "setp.ne.b32 p, %4, 0;\n\tmov.b32 m, %1;\n\tmov.b32 n, %2;\n\t"
#define PRODUCT_IN_SMEM             \
  "mov.b64 x, {m, %5};\n\tmov.b64 y, {n, %5};\n\t" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
#define PRODUCT_OF_TMEM    \
  "mov.b64 y, {n, %5};\n\t" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [m], y, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
#define GO_ON(by_a, by_b) "add.u32 m, m, " #by_a ";\n\tadd.u32 n, n, " #by_b ";\n\t"
#define FOUR_IN_SMEM PRODUCT_IN_SMEM GO_ON(2, 2) PRODUCT_IN_SMEM GO_ON(2, 2) PRODUCT_IN_SMEM GO_ON(2, 2) PRODUCT_IN_SMEM
#define FOUR_OF_TMEM \
  PRODUCT_OF_TMEM GO_ON(8, 128) PRODUCT_OF_TMEM GO_ON(8, 128) PRODUCT_OF_TMEM GO_ON(8, 128) PRODUCT_OF_TMEM
// A panel is 64 columns, 128 rows of 128 bytes.
template <int DP>
__device__ __forceinline__ void product_of_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t desc) {
  if constexpr (DP == 128)
    asm volatile(BEGIN_PRODUCTS FOUR_IN_SMEM GO_ON(1018, 1018) FOUR_IN_SMEM "}" ::"r"(d), "r"(a), "r"(b), "r"(desc), "r"(0),
                 "n"(kUpper)
                 : "memory");
  else
    asm volatile(BEGIN_PRODUCTS FOUR_IN_SMEM "}" ::"r"(d), "r"(a), "r"(b), "r"(desc), "r"(0), "n"(kUpper) : "memory");
}
// A (the weights) from tensor memory, B 16 of its 128 rows at a time.
__device__ __forceinline__ void product_of_weights(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, uint32_t accumulate) {
  asm volatile(BEGIN_PRODUCTS FOUR_OF_TMEM GO_ON(8, 128) FOUR_OF_TMEM "}" ::"r"(d), "r"(a), "r"(b), "r"(desc), "r"(accumulate),
               "n"(kUpper)
               : "memory");
}
#undef BEGIN_PRODUCTS
#undef PRODUCT_IN_SMEM
#undef PRODUCT_OF_TMEM
#undef GO_ON
#undef FOUR_IN_SMEM
#undef FOUR_OF_TMEM
__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
#define R8(x, i) "=f"(x[i]), "=f"(x[i + 1]), "=f"(x[i + 2]), "=f"(x[i + 3]), "=f"(x[i + 4]), "=f"(x[i + 5]), "=f"(x[i + 6]), "=f"(x[i + 7])
// 64 columns of this warp's lanes, and 128.
__device__ __forceinline__ void tmem_load64(uint32_t at, float* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R8(x, 0), R8(x, 8), R8(x, 16), R8(x, 24), R8(x, 32), R8(x, 40), R8(x, 48), R8(x, 56)
      : "r"(at), "r"(at + 32)
      : "memory");
}
__device__ __forceinline__ void tmem_load128(uint32_t at, float* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R8(x, 0), R8(x, 8), R8(x, 16), R8(x, 24), R8(x, 32), R8(x, 40), R8(x, 48), R8(x, 56), R8(x, 64), R8(x, 72), R8(x, 80),
        R8(x, 88), R8(x, 96), R8(x, 104), R8(x, 112), R8(x, 120)
      : "r"(at), "r"(at + 32), "r"(at + 64), "r"(at + 96)
      : "memory");
}
#undef R8
__device__ __forceinline__ float tmem_load1(uint32_t at) {
  float x;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=f"(x) : "r"(at) : "memory");
  return x;
}
// 16 packed columns (32 weights).
__device__ __forceinline__ void tmem_store_u16(uint32_t at, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]),
      "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
      : "memory");
}
// 32 bytes, at once where they are aligned to as many.
__device__ __forceinline__ void store32(void* p, const uint32_t* x, bool at_once) {
  if (at_once)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  else
    store16(p, make_uint4(x[0], x[1], x[2], x[3])), store16(static_cast<char*>(p) + 16, make_uint4(x[4], x[5], x[6], x[7]));
}
struct Two {
  unsigned long long v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void apart(Two x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// ------------------------------------------------------------------------------- the plan

// The tiles that a block of rows (an item without its head) sees.
struct Block {
  int b;                  // its number
  int first, tiles;       // first: position of the first tile's first token
  int last0, last1;       // last position that the first and the last row see (below 0: nothing)
};
// The nth block of a request in the order of the deal: first, last, second, last but one ... (causal blocks
// see more and more tiles, and an item costs something whatever it sees: every CTA gets short and long ones).
__device__ __forceinline__ int nth_block(const Request& k, int n) { return n & 1 ? k.blocks - 1 - (n >> 1) : n >> 1; }
__device__ __forceinline__ Block block_of(const AttentionArgs& a, const Request& k, int n) {
  const int b = nth_block(k, n);
  Block x;
  x.b = b;
  const int row0 = b * kItem, before = k.len - k.nq;
  const int i0 = row0 / a.G, i1 = min(k.nq - 1, (row0 + kItem - 1) / a.G);
  x.last0 = before + i0;
  x.last1 = before + i1;
  x.first = a.window > 0 ? max(0, x.last0 - a.window + 1) / kTile * kTile : 0;
  x.tiles = x.last1 < x.first ? 1 : (x.last1 - x.first) / kTile + 1;
  return x;
}

// Where a CTA stands: tile t of the nth block of head h of request r.
struct Place {
  Request k;
  Block x;
  int r, h, n, t;
};
__device__ __forceinline__ void next_item(const AttentionArgs& a, Place& c) {
  c.t = 0;
  if (++c.n == c.k.blocks) {
    c.n = 0;
    if (++c.h == a.Hkv) {
      c.h = 0;
      do {
        if (++c.r >= a.R) return;
        c.k = request<kTile, kItem>(a, c.r, false);
      } while (c.k.chunks == 0);
    }
  }
  c.x = block_of(a, c.k, c.n);
}
__device__ __forceinline__ bool two_tiles(const AttentionArgs& a, const Place& c) { return c.k.nq * a.G - c.x.b * kItem > kRowsOf; }
// Does a row of the item not see all of the tile that begins at p0?
__device__ __forceinline__ bool at_edge(const AttentionArgs& a, const Block& x, int p0) {
  return p0 + kTile - 1 > x.last0 || (a.window > 0 && p0 <= x.last1 - a.window);
}

// (a worker's part of an item ends with the worker's last tile)
__device__ __forceinline__ uint32_t unit_of(const AttentionArgs& a, const Place& c, bool last) {
  return (last || c.t + 1 == c.x.tiles ? kEnds : 0u) | (two_tiles(a, c) ? kTwo : 0u) |
         (at_edge(a, c.x, c.x.first + c.t * kTile) ? kEdge : 0u);
}

// ------------------------------------------------------------------------- shared memory

template <bool Q8, int DP>
struct Plan {
  static constexpr int softmax_warp = Q8 ? 8 : 4;  // the first
  static constexpr int threads = 32 * softmax_warp + 2 * kGroupThreads;
  static constexpr int panels = DP / 64;
  static constexpr int tile = panels * kTile * 128;  // keys, or values, of a tile, as the products read them
  static constexpr int raw = kTile * 128;            // ... of an e4m3 cache, as they are copied
  static constexpr int k_stages = Q8 ? 2 : (DP == 64 ? 4 : 2), v_stages = Q8 ? 2 : (DP == 64 ? 4 : 3);
  static constexpr int q = 0;                           // [2][panels][128 rows][128]
  static constexpr int k = q + 2 * tile;                // [k_stages][tile]
  static constexpr int v = k + k_stages * tile;         // [v_stages][tile]
  static constexpr int k_raw = v + v_stages * tile;     // e4m3: [raw]
  static constexpr int v_raw = k_raw + (Q8 ? raw : 0);  // [raw]
  static constexpr int odd = v_raw + (Q8 ? raw : 0);    // [v_stages][4] words: tokens that rows add on their own
  static constexpr int odd_told = odd + 16 * v_stages;  // [2][4]: the same, of a row tile's last tile at an edge
  static constexpr int unit = odd_told + 32;  // [v_stages]: what the products have to know of the stage's tile
  static constexpr int bars = (unit + 4 * v_stages + 7) / 8 * 8;
  // barriers
  static constexpr int k_full = 0, k_empty = k_full + k_stages, v_full = k_empty + k_stages, v_empty = v_full + v_stages,
                       v_ok = v_empty + v_stages, s_full = v_ok + v_stages, p_ready = s_full + 2, told = p_ready + 2,
                       pv_done = told + 2, odd_done = pv_done + 2, o_done = odd_done + 2, q_ready = o_done + 2,
                       drained = q_ready + 2, kr_full = drained + 1, kr_empty = kr_full + 1, vr_full = kr_empty + 1,
                       vr_empty = vr_full + 1, n_bars = vr_empty + 1;
  static constexpr int scan = bars + 8 * n_bars;     // [32] long long
  static constexpr int start_off = scan + 8 * 32;    // long long
  static constexpr int start_r = start_off + 8;      // int, then head, block, tile
  static constexpr int tmem = start_r + 16, abort_flag = tmem + 4;
  static constexpr int places = abort_flag + 4;      // [8] of the softmax warps
  static constexpr int total = places + 8 * sizeof(Place);
  static_assert(total <= 232448, "227 KB");
  static_assert(k + 8 * kMaxSlots <= odd, "the requests' units, before the copies begin");
};

template <int REGS>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// Deals the tiles out evenly: where this worker begins is left in shared memory.
template <typename L>
__device__ Deal deal_tiles(const AttentionArgs& a, long long worker, long long workers, unsigned char* smem) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long* units = reinterpret_cast<long long*>(smem + L::k);  // [R]: of a head
  long long* scan = reinterpret_cast<long long*>(smem + L::scan);
  int* start = reinterpret_cast<int*>(smem + L::start_r);
  long long* start_off = reinterpret_cast<long long*>(smem + L::start_off);
  // a request's tiles: by its thread, or by the warp where it has many blocks
  for (int base = warp * 32; base < a.R; base += L::threads) {
    const int r = base + lane;
    Request k = {};
    if (r < a.R) k = request<kTile, kItem>(a, r, worker == 0);
    const int blocks = k.chunks > 0 ? k.blocks : 0;
    long long n = 0;
    if (blocks <= 8)
      for (int b = 0; b < blocks; ++b) n += block_of(a, k, b).tiles;
    for (uint32_t many = __ballot_sync(~0u, blocks > 8); many != 0; many &= many - 1) {
      const int from = __ffs(many) - 1;
      Request big = {};
      big.len = __shfl_sync(~0u, k.len, from);
      big.nq = __shfl_sync(~0u, k.nq, from);
      big.blocks = __shfl_sync(~0u, blocks, from);
      long long mine = 0;
      for (int b = lane; b < big.blocks; b += 32) mine += block_of(a, big, b).tiles;
#pragma unroll
      for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(~0u, mine, d);
      if (lane == from) n = mine;
    }
    if (r < a.R) units[r] = n;
  }
  __syncthreads();
  const int slice = (a.R + L::threads - 1) / L::threads, r_lo = min(tid * slice, a.R), r_hi = min(r_lo + slice, a.R);
  long long mine = 0;
  for (int r = r_lo; r < r_hi; ++r) mine += a.Hkv * units[r];
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
  for (int w = 0; w < L::threads / 32; ++w) {
    if (w < warp) upto += scan[w];
    deal.total += scan[w];
  }
  deal.per = max((long long)kMinUnits, (deal.total + workers - 1) / workers);
  const long long u = worker * deal.per;
  if (u >= upto - mine && u < upto) {
    long long off = u - (upto - mine);
    int r = r_lo;
    while (off >= a.Hkv * units[r]) off -= a.Hkv * units[r++];
    start[0] = r;
    start[1] = (int)(off / units[r]);
    *start_off = off % units[r];
  }
  __syncthreads();
  if (warp == 0 && u < deal.total) {  // the block, by a warp
    const Request k = request<kTile, kItem>(a, start[0], false);
    long long off = *start_off;
    for (int base = 0;; base += 32) {
      const int b = base + lane, n = b < k.blocks ? block_of(a, k, b).tiles : 0;
      int sum = n;  // (32 times less than 2^24 tiles)
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += o;
      }
      const uint32_t past = __ballot_sync(~0u, sum > off);
      if (past != 0 || base >= k.blocks) {
        if (past != 0 && lane == __ffs(past) - 1) {
          start[2] = b;
          start[3] = (int)(off - (sum - n));
        }
        break;
      }
      off -= __shfl_sync(~0u, sum, 31);
    }
  }
  __syncthreads();
  return deal;
}

// BFQ: queries and outputs bf16, else fp16.  Q8: an e4m3 cache.  DP: elements of a row, padded.
template <bool BFQ, bool Q8, int DP>
__global__ void __launch_bounds__(Plan<Q8, DP>::threads, 1)
    chunk_attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Maps maps, int box, Scratch scr) {
  using L = Plan<Q8, DP>;
  using H = Half16<BFQ && !Q8>;  // type of the products
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return base + L::bars + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::abort_flag);
  volatile uint32_t* odd = reinterpret_cast<volatile uint32_t*>(smem + L::odd);
  volatile uint32_t* odd_told = reinterpret_cast<volatile uint32_t*>(smem + L::odd_told);
  volatile uint32_t* unit = reinterpret_cast<volatile uint32_t*>(smem + L::unit);
  const long long worker = blockIdx.x, workers = gridDim.x;
  const int G = a.G;

  if (tid == 0) {
    constexpr int writers = Q8 ? kGroupThreads / 32 : 1;
    for (int i = 0; i < L::k_stages; ++i) mbar_init(bar(L::k_full + i), writers), mbar_init(bar(L::k_empty + i), 1);
    for (int i = 0; i < L::v_stages; ++i) {
      mbar_init(bar(L::v_full + i), writers), mbar_init(bar(L::v_empty + i), 1), mbar_init(bar(L::v_ok + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::s_full + i), 1), mbar_init(bar(L::o_done + i), 1), mbar_init(bar(L::q_ready + i), kGroupThreads / 32);
      mbar_init(bar(L::p_ready + i), kGroupThreads / 32);
      mbar_init(bar(L::told + i), 1), mbar_init(bar(L::pv_done + i), 1), mbar_init(bar(L::odd_done + i), kGroupThreads / 32);
    }
    mbar_init(bar(L::drained), 1);
    mbar_init(bar(L::kr_full), 1), mbar_init(bar(L::kr_empty), kGroupThreads / 32);
    mbar_init(bar(L::vr_full), 1), mbar_init(bar(L::vr_empty), kGroupThreads / 32);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + L::tmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  griddep_wait();
  griddep_allow_next();
  const Deal d = deal_tiles<L>(a, worker, workers, smem);
  fence_smem();  // (its table lay where copies will land)
  fence_before();
  constexpr uint32_t tmem = 0;  // (an allocation of all 512 columns begins at the first)
  const long long u_begin = worker * d.per, u_end = min(d.total, u_begin + d.per);
  if (tid == 0) {
    scr.share[worker].r = -1;
    if (worker == 0) *scr.per = d.per;
    *reinterpret_cast<volatile long long*>(smem + L::start_off) = u_begin;
  }
  __syncthreads();
  fence_after();
  // (shared memory as the swizzle wants it, which it is without static arrays; tensor memory as said above)
  const bool aligned = (base & 1023u) == 0 && *reinterpret_cast<volatile uint32_t*>(smem + L::tmem) == tmem;
  if (!aligned && tid == 0) report_bad_input(a.status, 632);
  const int tiles = aligned && u_begin < u_end ? (int)(u_end - u_begin) : 0;
#ifdef DSPARK_TEST_WAIT_LIMIT
  const int all_tiles = tiles;
#endif
  auto stand = [&]() {
    Place p = {};
    if (tiles > 0) {
      const volatile int* start = reinterpret_cast<const volatile int*>(smem + L::start_r);
      p.r = start[0], p.h = start[1], p.n = start[2], p.t = start[3];
      p.k = request<kTile, kItem>(a, p.r, false);
      p.x = block_of(a, p.k, p.n);
    }
    return p;
  };
  // The register file, 65536 less what the launch rounds off: 384 threads of 168, or 512 of 128.
  if (warp < L::softmax_warp) {
  fewer_registers<Q8 ? 80 : 88>();
  if (warp == 0 || warp == 2) {
    // ---- copies, of keys (warp 0) and of values (warp 2): a lane per box of a tile, its page looked up
    // one tile ahead
    Place use = stand();
    const bool keys = warp == 0;
#ifdef DSPARK_TEST_WAIT_LIMIT
    const int tiles = !keys && a.window == kTestStallWindow ? 0 : all_tiles;
#endif
    const int boxes = kTile / box;
    const int stages = Q8 ? 1 : (keys ? L::k_stages : L::v_stages);
    const int full = Q8 ? (keys ? L::kr_full : L::vr_full) : (keys ? L::k_full : L::v_full),
              empty = Q8 ? (keys ? L::kr_empty : L::vr_empty) : (keys ? L::k_empty : L::v_empty);
    constexpr int bytes = Q8 ? L::raw : L::tile, panels = Q8 ? 1 : L::panels;
    const uint32_t ring = base + (Q8 ? (keys ? L::k_raw : L::v_raw) : (keys ? L::k : L::v));
    const CUtensorMap* map = keys ? &maps.k : &maps.v;
    int page = -1, slot = 0;
    bool inside = false;
    auto look_up = [&]() {
      const int pos = use.x.first + use.t * kTile + lane * box, nth = pos / a.page_size;
      slot = pos - nth * a.page_size;
      inside = lane < boxes && pos <= use.x.last1 && (a.window == 0 || pos + box - 1 > use.x.last0 - a.window);
      page = inside ? a.page_table[use.r * a.table_stride + nth] : -1;
    };
    if (tiles > 0) look_up();
    int filled = 0, stage = 0, phase = 1;  // (the first round finds every stage empty)
    for (int i = 0; i < tiles; ++i) {
      const bool there = page >= 0 && page < a.num_pages;
      if (inside && !there) report_bad_input(a.status, kBadPage);
      const int from = there ? page : a.num_pages;  // past the pool: zeros
      if (i >= stages && !wait_for(bar(empty + stage), phase, abort_flag, a.status, 621)) break;
      if (lane == 0) mbar_expect(bar(full + stage), bytes);
      __syncwarp();
      if (lane < boxes)
#pragma unroll
        for (int n = 0; n < panels; ++n)
          tma_box(ring + stage * bytes + n * (kTile * 128) + lane * box * 128, map, bar(full + stage), 64 * n, slot, use.h, from);
      filled = i + 1;
      if (++stage == stages) stage = 0, phase ^= 1;
      if (i + 1 < tiles) {
        if (++use.t == use.x.tiles) next_item(a, use);
        look_up();
      }
    }
    // every copy lands before the CTA ends (at once, unless a role gave up)
    for (int i = max(0, filled - stages); i < filled; ++i) mbar_drain(bar(full + i % stages), (i / stages) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // ---- products.  The tensor cores execute them in the order of their issue, so that S of the next tile
    // may follow the product that reads the weights in its place.  What happens between two products is time
    // that the tensor cores stand still, and the other roles' loops leave little of the instruction cache: so
    // what a tile needs (whether its item ends, its second row tile, an edge) is told with its values, a matrix's
    // products are one statement, and the whole warp goes along in branches that votes make uniform, so that
    // descriptors are formed in uniform registers (2048 queries at 32768 tokens took 797 us with an election for each
    // product, 969 by one lane in a branch of its own, 988 with the lane chosen by its number; 8192 causal queries
    // 461 us with this warp finding out about the tiles by itself, 447 so).
    auto all = [](bool x) { return __all_sync(~0u, x) != 0; };
    // (a negative scale turns the queries' signs)
    const uint32_t s_desc = idesc<BFQ && !Q8>(kTile, false, false) | (a.scale < 0.f ? 1u << 13 : 0u);
    constexpr uint32_t o_desc = idesc<BFQ && !Q8>(DP, false, true);
    // (the descriptors' lower halves)
    const uint32_t q_first = (uint32_t)sw128(base + L::q, 16, 1024), k_first = (uint32_t)sw128(base + L::k, 16, 1024),
                   v_first = (uint32_t)sw128(base + L::v, L::panels > 1 ? kTile * 128 : 0, 1024);
    int ks = 0, vs = 0;
    uint32_t k_round = 0, v_round = 0, q_rounds = 0, p1_round = 0, odd_rounds = 0;  // (a bit per row tile)
    // (after a wait that gave up the products go on over what is there, and nobody takes their results)
    auto wait = [&](uint32_t at, uint32_t parity, int where) {
      if (!all(mbar_test(at, parity))) wait_on(at, parity, abort_flag, a.status, where);
    };
    auto scores = [&](int x) {
      product_of_rows<DP>(tmem + x * kTile, q_first + x * (L::tile / 16), k_first + ks * (L::tile / 16), s_desc);
      commit_one(bar(L::s_full + x));
    };
    auto queries = [&](int x) {
      wait(bar(L::q_ready + x), q_rounds >> x & 1, 623);
      q_rounds ^= 1u << x;
      fence_after();
    };
    auto next_keys = [&]() {
      commit_one(bar(L::k_empty + ks));
      if (++ks == L::k_stages) ks = 0, k_round ^= 1;
    };
    const int total = __shfl_sync(~0u, tiles, 0);
    uint32_t now = 0;  // what there is to know of the tile
    if (total > 0) {
      wait(bar(L::k_full), 0, 622);
      wait(bar(Q8 ? L::v_full : L::v_ok), 0, 624);
      now = unit[0];
      queries(0);
      scores(0);
      if (all((now & kTwo) != 0)) queries(1), scores(1);
      next_keys();
      if (total > 1) wait(bar(L::k_full + ks), k_round, 622);
    }
    uint32_t add = 0;  // does the tile's product add? (the first of an item does not)
    for (int i = 0; i < total; ++i) {
      const bool ends = all((now & kEnds) != 0), last = i + 1 == total;
      const int stage = vs;
      auto product = [&](int x, uint32_t round) {
        wait(bar(L::p_ready + x), round, 626);
        fence_after();
        product_of_weights(tmem + 2 * kTile + x * DP, tmem + x * kTile, v_first + stage * (L::tile / 16), o_desc, add);
        if (all((now & kEdge) != 0)) {
          const uint32_t word = lane < 4 ? odd[4 * stage + lane] : 0u;
          if (lane < 4) odd_told[4 * x + lane] = word;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::told + x));
          if (__any_sync(~0u, word != 0)) {  // the rows read the weights and add theirs before either is written again
            commit_one(bar(L::pv_done + x));
            wait(bar(L::odd_done + x), odd_rounds >> x & 1, 637);
            odd_rounds ^= 1u << x;
            fence_after();
          }
        }
        if (ends) commit_one(bar(L::o_done + x));
      };
      product(0, i & 1);
      uint32_t then = 0;
      if (!last) {
        if (ends) queries(0);
        scores(0);
        // the next tile's values, and what there is to know of it
        if (++vs == L::v_stages) vs = 0, v_round ^= 1;
        wait(bar((Q8 ? L::v_full : L::v_ok) + vs), v_round, 624);
        then = unit[vs];
      }
      if (all((now & kTwo) != 0)) product(1, p1_round), p1_round ^= 1;
      commit_one(bar(L::v_empty + stage));
      if (last) break;
      if (all((then & kTwo) != 0)) {
        if (ends) queries(1);
        scores(1);
      }
      next_keys();
      if (i + 2 < total) wait(bar(L::k_full + ks), k_round, 622);
      add = !ends;
      now = then;
    }
    // every product is done before the CTA gives its tensor memory back
    commit_one(bar(L::drained));
    mbar_drain(bar(L::drained), 0);
    __syncwarp();
  } else if (!Q8 && warp == 3) {
    Place use = stand();
    // ---- the values at edges: four tokens a lane
    for (int i = 0; i < tiles; ++i) {
      const int vs = i % L::v_stages;
      if (!wait_for(bar(L::v_full + vs), (i / L::v_stages) & 1, abort_flag, a.status, 627)) break;
      const int p0 = use.x.first + use.t * kTile;
      if (at_edge(a, use.x, p0)) {
        for (int j = 0; j < 4; ++j) {
          const int token = 32 * j + lane, pos = p0 + token;
          const uint32_t row = base + L::v + vs * L::tile + token * 128;
          auto piece = [&](int c) { return row + (c >> 3) * (kTile * 128) + (((c & 7) ^ (token & 7)) << 4); };
          const bool unseen = pos > use.x.last1 || (a.window > 0 && pos <= use.x.last0 - a.window);
          const bool partly = !unseen && (pos > use.x.last0 || (a.window > 0 && pos <= use.x.last1 - a.window));
          uint32_t top = 0;  // the largest exponents, by halves
          if (__any_sync(~0u, partly))
#pragma unroll 4
            for (int c = 0; c < L::panels * 8; ++c) {
              const uint4 v = lds16(piece(c));
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs)));
            }
          const bool strange = partly && ((top & 0xFFFFu) >= H::kExp || (top >> 16) >= H::kExp);
          const uint32_t strangers = __ballot_sync(~0u, strange);
          if (lane == 0) odd[4 * vs + j] = strangers;
          if (unseen || strange)
            for (int c = 0; c < L::panels * 8; ++c) sts16(piece(c), make_uint4(0, 0, 0, 0));
        }
        fence_smem();
        __syncwarp();
      }
      if (lane == 0) unit[vs] = unit_of(a, use, i + 1 == tiles), mbar_arrive(bar(L::v_ok + vs));
      if (i + 1 < tiles && ++use.t == use.x.tiles) next_item(a, use);
    }
  } else if (Q8 && warp >= 4 && warp < 8) {
    // ---- e4m3 to fp16: a thread per token, 16 elements (one piece) into two pieces at a time
    Place use = stand();
    const int token = tid - 128;
    for (int i = 0; i < tiles; ++i) {
      const int ks = i % L::k_stages, vs = i % L::v_stages, p0 = use.x.first + use.t * kTile, pos = p0 + token;
      auto convert = [&](uint32_t from, uint32_t to, bool clear, bool look) {
        bool strange = false;
#pragma unroll 1  // (unrolled, it crowds the instruction cache: 8192 queries took 570 us for 542, 65536 tokens the same)
        for (int c = 0; c < 8; ++c) {
          const uint4 x = lds16(from + token * 128 + ((c ^ (token & 7)) << 4));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[2 * e] = e4m3_to_half2(w[e]), h[2 * e + 1] = e4m3_to_half2(w[e] >> 16);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (look) strange |= (h[e] & H::kExp) == H::kExp || ((h[e] >> 16) & H::kExp) == H::kExp;
            if (clear) h[e] = 0;
          }
          const uint32_t row = to + (c >> 2) * (kTile * 128) + token * 128;
          const int piece = 2 * c & 7;
          sts16(row + ((piece ^ (token & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
          sts16(row + (((piece + 1) ^ (token & 7)) << 4), make_uint4(h[4], h[5], h[6], h[7]));
        }
        return strange;
      };
      if (!wait_for(bar(L::kr_full), i & 1, abort_flag, a.status, 628)) break;
      if (i >= L::k_stages && !wait_for(bar(L::k_empty + ks), (i / L::k_stages - 1) & 1, abort_flag, a.status, 629)) break;
      convert(base + L::k_raw, base + L::k + ks * L::tile, false, false);
      fence_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kr_empty)), mbar_arrive(bar(L::k_full + ks));
      if (!wait_for(bar(L::vr_full), i & 1, abort_flag, a.status, 630)) break;
      if (i >= L::v_stages && !wait_for(bar(L::v_empty + vs), (i / L::v_stages - 1) & 1, abort_flag, a.status, 631)) break;
      const uint32_t to = base + L::v + vs * L::tile;
      if (at_edge(a, use.x, p0)) {
        const bool unseen = pos > use.x.last1 || (a.window > 0 && pos <= use.x.last0 - a.window);
        const bool partly = !unseen && (pos > use.x.last0 || (a.window > 0 && pos <= use.x.last1 - a.window));
        const bool strange = convert(base + L::v_raw, to, unseen, partly);
        const uint32_t strangers = __ballot_sync(~0u, strange);
        if (lane == 0) odd[4 * vs + warp - 4] = strangers;
        if (strange)
          for (int c = 0; c < L::panels * 8; ++c)
            sts16(to + (c >> 3) * (kTile * 128) + token * 128 + (((c & 7) ^ (token & 7)) << 4), make_uint4(0, 0, 0, 0));
      } else {
        convert(base + L::v_raw, to, false, false);
      }
      fence_smem();
      if (warp == 4 && lane == 0) unit[vs] = unit_of(a, use, i + 1 == tiles);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::vr_empty)), mbar_arrive(bar(L::v_full + vs));
      if (i + 1 < tiles && ++use.t == use.x.tiles) next_item(a, use);
    }
  }
  } else {
    more_registers<Q8 ? 176 : 208>();
    // ---- softmax: group x has row tile x; a thread, the row of its TMEM lane
    // (where it stands lies in shared memory, a copy a warp: it is looked at between items only, and registers are few)
    Place& use = *reinterpret_cast<Place*>(smem + L::places + (warp - L::softmax_warp) * sizeof(Place));
    const Place begins = stand();
    if (lane == 0) use = begins;
    __syncwarp();
    const int x = (warp - L::softmax_warp) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + x * kTile, o_at = tmem + lanes + 2 * kTile + x * DP;
    int item_begin = -use.t;  // where the item begins among the worker's tiles
    // The item's row of this thread: its query's number (of the request) and head, or none; scores in base 2 are
    // c2 times what the products give (never 0, so that what is masked stays -inf).  The warp copies its 32 query
    // rows to where the products read them, DP / 8 lanes a row, and says so when they have come.
    bool there;
    int query, head;
    float c2;
    const float per_g = 1.f / (float)G;
    auto fetch = [&]() {
      constexpr int kPieces = DP / 8, kRows = 32 / kPieces;  // of a row; rows at a time
      const int warp_row = use.x.b * kItem + x * kRowsOf + (row & ~31), q0 = warp_row / G, g0 = warp_row - q0 * G;
      auto query_of = [&](int r) { return (int)(((float)(g0 + r) + 0.5f) * per_g); };  // from q0 on (exact: below 2^8)
      const int c = lane % kPieces, left = use.k.nq - q0;
      const uint16_t* from = static_cast<const uint16_t*>(a.q) + (int64_t)(use.k.q0 + q0) * a.q_stride_token +
                             (int64_t)use.h * G * a.q_stride_head + c * 8;
#pragma unroll 4
      for (int r = lane / kPieces; r < 32; r += kRows) {
        const int q = query_of(r), at = (row & ~31) + r;
        const bool real = q < left && c * 8 < a.D;
        copy16(base + L::q + x * L::tile + at * 128 + (c >> 3) * (kTile * 128) + (((c & 7) ^ (at & 7)) << 4),
               real ? from + q * a.q_stride_token + (g0 + r - q * G) * a.q_stride_head : a.q, real);
      }
      copy_commit();
      query = query_of(lane);
      there = query < left;
      head = use.h * G + g0 + lane - query * G;
      query += q0;
    };
    auto fetched = [&]() {
      copy_wait<0>();
      if constexpr (Q8) {
        float by = fabsf(a.scale) * kLog2e * a.k_scale[use.h];  // (the sign of the first is in the products)
        __syncwarp();
        const uint32_t mine = base + L::q + x * L::tile + row * 128;
        auto piece = [&](int c) { return mine + (c >> 3) * (kTile * 128) + (((c & 7) ^ (row & 7)) << 4); };
        if constexpr (BFQ) {
          // fp16 operands: the row is scaled by a power of two to a maximum in [1, 2) (what falls below 2^-24 of
          // it is lost, far under the sums' rounding)
          uint32_t top = 0;  // (floats without their signs are in the order of their bits)
#pragma unroll 4
          for (int c = 0; c < DP / 8; ++c) {
            const uint4 v = lds16(piece(c));
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs)));
          }
          const int most = (int)(max(top & 0xFFFFu, top >> 16) >> 7);  // its exponent's bits
          int e2 = most == 0xFF ? 0 : min(max(most, 1), 253) - 127;
          if (top == 0) e2 = 0;
          by *= __int_as_float((127 + e2) << 23);
          const float down = __int_as_float((127 - e2) << 23);
#pragma unroll 2
          for (int c = 0; c < DP / 8; ++c) {
            const uint4 v = lds16(piece(c));
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = Half16<false>::pack(Half16<true>::lo(w[e]) * down, Half16<true>::hi(w[e]) * down);
            sts16(piece(c), make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
        // A k_scale below 0 turns the queries' signs, one that is no number makes them none, as masks are put into the
        // scores and must stay -inf times c2.  (With this loop in line 512 queries at 65536 tokens took 484 us, so 420; 415
        // without it.)
        if (!(by >= 0.f)) odd_scale(mine, row & 7, DP / 8, by < 0.f);
        c2 = fmaxf(fabsf(by), 0x1p-149f);
      } else {
        c2 = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-149f);
      }
      fence_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::q_ready + x));
    };
    int i = 0, done = 0, items = 0, edges = 0, odds = 0;  // tiles; this group's tiles, items, tiles at edges, with odd values
    bool ok = true, mine = x == 0 || two_tiles(a, use);
    if (tiles > 0 && mine) fetch(), fetched();
    while (i < tiles) {
      const int n = min(use.x.tiles - use.t, tiles - i);
      // what is asked about the item when the next one has been opened
      const int item_end = item_begin + use.x.tiles;
      const bool whole = item_begin >= 0 && item_end <= tiles;
      const int part = item_begin >= 0;  // part 0 began before the worker's range
      const bool was_mine = mine, was_there = there, more = i + n < tiles;
      const int r = use.r, h = use.h, last = there ? use.k.len - use.k.nq + query : -1;
      const int64_t place = (int64_t)(use.k.q0 + query) * a.Hq + head;
      const long long first_unit = *reinterpret_cast<volatile long long*>(smem + L::start_off);
      if (!whole && part == 1 && x == 0 && row == 0)
        scr.share[worker] = Share{r, h * use.k.blocks + use.x.b, use.k.q0, use.k.nq, first_unit + item_begin, first_unit + item_end};
      item_begin = item_end;
      // the row tile's first and last row
      const int tile_row = use.x.b * kItem + x * kRowsOf;
      const int last0 = use.k.len - use.k.nq + tile_row / G,
                last1 = use.k.len - use.k.nq + min(use.k.nq - 1, (tile_row + kRowsOf - 1) / G);
      const int begin = use.x.first + use.t * kTile;
      const int gate_from = use.x.last0 - kTile + 2, gate_upto = a.window > 0 ? use.x.last1 - a.window : -1;
      float ref = kUnset;
      Two sum0 = two(0.f, 0.f), sum1 = two(0.f, 0.f);
      for (int t = mine ? 0 : n - 1; t < n; ++t) {
        if (was_mine) {
          ok = mbar_wait(bar(L::s_full + x), done++ & 1, abort_flag, a.status, 633);
          if (__any_sync(~0u, !ok)) {
            ok = false;
            break;
          }
          fence_after();  // (and the tile before is in O: its product was issued before this S)
        }
        const int p0 = begin + t * kTile;
        // (a request's or a window's end may be an edge of the item and none of this row tile)
        const bool gated = p0 >= gate_from || p0 <= gate_upto, leaves = t + 1 == n && more;
        if (__builtin_expect(leaves, 0)) {  // the next item's queries are on their way from here on
          Place next = use;
          next_item(a, next);
          __syncwarp();
          if (lane == 0) use = next;
          __syncwarp();
          mine = x == 0 || two_tiles(a, use);
          if (mine) fetch();
        }
        if (was_mine) {
          const bool edge = __builtin_expect(gated, 0) && (p0 + kTile - 1 > last0 || (a.window > 0 && p0 <= last1 - a.window));
          // a new reference where a score passes the old one by too much
          auto refer = [&](float most) {
            if (!__any_sync(~0u, most > ref + (kSlack + H::kLift))) return;
            const float now = fmaxf(ref, most - H::kLift), f = ex2(ref - now);
            ref = now;
            const Two ff = two(f, f), zero = two(0.f, 0.f);
            sum0 = fma2(sum0, ff, zero), sum1 = fma2(sum1, ff, zero);
            if (t == 0) return;
#pragma unroll 1
            for (int c = 0; c < DP; c += 16) {
              float o[16];
              tmem_load(o_at + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tmem_store(o_at + c, o);
            }
          };
          // what the row does not see goes out of its scores, in a pass of its own: the loops below stay short (with
          // the selects in them, 8192 causal queries took 474 us for 460, and with D = 64 452 for 419)
          if (edge) {
            const int hi = last - p0, lo = a.window > 0 ? hi - a.window + 1 : 0;
#pragma unroll 1
            for (int c = 0; c < kTile; c += 16) {
              float s[16];
              tmem_load(s_at + c, s);
              // a bit for each of the columns that it does see
              const uint32_t upto = hi - c >= 31 ? ~0u : (hi < c ? 0u : (2u << (hi - c)) - 1),
                             before = lo <= c ? 0u : (lo - c >= 32 ? ~0u : (1u << (lo - c)) - 1), bits = upto & ~before;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!((bits >> e) & 1u)) s[e] = -INFINITY;
              tmem_store(s_at + c, s);
            }
            tmem_store_wait();
          }
          float m[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) m[k] = -INFINITY;
          auto largest = [&](const float* s) {
#pragma unroll
            for (int e = 0; e < 32; e += 16)
#pragma unroll
              for (int k = 0; k < 8; ++k) m[k] = max3(m[k], s[e + k], s[e + k + 8]);
          };
          // A row's scores, all at once in registers where there are enough; an e4m3 cache's converters leave too few
          // of them, and half a row's scores are read again (2048 queries at 32768 tokens: 725 us at once, 786 by 32
          // columns, all read twice; 512 at 65536 over e4m3: 462 with 128 held, 415 with 64, 435 with 32).  Short items
          // lose by it: 64 prompts of 512 take 250 us by 32 columns and 273 at once, one of 8192 445 and 410.
          constexpr int kHeld = Q8 ? 64 : kTile;
          float s[kHeld];
          if constexpr (!Q8) {
            tmem_load128(s_at, s);
#pragma unroll
            for (int c = 0; c < kTile; c += 32) largest(s + c);
          } else {
#pragma unroll 1
            for (int c = 64; c >= 0; c -= 64) tmem_load64(s_at + c, s), largest(s), largest(s + 32);
          }
          refer(max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], m[5]), fmaxf(m[6], m[7])) * c2);
          const Two cc = two(c2, c2), rr2 = two(-ref, -ref);
          // The weights are rounded to the product's 16 bits, as the instruction wants both operands of one type; the
          // normaliser adds them unrounded.  Each is off by half a step, 2^-8 (bf16) or 2^-11 (fp16, and over e4m3) of
          // itself, independently: the outputs' relative error goes from the 1.6e-3 of their own rounding to bf16 to 2.1e-3
          // (fp16 2.1e-4 to 2.9e-4).
          auto weigh = [&](const float* s, int c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float p0_, p1_, p2_, p3_;
              apart(fma2(two(s[e], s[e + 1]), cc, rr2), p0_, p1_);
              apart(fma2(two(s[e + 2], s[e + 3]), cc, rr2), p2_, p3_);
              p0_ = ex2(p0_), p1_ = ex2(p1_), p2_ = ex2(p2_), p3_ = ex2(p3_);
              sum0 = add2(sum0, two(p0_, p1_)), sum1 = add2(sum1, two(p2_, p3_));
              w[e / 2] = H::pack(p0_, p1_), w[e / 2 + 1] = H::pack(p2_, p3_);
            }
            tmem_store_u16(s_at + c / 2, w);
          };
          if constexpr (!Q8) {
#pragma unroll
            for (int c = 0; c < kTile; c += 32) weigh(s + c, c);
          } else {
#pragma unroll 1
            for (int c = 0; c < kTile; c += 64) {
              if (c > 0) tmem_load64(s_at + c, s);
              weigh(s, c), weigh(s + 32, c + 32);
            }
          }
          tmem_store_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::p_ready + x));
        }
        if (__builtin_expect(leaves && mine, 0)) fetched();
        // values that are not finite, where only some rows see them, have been taken out of the product: the
        // rows that do add them on their own, with the weights as they were told
        if (__builtin_expect(was_mine && gated, 0)) {
          ok = mbar_wait(bar(L::told + x), edges & 1, abort_flag, a.status, 634);
          ++edges;
          // (uniform over the group: these words are not written before it has told its next weights)
          const bool some = ok && (odd_told[4 * x] | odd_told[4 * x + 1] | odd_told[4 * x + 2] | odd_told[4 * x + 3]) != 0;
          if (some) ok = mbar_wait(bar(L::pv_done + x), odds & 1, abort_flag, a.status, 638);
          if (__any_sync(~0u, !ok)) {
            ok = false;
            break;
          }
          if (some) {
            ++odds;
            fence_after();
#pragma unroll 1
            for (int k = 0; k < kTile; ++k) {
              if (((odd_told[4 * x + (k >> 5)] >> (k & 31)) & 1u) == 0) continue;
              const int pos = p0 + k, nth = pos / a.page_size, page = a.page_table[r * a.table_stride + nth];
              const uint32_t two_weights = __float_as_uint(tmem_load1(s_at + k / 2));
              const float p = k & 1 ? H::hi(two_weights) : H::lo(two_weights);
              const bool sees = pos <= last && (a.window == 0 || pos > last - a.window) && page >= 0 && page < a.num_pages;
              const int64_t at = page * a.page_stride + h * a.head_stride + (pos - nth * a.page_size) * a.token_stride;
#pragma unroll 1
              for (int c = 0; c < DP; c += 16) {
                float o[16];
                tmem_load(o_at + c, o);
                if (sees && c < a.D) {
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    float v;
                    if (Q8) v = Half16<false>::lo(e4m3_to_half2(static_cast<const uint8_t*>(a.v_pool)[at + c + e]));
                    else v = H::lo(static_cast<const uint16_t*>(a.v_pool)[at + c + e]);
                    o[e] = fmaf(p, v, o[e]);
                  }
                }
                tmem_store(o_at + c, o);
                tmem_store_wait();
              }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::odd_done + x));
          }
        }
      }
      i += n;
      if (!ok) break;
      if (!was_mine) continue;
      ok = mbar_wait(bar(L::o_done + x), items++ & 1, abort_flag, a.status, 635);
      if (__any_sync(~0u, !ok)) break;
      fence_after();
      float l0, l1, l2, l3;
      apart(sum0, l0, l1), apart(sum1, l2, l3);
      const float sum = (l0 + l1) + (l2 + l3), f = sum == 0.f ? 0.f : (Q8 ? a.v_scale[h] : 1.f) / sum;
      const size_t out_row = (size_t)(worker * 2 + part) * kItem + x * kRowsOf + row;
      if (was_there && whole && a.lse_out != nullptr) a.lse_out[place] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
      if (was_there && !whole) scr.stats[out_row] = make_float2(sum == 0.f ? -INFINITY : ref, sum);
      const bool in_32 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
#pragma unroll 1
      for (int c = 0; c < DP; c += 16) {
        float o[16];
        tmem_load(o_at + c, o);
        if (!was_there) continue;
        if (!whole) {
          store32(scr.out + out_row * DP + c, reinterpret_cast<const uint32_t*>(o), true);
          store32(scr.out + out_row * DP + c + 8, reinterpret_cast<const uint32_t*>(o + 8), true);
        } else if (c < a.D) {
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = sum == 0.f ? 0u : Half16<BFQ>::pack(o[2 * j] * f, o[2 * j + 1] * f);
          store32(static_cast<uint16_t*>(a.out) + place * a.D + c, w, in_32);
        }
      }
      fence_before();
    }
    copy_wait<0>();  // (a role that gave up may have left some on their way)
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*reinterpret_cast<volatile uint32_t*>(smem + L::tmem)) : "memory");
  }
}

// ------------------------------------------------------------------------------ host side

template <bool BFQ, bool Q8, int DP>
cudaError_t launch(const AttentionArgs& a, const Maps& maps, int box, void* scratch, cudaStream_t s) {
  using L = Plan<Q8, DP>;
  auto* kernel = chunk_attention_kernel<BFQ, Q8, DP>;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(kernel, L::total, done);
  if (e != cudaSuccess) return e;
  const int workers = std::min(sm_count(), kMaxSms);
  const Scratch scr = scratch_at(scratch, kMaxSms, kItem);
  e = launch_chained(kernel, dim3(workers), dim3(L::threads), L::total, s, 1, a, maps, box, scr);
  return e != cudaSuccess ? e : launch_join<BFQ, DP, kItem>(a, scr, workers, s);
}

}  // namespace

size_t chunk_attention_scratch(int Hq, int Hkv, int D) {
  return std::max(attention_rows_scratch(Hq, Hkv, D), D > 128 ? 0 : scratch_bytes(kMaxSms, kItem, 128));
}

cudaError_t launch_chunk_attention(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  const int box = box_tokens(a.page_size);
  Maps maps;
  if (a.D > 128 || box == 0 || !encode_pool(&maps.k, a, a.k_pool, box) || !encode_pool(&maps.v, a, a.v_pool, box))
    return launch_attention_rows(a, scratch, s);
  const bool bf = a.dtype_q == DSPARK_BF16;
  if (a.dtype_kv == DSPARK_E4M3)
    return bf ? launch<true, true, 128>(a, maps, box, scratch, s) : launch<false, true, 128>(a, maps, box, scratch, s);
  if (a.D <= 64)
    return bf ? launch<true, false, 64>(a, maps, box, scratch, s) : launch<false, false, 64>(a, maps, box, scratch, s);
  return bf ? launch<true, false, 128>(a, maps, box, scratch, s) : launch<false, false, 128>(a, maps, box, scratch, s);
}

}  // namespace dspark
