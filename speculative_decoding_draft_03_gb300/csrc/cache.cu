// cache.cu — page operations of the paged key-value cache: fork, reserve (with copy on
// write), write, truncate, compact.
//
// The free pages are the zeros of ref_count, and which pages a call takes follows from the
// tables alone: the i-th page that the slots need, in slot order, is the i-th lowest free
// one.  Finding it is two prefix sums, one over the slots' needs and one over the free
// pages.  Both fit one thread-block cluster: each CTA keeps its slice of the pool as a bit
// mask in shared memory with a running count per word, the CTAs exchange their totals
// through distributed shared memory, and every needed page is then found by two binary
// searches, independently of the others.  Moving page data is a plain streaming copy.
// What bounds them: latency (a round of 256 slots with 64 forks over 6000 pages and 4 layers is
// eight launches of 39.5 us together, whose bytes take 13 us), and for compaction the device memory
// (537 MB moved in 78 us).
#include <cooperative_groups.h>

#include <algorithm>

#include "serving.cuh"

namespace dspark {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;  // 16-byte pieces in flight per thread

// where-codes of the status word
enum { kBadLen = 40, kBadPage = 41, kBadCount = 42, kBadSlot = 43, kBadQueries = 44 };

// One CTA walks a pool of up to this many pages; larger pools take a cluster of eight, whose
// start and two cluster barriers cost more than a few round trips of loads (a round of 256 slots
// over 6000 pages takes 39.5 us with one CTA, 40.8 with eight).
constexpr int kOneCtaPages = 16384;
int plan_ctas(int num_pages) { return num_pages <= kOneCtaPages ? 1 : 8; }
int slice_words(int num_pages, int ctas) { return (((num_pages + 31) / 32) + ctas - 1) / ctas; }

// This CTA's slice of the pool as a bit mask (bit set: free, or used) with the number of set
// bits before each word.  Returns the slice's count.
__device__ int mask_slice(const int32_t* ref_count, int num_pages, int first_page, int words, bool want_free,
                          uint32_t* mask, int* before, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w0 = warp; w0 < words; w0 += 32 * 4) {
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = first_page + (w0 + 32 * i) * 32 + lane;
      v[i] = w0 + 32 * i < words && p < num_pages ? ref_count[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = __ballot_sync(~0u, want_free ? v[i] == 0 : v[i] > 0);
      if (lane == 0 && w0 + 32 * i < words) mask[w0 + 32 * i] = bits;
    }
  }
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < words; base += blockDim.x) {
    const int w = base + threadIdx.x;
    const int c = w < words ? __popc(mask[w]) : 0;
    int total;
    const int upto = block_scan(c, warp_sums, total);
    if (w < words) before[w] = carry + upto - c;
    carry += total;
  }
  __syncthreads();
  return carry;
}

// Totals of the cluster's CTAs: the sum over lower ranks, and over all.
__device__ void cluster_sums(cg::cluster_group& cluster, int* slot, int mine, int& lower, int& all) {
  if (threadIdx.x == 0) *slot = mine;
  cluster.sync();
  lower = all = 0;
  for (unsigned c = 0; c < cluster.num_blocks(); ++c) {
    const int v = *cluster.map_shared_rank(slot, c);
    if (c < cluster.block_rank()) lower += v;
    all += v;
  }
}

struct Need {
  int len, have, n;
  int pages;      // pages to take, the copy included
  bool copy;      // the partly filled last page is shared
  bool refused;   // the table row is too short, or its entries are invalid
};

__device__ Need slot_need(const CacheTables& t, const int32_t* n_new, int r, bool report) {
  Need k = {};
  const int len = t.seq_len[r];
  const int n = n_new[r];
  if (len < 0 || len > t.max_pages * t.page_size || n < 0) {
    if (report) report_bad_input(t.status, n < 0 ? kBadCount : kBadLen);
    k.refused = true;
    return k;
  }
  k.len = len;
  k.n = n;
  k.have = ceil_div_dev(len, t.page_size);
  const long long want = ((long long)len + n + t.page_size - 1) / t.page_size;
  if (want > t.max_pages) {
    k.refused = true;
    return k;
  }
  if (n > 0 && len % t.page_size != 0) {
    const int last = t.page_table[r * t.table_stride + k.have - 1];
    if (last < 0 || last >= t.num_pages) {
      if (report) report_bad_input(t.status, kBadPage);
      k.refused = true;
      return k;
    }
    k.copy = t.ref_count[last] > 1;
  }
  k.pages = min((int)want - k.have + (k.copy ? 1 : 0), kScanCap);
  return k;
}

// Shared memory: end[R] (pages that slots 0..r take, held at kScanCap, which is more than any
// pool has), flags[R], mask and before [words].
constexpr int kCopies = 1, kTakesPages = 2, kRefused = 4;
__global__ void __launch_bounds__(kPlanThreads) cache_reserve_kernel(CacheTables t, const int32_t* n_new,
                                                                     int32_t* granted, int32_t* copies, int words) {
  extern __shared__ int smem[];
  __shared__ int warp_sums[32], slot;
  int* end = smem;
  uint32_t* mask = reinterpret_cast<uint32_t*>(end + t.R);
  int* before = reinterpret_cast<int*>(mask + words);
  uint8_t* flags = reinterpret_cast<uint8_t*>(before + words);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ctas = cluster.num_blocks();

  griddep_wait();
  griddep_allow_next();
  // (the slots' loads, which depend on one another, overlap with those of the pool)
  Need own = {};
  if (threadIdx.x < t.R) own = slot_need(t, n_new, threadIdx.x, rank == 0);
  const int first_page = rank * words * 32;
  const int free_here = mask_slice(t.ref_count, t.num_pages, first_page, words, true, mask, before, warp_sums);
  int demand = 0;
  for (int base = 0; base < t.R; base += blockDim.x) {
    const int r = base + threadIdx.x;
    Need k = own;
    if (base > 0) {
      k = Need{};
      if (r < t.R) k = slot_need(t, n_new, r, rank == 0);
    }
    int total;
    const int upto = block_scan(k.pages, warp_sums, total);
    if (r < t.R) {
      end[r] = min(demand + upto, kScanCap);
      flags[r] = (k.copy ? kCopies : 0) | (k.pages > 0 ? kTakesPages : 0) | (k.refused ? kRefused : 0);
    }
    demand = min(demand + total, kScanCap);
  }
  int lower, free_total;
  cluster_sums(cluster, &slot, free_here, lower, free_total);  // also: every CTA has read the tables

  const int limit = min(demand, free_total);
  for (int q = threadIdx.x; q < free_here && lower + q < limit; q += blockDim.x) {
    const int r = upper_bound(end, t.R, lower + q);
    if (end[r] > free_total) continue;  // not granted
    const int w = upper_bound(before, words, q) - 1;
    const int page = first_page + w * 32 + __fns(mask[w], 0, q - before[w] + 1);
    const int k = lower + q - (r > 0 ? end[r - 1] : 0);
    int32_t* row = t.page_table + r * t.table_stride;
    const int have = ceil_div_dev(t.seq_len[r], t.page_size);
    const int copies_first = flags[r] & kCopies;
    if (copies_first && k == 0) {
      const int old = row[have - 1];
      row[have - 1] = page;
      atomicSub(t.ref_count + old, 1);
      copies[2 * r] = old;
      copies[2 * r + 1] = page;
    } else {
      row[have + k - copies_first] = page;
    }
    t.ref_count[page] = 1;
  }
  cluster.sync();  // lengths are read above and change below
  for (int r = rank * blockDim.x + threadIdx.x; r < t.R; r += ctas * blockDim.x) {
    const int len = r == threadIdx.x ? own.len : t.seq_len[r], n = r == threadIdx.x ? own.n : n_new[r];
    const bool ok = n > 0 && !(flags[r] & kRefused) && (!(flags[r] & kTakesPages) || end[r] <= free_total);
    granted[r] = ok ? n : 0;
    if (ok) t.seq_len[r] = len + n;
    if (!(ok && (flags[r] & kCopies))) copies[2 * r] = copies[2 * r + 1] = -1;
  }
}

// The pools as a kernel takes them: room for few, or for all (4 KB of parameters, which cost the
// host 1 us a launch more).
template <int N>
struct PoolList {
  int n;
  size_t page_bytes;
  void* base[N];
};
constexpr int kFewPools = 24;
template <int N>
PoolList<N> pool_list(const PagePools& p) {
  PoolList<N> l;
  l.n = p.n;
  l.page_bytes = p.page_bytes;
  for (int i = 0; i < p.n; ++i) l.base[i] = p.base[i];
  return l;
}

// One page of one pool, by a whole CTA.
__device__ __forceinline__ void copy_page(char* pool, size_t page_bytes, int from, int to) {
  const uint4* src = reinterpret_cast<const uint4*>(pool + (size_t)from * page_bytes);
  uint4* dst = reinterpret_cast<uint4*>(pool + (size_t)to * page_bytes);
  const int n = (int)(page_bytes / 16);
  int i = threadIdx.x;
  for (; i + (kCopyUnroll - 1) * kCopyThreads < n; i += kCopyUnroll * kCopyThreads) {
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) v[u] = load_once16(src + i + u * kCopyThreads);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) store16(dst + i + u * kCopyThreads, v[u]);
  }
  for (; i < n; i += kCopyThreads) store16(dst + i, load_once16(src + i));
}

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_on_write_kernel(const int32_t* copies, int R,
                                                                     const __grid_constant__ PoolList<N> pools) {
  griddep_wait();
  const int items = R * pools.n;
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int r = i / pools.n, from = copies[2 * r], to = copies[2 * r + 1];
    if (from >= 0) copy_page(static_cast<char*>(pools.base[i % pools.n]), pools.page_bytes, from, to);
  }
}

__global__ void __launch_bounds__(256) cache_fork_kernel(CacheTables t, int F, const int32_t* src,
                                                         const int32_t* dst) {
  griddep_wait();
  const int f = blockIdx.x, s = src[f], d = dst[f];
  bool bad = s < 0 || s >= t.R || d < 0 || d >= t.R;
  for (int i = threadIdx.x; i < F; i += blockDim.x) bad |= dst[i] == s || (i < f && dst[i] == d);
  int len = 0;
  if (!bad) {
    len = t.seq_len[s];
    bad = t.seq_len[d] != 0 || len < 0 || len > t.max_pages * t.page_size;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report_bad_input(t.status, kBadSlot);
    return;
  }
  // (every thread has read seq_len[d]: the barrier above)
  const int32_t* from = t.page_table + s * t.table_stride;
  int32_t* to = t.page_table + d * t.table_stride;
  const int pages = ceil_div_dev(len, t.page_size);
  for (int j = threadIdx.x; j < t.max_pages; j += blockDim.x) {
    const int p = j < pages ? from[j] : -1;
    to[j] = p;
    if (p >= 0 && p < t.num_pages) atomicAdd(t.ref_count + p, 1);
    else if (j < pages) report_bad_input(t.status, kBadPage);
  }
  if (threadIdx.x == 0) t.seq_len[d] = len;
}

__global__ void __launch_bounds__(256) cache_truncate_kernel(CacheTables t, const int32_t* new_len) {
  griddep_wait();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= t.R) return;
  int len = t.seq_len[r], keep = new_len[r];
  if (len < 0 || len > t.max_pages * t.page_size) {
    if (lane == 0) report_bad_input(t.status, kBadLen);
    return;
  }
  if (keep < 0) {
    if (lane == 0) report_bad_input(t.status, kBadCount);
    keep = 0;
  }
  if (keep >= len) return;
  int32_t* row = t.page_table + r * t.table_stride;
  const int end = ceil_div_dev(len, t.page_size);
  for (int j = ceil_div_dev(keep, t.page_size) + lane; j < end; j += 32) {
    const int p = row[j];
    if (p >= 0 && p < t.num_pages) atomicSub(t.ref_count + p, 1);
    else report_bad_input(t.status, kBadPage);
    row[j] = -1;
  }
  __syncwarp();
  if (lane == 0) t.seq_len[r] = keep;
}

// The free pages below the number of pages in use, and the used pages at or past it.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(CacheTables t, CompactLists l, int32_t* n_moves,
                                                                    int words) {
  extern __shared__ int smem[];
  __shared__ int warp_sums[32], slot, slot_low;
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem);
  int* before = smem + words;
  cg::cluster_group cluster = cg::this_cluster();
  griddep_wait();
  const int first_page = (int)cluster.block_rank() * words * 32;
  const int used_here = mask_slice(t.ref_count, t.num_pages, first_page, words, false, mask, before, warp_sums);
  int lower, used;
  cluster_sums(cluster, &slot, used_here, lower, used);
  // used pages of this slice below index `used`
  const int cut = min(max(used - first_page, 0), words * 32);
  int low_here = used_here;
  if (cut < words * 32) low_here = before[cut >> 5] + __popc(mask[cut >> 5] & ((1u << (cut & 31)) - 1u));
  int unused, low;
  cluster_sums(cluster, &slot_low, low_here, unused, low);
  for (int i = threadIdx.x; i < words * 32; i += blockDim.x) {
    const int p = first_page + i;
    if (p >= t.num_pages) break;
    const uint32_t m = mask[i >> 5], bit = 1u << (i & 31);
    const int rank = lower + before[i >> 5] + __popc(m & (bit - 1u));  // used pages before p
    if (p < used && !(m & bit)) l.hole[p - rank] = p;
    if (p >= used && (m & bit)) {
      l.mover[rank - low] = p;
      l.rank[p] = rank - low;
    }
  }
  if (cluster.block_rank() == 0 && threadIdx.x == 0) {
    l.counts[0] = used;
    l.counts[1] = used - low;
    *n_moves = used - low;
  }
  cluster.sync();  // no CTA leaves while another reads its totals
}

template <int N>
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(CacheTables t, CompactLists l,
                                                                    const __grid_constant__ PoolList<N> pools) {
  griddep_wait();
  const int used = l.counts[0], moves = l.counts[1];
  if (moves == 0) return;
  const long long stride = (long long)gridDim.x * blockDim.x, at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long i = at; i < (long long)t.R * t.max_pages; i += stride) {
    int32_t* e = t.page_table + (i / t.max_pages) * t.table_stride + i % t.max_pages;
    const int p = *e;
    if (p < used) continue;
    if (p >= t.num_pages) {
      report_bad_input(t.status, kBadPage);
      continue;
    }
    const int k = l.rank[p];
    if (k >= 0 && k < moves && l.mover[k] == p) *e = l.hole[k];
    else report_bad_input(t.status, kBadPage);  // an entry that names a free page
  }
  for (long long i = at; i < moves; i += stride) {
    const int from = l.mover[i];
    t.ref_count[l.hole[i]] = t.ref_count[from];
    t.ref_count[from] = 0;
  }
  const long long items = (long long)moves * pools.n;
  for (long long i = blockIdx.x; i < items; i += gridDim.x) {
    const int k = (int)(i / pools.n);
    copy_page(static_cast<char*>(pools.base[i % pools.n]), pools.page_bytes, l.mover[k], l.hole[k]);
  }
}

// ------------------------------------------------------------------------------- write

// The last r in [0, R] with q_start[r] <= t (-1: none), by a warp for one t: 32 places of the
// remaining range are looked at per step, so R slots take log_32(R) loads one after the other.
__device__ __forceinline__ int warp_request_of(const int32_t* q_start, int R, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = R + 1;  // q_start[lo - 1] <= t < q_start[lo + n], where those exist
  while (n > 0) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const uint32_t below = __ballot_sync(~0u, lane * step < n && q_start[at] <= t);
    if (below == 0) break;
    const int last = 31 - __clz(below);  // the places of a sorted array: below's bits are its lowest
    const int end = lo + n;
    lo += last * step + 1;
    n = min(step - 1, end - lo);
  }
  return lo - 1;
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ uint2 quantise8(uint4 raw, float scale) {
  const T* x = reinterpret_cast<const T*>(&raw);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint16_t p[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = __fdiv_rn(to_float(x[4 * h + 2 * i]), scale), b = __fdiv_rn(to_float(x[4 * h + 2 * i + 1]), scale);
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p[i]) : "f"(b), "f"(a));
    }
    w[h] = p[0] | ((uint32_t)p[1] << 16);
  }
  return make_uint2(w[0], w[1]);
}

// One thread per 8 elements of a row; both pools.  What bounds it at serving's sizes is the chain
// of loads (the token's slot, its length, its page), so the rows are on their way meanwhile.
template <typename T, bool QUANT>
__global__ void __launch_bounds__(256) cache_write_kernel(CacheWriteArgs a) {
  griddep_wait();
  griddep_allow_next();
  const int per_row = a.D / 8, per_token = a.Hkv * per_row;
  const long long total = (long long)a.T * per_token, at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const bool mine = at < total;
  const int t = (int)((mine ? at : total - 1) / per_token), rest = (int)(at - (long long)t * per_token);
  const int h = rest / per_row, d = (rest - h * per_row) * 8;
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (mine) {
    const int64_t from = t * a.in_stride_token + h * a.in_stride_head + d;
    k = load_once16(static_cast<const T*>(a.k) + from);
    v = load_once16(static_cast<const T*>(a.v) + from);
  }
  // the slot of the warp's first token; a later token's is there or further on
  int r = warp_request_of(a.q_start, a.R, __shfl_sync(~0u, t, 0));
  if (!mine) return;
  while (r < a.R && a.q_start[r + 1] <= t) ++r;
  if (r < 0 || r >= a.R || (a.granted != nullptr && a.granted[r] == 0)) return;
  const int begin = a.q_start[r], n = a.q_start[r + 1] - begin, i = t - begin;
  const int len = a.seq_len[r];
  const long long pos = (long long)len - n + i;
  if (i < 0 || i >= n || pos < 0 || pos >= (long long)a.max_pages * a.page_size) {
    report_bad_input(a.status, kBadQueries);
    return;
  }
  const int nth = (int)pos / a.page_size;
  const int page = a.page_table[r * a.table_stride + nth];
  if (page < 0 || page >= a.num_pages) {
    report_bad_input(a.status, kBadPage);
    return;
  }
  const int64_t to = page * a.page_stride + h * a.head_stride + ((int)pos - nth * a.page_size) * a.token_stride + d;
  if (QUANT) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.k_pool) + to) = quantise8<T>(k, a.k_scale[h]);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v_pool) + to) = quantise8<T>(v, a.v_scale[h]);
  } else {
    store16(static_cast<T*>(a.k_pool) + to, k);
    store16(static_cast<T*>(a.v_pool) + to, v);
  }
}

// The planning kernels' shared memory grows with the pool and the slots; the limit that fits
// the largest of both is set once.
constexpr size_t kPlanSmem = 4 * (size_t)kMaxSlots + kMaxSlots + 8 * (size_t)(kMaxPages / 32 / 8);
static_assert(kPlanSmem <= 227 * 1024, "the plan must fit into shared memory");

}  // namespace

cudaError_t launch_cache_fork(const CacheTables& t, int F, const int32_t* src, const int32_t* dst, cudaStream_t s) {
  return launch_chained(cache_fork_kernel, dim3(F), dim3(256), 0, s, 1, t, F, src, dst);
}

cudaError_t launch_cache_reserve(const CacheTables& t, const int32_t* n_new, int32_t* granted, int32_t* copies,
                                 const PagePools& pools, cudaStream_t s) {
  const int ctas = plan_ctas(t.num_pages), words = slice_words(t.num_pages, ctas);
  const size_t smem = 4 * (size_t)t.R + 8 * (size_t)words + t.R;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(cache_reserve_kernel, kPlanSmem, done);
  if (e != cudaSuccess) return e;
  e = launch_chained(cache_reserve_kernel, dim3(ctas), dim3(kPlanThreads), smem, s, ctas, t, n_new, granted, copies,
                     words);
  if (e != cudaSuccess || pools.n == 0) return e;
  const int grid = (int)std::min<long long>((long long)t.R * pools.n, 8ll * sm_count());
  const int32_t* pairs = copies;
  return pools.n <= kFewPools ? launch_chained(copy_on_write_kernel<kFewPools>, dim3(grid), dim3(kCopyThreads), 0, s, 1, pairs,
                                               t.R, pool_list<kFewPools>(pools))
                              : launch_chained(copy_on_write_kernel<kMaxPools>, dim3(grid), dim3(kCopyThreads), 0, s, 1, pairs,
                                               t.R, pool_list<kMaxPools>(pools));
}

cudaError_t launch_cache_truncate(const CacheTables& t, const int32_t* new_len, cudaStream_t s) {
  return launch_chained(cache_truncate_kernel, dim3((t.R + 7) / 8), dim3(256), 0, s, 1, t, new_len);
}

cudaError_t launch_cache_compact(const CacheTables& t, const CompactLists& l, int32_t* n_moves, const PagePools& pools,
                                 cudaStream_t s) {
  const int ctas = plan_ctas(t.num_pages), words = slice_words(t.num_pages, ctas);
  const size_t smem = 8 * (size_t)words;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(compact_plan_kernel, kPlanSmem, done);
  if (e != cudaSuccess) return e;
  e = launch_chained(compact_plan_kernel, dim3(ctas), dim3(kPlanThreads), smem, s, ctas, t, l, n_moves, words);
  if (e != cudaSuccess) return e;
  const dim3 grid(8 * sm_count());
  return pools.n <= kFewPools ? launch_chained(compact_move_kernel<kFewPools>, grid, dim3(kCopyThreads), 0, s, 1, t, l,
                                               pool_list<kFewPools>(pools))
                              : launch_chained(compact_move_kernel<kMaxPools>, grid, dim3(kCopyThreads), 0, s, 1, t, l,
                                               pool_list<kMaxPools>(pools));
}

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t s) {
  const long long n = (long long)a.T * a.Hkv * (a.D / 8);
  if (n > (1ll << 31) * 255) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((n + 255) / 256));
  const bool quant = a.dtype_kv == DSPARK_E4M3;
  if (a.dtype_in == DSPARK_BF16)
    return quant ? launch_chained(cache_write_kernel<__nv_bfloat16, true>, grid, dim3(256), 0, s, 1, a)
                 : launch_chained(cache_write_kernel<__nv_bfloat16, false>, grid, dim3(256), 0, s, 1, a);
  return quant ? launch_chained(cache_write_kernel<__half, true>, grid, dim3(256), 0, s, 1, a)
               : launch_chained(cache_write_kernel<__half, false>, grid, dim3(256), 0, s, 1, a);
}

}  // namespace dspark
