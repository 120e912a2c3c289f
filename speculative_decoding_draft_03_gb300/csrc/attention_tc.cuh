// attention_tc.cuh — what the tcgen05 kernels of attention over a paged cache share: barriers with bounded
// waits, copies of page boxes, matrix descriptors, tensor memory, and the pools' tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attention.cuh"

namespace dspark {
namespace attention {

constexpr int kTile = 128;  // tokens
constexpr float kSlack = 8.f;
constexpr float kUnset = -1e30f;  // the reference of a column that has seen nothing: any score passes it
#ifdef DSPARK_TEST_WAIT_LIMIT
// Test builds only: a short limit, and attention of long blocks with a window of kTestStallWindow copies no values,
// so that the first wait for them gives up.
constexpr long long kWaitCycles = DSPARK_TEST_WAIT_LIMIT;
constexpr int kTestStallWindow = 0x5EED;
#else
constexpr long long kWaitCycles = 4000000000ll;  // ~2 s
#endif

// ---------------------------------------------------------------------------- wrappers

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same, suspended for up to NS ns (262 us) while the phase is open.
template <int NS = 1 << 18>
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "n"(NS)
      : "memory");
  return ok != 0;
}
// False (and the flag set) if the phase stays open for kWaitCycles, or another role gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, DeviceStatus* st, int where) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_sleep(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort_flag = 1;
      report_timeout(st, where);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_sleep(bar, parity))
    if (clock64() - t0 > kWaitCycles) return;
}
// A box of a pool, seen as [pages][heads][tokens][D].
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int d, int token, int head,
                                        int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(d), "r"(token), "r"(head), "r"(page)
      : "memory");
}
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
// Shared-memory matrix descriptor, 128-byte swizzle: start, leading and stride byte offsets in
// units of 16 bytes, version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t sw128(uint32_t at, uint32_t leading, uint32_t stride) {
  return (uint64_t)((at >> 4) & 0x3FFFu) | (uint64_t)((leading >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((stride >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor of kind::f16: fp32 sums, A and B both bf16 or both fp16, 128 x N.
template <bool BF>
__device__ constexpr uint32_t idesc(int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((BF ? 1u : 0u) << 7) | ((BF ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) |
         ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 columns of this warp's lanes.
__device__ __forceinline__ void tmem_load(uint32_t at, float* x) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_store(uint32_t at, const float* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "f"(x[8]), "f"(x[9]),
      "f"(x[10]), "f"(x[11]), "f"(x[12]), "f"(x[13]), "f"(x[14]), "f"(x[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

struct Maps {
  CUtensorMap k, v;
};

// ------------------------------------------------------------------------------ host side

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_acquire);
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    known.store(fn, std::memory_order_release);
  }
  return fn;
}

// A pool as [pages][heads][tokens][D] with boxes of `box` tokens by 128 bytes, swizzled.
inline bool encode_pool(CUtensorMap* map, const AttentionArgs& a, const void* pool, int box) {
  auto fn = encoder();
  if (fn == nullptr) return false;
  const cuuint64_t size = a.dtype_kv == DSPARK_E4M3 ? 1 : 2;
  // Entries that lie on one another (a pool expanded over its heads, say) are not something a map
  // can say: the other kernel reads them.  A dimension of one entry has no stride of its own: any
  // that is allowed will do.
  if ((a.token_stride == 0 && a.page_size > 1) || (a.head_stride == 0 && a.Hkv > 1) ||
      (a.page_stride == 0 && a.num_pages > 1))
    return false;
  const cuuint64_t row = (cuuint64_t)a.D * size;
  const cuuint64_t strides[3] = {a.token_stride ? (cuuint64_t)a.token_stride * size : row,
                                 a.head_stride ? (cuuint64_t)a.head_stride * size : row,
                                 a.page_stride ? (cuuint64_t)a.page_stride * size : row};
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
  const cuuint32_t boxes[4] = {(cuuint32_t)(128 / size), (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
  return fn(map, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(pool), dims, strides, boxes, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens per box: the largest power of two that divides the page, 8 (the swizzle's period) to a
// tile's 128; 0 where there is none.
inline int box_tokens(int page_size) {
  int box = kTile;
  while (page_size % box != 0) box /= 2;
  return box >= 8 ? box : 0;
}

}  // namespace attention
}  // namespace dspark
