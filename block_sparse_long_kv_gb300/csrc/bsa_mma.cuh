// Pieces that the tcgen05 kernels over the paged cache share: products with descriptors moved on by constants, copies
// of cache rows, bounded waits that park the warp, and small conversions.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "bsa_cache.h"
#include "bsa_internal.h"
#include "bsa_tree.cuh"
#include "bsa_wait.cuh"
#include "sm103_ptx.cuh"

namespace bsa {
namespace mma {

using wait::Ctl;

// 2^k as f16 in both halves, 0 below the smallest subnormal; k <= 15.
__device__ __forceinline__ uint32_t pow2_f16x2(int k) {
  const uint32_t h = k >= -14 ? static_cast<uint32_t>(k + 15) << 10 : k >= -24 ? 1u << (k + 24) : 0u;
  return h | h << 16;
}
__device__ __forceinline__ uint4 finite_bf16x8(const uint4 &v, uint32_t &lost) {
  return make_uint4(finite_bf16x2(v.x, lost), finite_bf16x2(v.y, lost), finite_bf16x2(v.z, lost), finite_bf16x2(v.w, lost));
}
__device__ __forceinline__ float amax8(const uint4 &v) {  // of eight bf16
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float am = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    am = fmaxf(am, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
  return am;
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// 3-D tiled load global -> shared, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// Offset of 16-byte unit u (of 8) of row r in swizzle chunk c of a tile at offset `tile`.
__device__ __forceinline__ uint32_t swizzled(uint32_t tile, int c, int r, int u) {
  return tile + static_cast<uint32_t>(c) * (128u * 128) + static_cast<uint32_t>(r) * 128 +
         static_cast<uint32_t>((u ^ (r & 7)) * 16);
}

// D[tmem] (+)= A[smem] * B[smem], the descriptors moved on by constants inside the instruction block: the
// issuing thread has few registers, and sums hoisted out of its loop would not stay in them.
template <int AO, int BO, bool FIRST>
__device__ __forceinline__ void mma_ss_at(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "add.s64 x, %1, %4;\n\tadd.s64 y, %2, %5;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "n"(AO), "n"(BO), "n"(FIRST ? 0 : 1)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
template <int AO, int BO>
__device__ __forceinline__ void mma_ts_at(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\t"
      "add.s32 x, %1, %5;\n\tadd.s64 y, %2, %6;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t}" ::"r"(d),
      "r"(at), "l"(bd), "r"(idesc), "r"(accumulate), "n"(AO), "n"(BO)
      : "memory");
}

template <int N>
struct Int {
  static constexpr int value = N;
};

// wait::wait_bar with a time for which the hardware may park the warp: twenty warps that poll would take
// issue slots from the ones that compute.
__device__ __forceinline__ bool try_wait_parked(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(100000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool is_complete(uint32_t bar, uint32_t parity) {  // a look, without waiting
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_parked(uint32_t bar, uint32_t parity, const Ctl &c) {
  if (try_wait_parked(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (;;) {
    if (try_wait_parked(bar, parity)) return true;
    if (*c.abort_flag) return false;
    if (ptx::globaltimer_ns() - t0 > wait::kWaitTimeoutNs) {
      wait::report(c, BSA_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
}

// Rows of a bf16 cache [pages * hkv, page, d]: box of 64 dimensions and 128 rows, or 64 where a page has no
// more; 128-byte swizzle.
inline bool chunk_map(EncodeTiledFn fn, CUtensorMap *map, const void *codes, const CacheDims &c) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.page),
                              static_cast<cuuint64_t>(c.pages) * c.hkv};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.d) * 2, static_cast<cuuint64_t>(c.page) * c.d * 2};
  const cuuint32_t box[3] = {64u, c.page >= 128 ? 128u : 64u, 1u}, estr[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mma
}  // namespace bsa
