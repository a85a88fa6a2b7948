// Paged cache of keys and values: quantising rows as they are written, and
// gathering sequences back as bf16.
//
// Write.  A row (one head of one token) belongs to D / 8 lanes, eight values
// each.  amax is a butterfly over the row's lanes; the row's power of two comes
// from amax's exponent and fraction bits alone, so x * 2^-k is exact and the
// code is one rounding of the exact quotient.  Every input byte is read once
// and every code written once: bound by HBM.
//
// E2M1's quotient x / s is not exact in fp32, and a quotient that lands on a
// tie by its rounding would take the wrong code.  x has 8 significant bits and
// s four, so a quotient is either a tie exactly or at least 2^-10 away from
// one (in the units of the codes).  x * (1 / s) is within 2^-20 of it; rounding
// that to a multiple of 2^-13 restores the ties and moves nothing across one.
//
// Read.  A row's codes are contiguous, so D / 16 lanes take sixteen values each
// and write two 16-byte words of bf16; the values are exact (a code has at most
// six significant bits after its group scale).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "bsa_cache.h"
#include "bsa_internal.h"
#include "sm103_ptx.cuh"

namespace bsa {
namespace {

constexpr int kCacheThreads = 256;

// 2^k for k in [-126, 127].
__device__ __forceinline__ float pow2i(int k) { return __int_as_float((k + 127) << 23); }

// The least k >= -126 with amax <= (1 + frac / 2^23) * 2^(bits + k); amax >= 0 finite.
__device__ __forceinline__ int row_exponent(float amax, int frac, int bits) {
  const int u = __float_as_int(amax);
  const int k = (u >> 23) - 127 - bits + ((u & 0x7FFFFF) > frac ? 1 : 0);
  return max(k, -126);
}

// Two e4m3 codes, a in the low byte, saturated to the largest finite code.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Two e2m1 codes, a in the low four bits, saturated at 6.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  uint16_t r;
  asm("{\n\t.reg .b8 c, z;\n\tmov.b16 {z, c}, 0;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tmov.b16 %0, {c, z};\n\t}"
      : "=h"(r)
      : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_f32(uint32_t two) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2 *>(&r));
}

__device__ __forceinline__ float2 e2m1x2_f32(uint32_t two) {
  const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(two & 0xFFu), __NV_E2M1);
  return __half22float2(*reinterpret_cast<const __half2 *>(&r));
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

// One step of a warp writes R = 32 / (D / 8) rows of one token: heads of k, then of v.
template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheWriteArgs a, int rows_per_warp,
                                                                    int warps_per_token) {
  constexpr int LPR = D / 8;
  constexpr int R = 32 / LPR;
  constexpr int U = 4;  // warp steps whose loads are in flight together: a token's eight rows
  constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;
  constexpr int PER = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / warps_per_token;
  if (t >= a.tokens) return;
  const int slot = __ldg(a.slots + t);  // needed only when the first rows have arrived
  const int sub = lane / LPR, c = lane % LPR;
  const int hkv = a.c.hkv, rows = 2 * hkv;
  const int r0 = static_cast<int>(w - t * warps_per_token) * rows_per_warp;
  const int r1 = min(rows, r0 + rows_per_warp);
  const uint16_t *ks = a.k + t * a.k_stride + 8 * c, *vs = a.v + t * a.v_stride + 8 * c;
  for (int rb = r0; rb < r1; rb += R * U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = rb + u * R + sub;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < r1)
        raw[u] = __ldcs(reinterpret_cast<const uint4 *>(r < hkv ? ks + static_cast<int64_t>(r) * D
                                                                : vs + static_cast<int64_t>(r - hkv) * D));
    }
    if (slot < 0) return;
    const int page = slot >> a.c.page_shift, off = slot & (a.c.page - 1);
    if (page >= a.c.pages) {
      if (a.status != nullptr && lane == 0) atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
      return;
    }
    const size_t tile0 = static_cast<size_t>(page) * hkv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = rb + u * R + sub;
      if (rb + u * R >= r1) break;  // warp-uniform
      const bool live = r < r1, is_k = r < hkv;
      const size_t tile = tile0 + (is_k ? r : r - hkv);
      uint8_t *codes = (is_k ? a.k_codes : a.v_codes) + (tile * a.c.page + off) * RB;
      if constexpr (FMT == BSA_CACHE_BF16) {
        if (live) *reinterpret_cast<uint4 *>(codes + 16 * c) = raw[u];
      } else {
        uint8_t *scales = (is_k ? a.k_scales : a.v_scales) + tile * a.c.page * PER;
        float x[8];
        unpack8(raw[u], x);
        float am = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(x[e]));
        if constexpr (FMT == BSA_CACHE_E4M3) {
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
          const int k = row_exponent(am, 0x600000, 8);  // 448 = 1.75 * 2^8
          const float inv = pow2i(-k);
          const uint2 out = make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16,
                                       e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16);
          if (live) {
            *reinterpret_cast<uint2 *>(codes + 8 * c) = out;
            if (c == 0) scales[off] = static_cast<uint8_t>(k + 127);
          }
        } else {
          // a group of 16 is two lanes
          float ag = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
          am = ag;
#pragma unroll
          for (int o = LPR / 2; o > 1; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
          const int k = row_exponent(am, 0x280000, 11);  // 2688 = 1.3125 * 2^11
          const float inv = pow2i(-k);
          const uint32_t s8 = e4m3x2(ag * inv / 6.f, 0.f);
          const float s = e4m3x2_f32(s8).x;
          const float f = s > 0.f ? 1.f / s : 0.f;
          uint32_t word = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // to a multiple of 2^-13: 1536 + |q| < 2048 keeps steps of 2^-13.  The sign of what
            // becomes zero is x's.
            const float q0 = __fadd_rn(__fadd_rn(x[2 * e] * inv * f, 1536.f), -1536.f);
            const float q1 = __fadd_rn(__fadd_rn(x[2 * e + 1] * inv * f, 1536.f), -1536.f);
            word |= e2m1x2(copysignf(q0, x[2 * e]), copysignf(q1, x[2 * e + 1])) << (8 * e);
          }
          if (!(s > 0.f)) word = 0u;
          if (live) {
            *reinterpret_cast<uint32_t *>(codes + 4 * c) = word;
            if (c == 0) scales[off] = static_cast<uint8_t>(k + 127);
            if ((c & 1) == 0) scales[a.c.page + off * (D / 16) + c / 2] = static_cast<uint8_t>(s8);
          }
        }
      }
    }
  }
}

template <int D, int FMT>
cudaError_t write_t(const CacheWriteArgs &a, cudaStream_t stream) {
  constexpr int R = 32 / (D / 8);
  const int rows = 2 * a.c.hkv;
  // a warp takes all rows of a token once there are enough tokens for every scheduler
  const int per = a.tokens < 152 * 16 ? R : rows;
  const int wpt = (rows + per - 1) / per;
  const int64_t warps = static_cast<int64_t>(a.tokens) * wpt;
  const int64_t grid = (warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  cache_write_kernel<D, FMT><<<static_cast<unsigned>(grid), kCacheThreads, 0, stream>>>(a, per, wpt);
  return cudaGetLastError();
}

// Thread (token, row piece of 16 values): the pieces of a token's heads are consecutive threads.
template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheReadArgs a, int64_t pieces) {
  constexpr int PPR = D / 16;
  constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;
  constexpr int PER = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x;
  if (blockIdx.x == 0)  // every entry is checked, whether or not a row of it is met below
    for (int b = threadIdx.x; b < a.batch; b += kCacheThreads) seq_span(a.cu, b, a.max_seqlen, a.total, a.status);
  if (x >= pieces) return;
  const int per_token = a.c.hkv * PPR;
  const int t = static_cast<int>(x / per_token);
  const int rest = static_cast<int>(x - static_cast<int64_t>(t) * per_token);
  const int g = rest / PPR, c = rest % PPR;
  // the sequence that holds row t: the last b with cu[b] <= t
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  const SeqSpan sp = seq_span(a.cu, lo, a.max_seqlen, a.total, a.status);
  const int i = t - sp.start;
  if (i < 0 || i >= sp.len) return;  // past the last sequence, or in none
  const int j = i >> a.c.page_shift, off = i & (a.c.page - 1);
  const int page = __ldg(a.table + static_cast<size_t>(lo) * a.table_stride + j);
  if (page < 0 || page >= a.c.pages) {
    if (a.status != nullptr) atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
    return;
  }
  const size_t tile = static_cast<size_t>(page) * a.c.hkv + g;
  const size_t row = tile * a.c.page + off;
  const size_t dst = (static_cast<size_t>(t) * a.c.hkv + g) * D + 16 * c;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t *codes = (kv == 0 ? a.k_codes : a.v_codes) + row * RB;
    uint4 *out = reinterpret_cast<uint4 *>((kv == 0 ? a.k : a.v) + dst);
    uint32_t o[8];
    if constexpr (FMT == BSA_CACHE_BF16) {
      const uint4 u0 = __ldcs(reinterpret_cast<const uint4 *>(codes + 32 * c));
      const uint4 u1 = __ldcs(reinterpret_cast<const uint4 *>(codes + 32 * c + 16));
      o[0] = u0.x; o[1] = u0.y; o[2] = u0.z; o[3] = u0.w;
      o[4] = u1.x; o[5] = u1.y; o[6] = u1.z; o[7] = u1.w;
    } else {
      const uint8_t *scales = (kv == 0 ? a.k_scales : a.v_scales) + tile * a.c.page * PER;
      const float s = pow2i(static_cast<int>(scales[off]) - 127);
      if constexpr (FMT == BSA_CACHE_E4M3) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(codes + 16 * c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = e4m3x2_f32(w[e]), q = e4m3x2_f32(w[e] >> 16);
          o[2 * e] = ptx::pack_bf16x2(p.x * s, p.y * s);
          o[2 * e + 1] = ptx::pack_bf16x2(q.x * s, q.y * s);
        }
      } else {
        const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(codes + 8 * c));
        const float gs = e4m3x2_f32(scales[a.c.page + off * (D / 16) + c]).x;
        const uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // the group scale first: its product with a code never leaves fp32's normal range
          const float2 p = e2m1x2_f32(w[e / 4] >> (8 * (e % 4)));
          o[e] = ptx::pack_bf16x2(p.x * gs * s, p.y * gs * s);
        }
      }
    }
    __stcs(out, make_uint4(o[0], o[1], o[2], o[3]));
    __stcs(out + 1, make_uint4(o[4], o[5], o[6], o[7]));
  }
}

template <int D, int FMT>
cudaError_t read_t(const CacheReadArgs &a, cudaStream_t stream) {
  const int64_t pieces = static_cast<int64_t>(a.total) * a.c.hkv * (D / 16);
  const int64_t grid = (pieces + kCacheThreads - 1) / kCacheThreads;
  cache_read_kernel<D, FMT><<<static_cast<unsigned>(grid), kCacheThreads, 0, stream>>>(a, pieces);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t stream) {
  const bool wide = a.c.d == 128;
  switch (a.c.format) {
    case BSA_CACHE_E4M3: return wide ? write_t<128, BSA_CACHE_E4M3>(a, stream) : write_t<64, BSA_CACHE_E4M3>(a, stream);
    case BSA_CACHE_E2M1: return wide ? write_t<128, BSA_CACHE_E2M1>(a, stream) : write_t<64, BSA_CACHE_E2M1>(a, stream);
    default: return wide ? write_t<128, BSA_CACHE_BF16>(a, stream) : write_t<64, BSA_CACHE_BF16>(a, stream);
  }
}

cudaError_t launch_cache_read(const CacheReadArgs &a, cudaStream_t stream) {
  const bool wide = a.c.d == 128;
  switch (a.c.format) {
    case BSA_CACHE_E4M3: return wide ? read_t<128, BSA_CACHE_E4M3>(a, stream) : read_t<64, BSA_CACHE_E4M3>(a, stream);
    case BSA_CACHE_E2M1: return wide ? read_t<128, BSA_CACHE_E2M1>(a, stream) : read_t<64, BSA_CACHE_E2M1>(a, stream);
    default: return wide ? read_t<128, BSA_CACHE_BF16>(a, stream) : read_t<64, BSA_CACHE_BF16>(a, stream);
  }
}

}  // namespace bsa
