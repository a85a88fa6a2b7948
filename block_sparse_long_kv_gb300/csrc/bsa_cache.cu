// Paged cache of keys and values: quantising rows as they are written, and
// gathering sequences back as bf16.
//
// Write.  A row (one head of one token) belongs to D / 16 lanes, sixteen values
// each: one group of E2M1.  amax is a butterfly over the row's lanes; the row's
// power of two comes from amax's exponent and fraction bits alone, so x * 2^-k is
// exact and the code is one rounding of the exact quotient.
//
// E2M1's quotient x / s is not exact in fp32, and a quotient that lands on a
// tie by its rounding would take the wrong code.  x has 8 significant bits and
// s four, so a quotient is either a tie exactly or at least 2^-10 away from
// one (in the units of the codes).  x * (1 / s) is within 2^-20 of it; rounding
// that to a multiple of 2^-13 restores the ties and moves nothing across one.
//
// Inf and NaN have no code in E4M3 but NaN's, and none in E2M1: there the group scale is NaN instead.  They do
// not count in the row's amax, so the other elements (in E2M1 the other groups) keep their bits.
//
// Read.  D / 16 lanes take sixteen values of a row each and write two 16-byte words
// of bf16; the values are exact (a code has at most six significant bits after its
// group scale).
//
// Both are bound by HBM, and what decides how near they come is the order of the
// accesses: a CTA is one head of a stretch of tokens, so that it meets neighbouring
// rows of codes and whole sectors of scale bytes, and the CTAs in flight move through
// both sides together.  131072 tokens x 4 heads of 128: into e4m3 61 us (6.7 TB/s; 84
// with a warp per token over all heads, whose scale bytes are scattered), back 63 us
// (6.4 TB/s; 91 with a long stretch for each warp, which scatters the writes).
// 19 sequences of 4500 to 9001 tokens back from e2m1 62 us (5.5 TB/s; 69 by token).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "bsa_cache.h"
#include "bsa_internal.h"
#include "sm103_ptx.cuh"

namespace bsa {
namespace {

// two warps: eight tokens of 128 dimensions (64, 128 and 256 threads differ by 3 % at most)
constexpr int kCacheThreads = 64;

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

// |a| and |b| by halves, the larger of each (a NaN gives way to a number).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.bf16x2 %0, x, y;\n\t}"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}
// As above, but a NaN stays one.
__device__ __forceinline__ uint32_t max_abs_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}
// Infinities become NaN (0 * x + x), all else stays.
__device__ __forceinline__ uint32_t inf_to_nan_bf16x2(uint32_t a) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %1;" : "=r"(r) : "r"(a), "r"(0u));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float lo_f32(uint32_t two) { return __uint_as_float(two << 16); }
__device__ __forceinline__ float hi_f32(uint32_t two) { return __uint_as_float(two & 0xFFFF0000u); }

// The larger of two halves that are not negative, as fp32; 0 where both are NaN.
__device__ __forceinline__ float larger_half(uint32_t two) { return fmaxf(lo_f32(two), fmaxf(hi_f32(two), 0.f)); }

// A warp takes the K and V rows of one head of R = 32 / (D / 16) tokens: their slots are mostly neighbours, so
// that their scale bytes meet in one sector.  Scaling by the row's power of two is done on bf16 pairs: what that
// rounds is below 2^-126 and has code 0 all the same.
template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int LPR = D / 16;
  constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;
  constexpr int PER = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
  const uint32_t block = blockIdx.x / a.c.hkv, g = blockIdx.x - block * a.c.hkv;
  const uint32_t t = block * (kCacheThreads / LPR) + threadIdx.x / LPR;  // (the last stretch may pass 2^31 tokens)
  const int c = threadIdx.x % LPR;
  uint4 raw[2][2];
  raw[0][0] = raw[0][1] = raw[1][0] = raw[1][1] = make_uint4(0u, 0u, 0u, 0u);
  int slot = -1;
  if (t < static_cast<uint32_t>(a.tokens)) {
    slot = __ldg(a.slots + t);  // needed only when the rows have arrived
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4 *from = reinterpret_cast<const uint4 *>((kv == 0 ? a.k + t * a.k_stride : a.v + t * a.v_stride) + g * D) + 2 * c;
      raw[kv][0] = __ldcs(from);
      raw[kv][1] = __ldcs(from + 1);
    }
  }
  const int page = slot >> a.c.page_shift, off = slot & (a.c.page - 1);
  const bool live = slot >= 0 && page < a.c.pages;
  if (slot >= 0 && !live && c == 0 && a.status != nullptr)
    atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
  if (!__any_sync(0xffffffffu, live)) return;
  const size_t tile = static_cast<size_t>(live ? page : 0) * a.c.hkv + g;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t *codes = (kv == 0 ? a.k_codes : a.v_codes) + (tile * a.c.page + off) * RB;
    if constexpr (FMT == BSA_CACHE_BF16) {
      if (live) {
        *reinterpret_cast<uint4 *>(codes + 32 * c) = raw[kv][0];
        *reinterpret_cast<uint4 *>(codes + 32 * c + 16) = raw[kv][1];
      }
    } else {
      uint8_t *scales = (kv == 0 ? a.k_scales : a.v_scales) + tile * a.c.page * PER;
      uint32_t x[8] = {raw[kv][0].x, raw[kv][0].y, raw[kv][0].z, raw[kv][0].w,
                       raw[kv][1].x, raw[kv][1].y, raw[kv][1].z, raw[kv][1].w};
      uint32_t mine;
      bool lost = false;  // the group holds Inf or NaN
      if constexpr (FMT == BSA_CACHE_E4M3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = inf_to_nan_bf16x2(x[e]);
        const uint32_t m0 = max_abs_bf16x2(max_abs_bf16x2(x[0], x[1]), max_abs_bf16x2(x[2], x[3]));
        const uint32_t m1 = max_abs_bf16x2(max_abs_bf16x2(x[4], x[5]), max_abs_bf16x2(x[6], x[7]));
        mine = max_abs_bf16x2(m0, m1);
      } else {
        const uint32_t m0 = max_abs_nan_bf16x2(max_abs_nan_bf16x2(x[0], x[1]), max_abs_nan_bf16x2(x[2], x[3]));
        const uint32_t m1 = max_abs_nan_bf16x2(max_abs_nan_bf16x2(x[4], x[5]), max_abs_nan_bf16x2(x[6], x[7]));
        mine = max_abs_nan_bf16x2(m0, m1);
        lost = (mine & 0x7F80u) == 0x7F80u || (mine & 0x7F800000u) == 0x7F800000u;
        if (lost) mine = 0u;
      }
      uint32_t all = mine;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) all = max_abs_bf16x2(all, __shfl_xor_sync(0xffffffffu, all, o));
      const float am = larger_half(all);
      if constexpr (FMT == BSA_CACHE_E4M3) {
        const int k = row_exponent(am, 0x600000, 8);  // 448 = 1.75 * 2^8
        const uint32_t inv = static_cast<uint32_t>(127 - k) * 0x00800080u;  // 2^-k twice
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t p = mul_bf16x2(x[2 * e], inv), q = mul_bf16x2(x[2 * e + 1], inv);
          out[e] = __byte_perm(e4m3x2(lo_f32(p), hi_f32(p)), e4m3x2(lo_f32(q), hi_f32(q)), 0x5410);
        }
        if (live) {
          *reinterpret_cast<uint4 *>(codes + 16 * c) = make_uint4(out[0], out[1], out[2], out[3]);
          if (c == 0) scales[off] = static_cast<uint8_t>(k + 127);
        }
      } else {
        // the lane's sixteen values are one group
        const int k = row_exponent(am, 0x280000, 11);  // 2688 = 1.3125 * 2^11
        const uint32_t inv = static_cast<uint32_t>(127 - k) * 0x00800080u;
        const uint32_t s8 = lost ? 0x7Fu : e4m3x2(larger_half(mine) * pow2i(-k) / 6.f, 0.f);
        const float s = e4m3x2_f32(s8).x;
        const float f = s > 0.f ? __frcp_rn(s) : 0.f;
        const uint64_t f2 = ptx::f32x2(f, f), up = ptx::f32x2(1536.f, 1536.f), down = ptx::f32x2(-1536.f, -1536.f);
        uint32_t word[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // to a multiple of 2^-13: 1536 + |q| < 2048 keeps steps of 2^-13.  The sign of what
            // becomes zero is x's.
            const uint32_t p = mul_bf16x2(x[4 * h + e], inv);
            const float p0 = lo_f32(p), p1 = hi_f32(p);
            float q0, q1;
            ptx::f32x2_split(ptx::add_f32x2(ptx::fma_f32x2(ptx::f32x2(p0, p1), f2, up), down), q0, q1);
            b[e] = e2m1x2(copysignf(q0, p0), copysignf(q1, p1));
          }
          word[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
          if (!(s > 0.f)) word[h] = 0u;
        }
        if (live) {
          *reinterpret_cast<uint2 *>(codes + 8 * c) = make_uint2(word[0], word[1]);
          if (c == 0) scales[off] = static_cast<uint8_t>(k + 127);
          scales[a.c.page + off * (D / 16) + c] = static_cast<uint8_t>(s8);
        }
      }
    }
  }
}

template <int D, int FMT>
cudaError_t write_t(const CacheWriteArgs &a, cudaStream_t stream) {
  cache_write_kernel<D, FMT><<<static_cast<unsigned>(cache_ctas(a.c, a.tokens)), kCacheThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// Eight e2m1 codes as bf16 pairs, first code in the low half of o[0].  The eight magnitudes are looked up a
// byte of the bf16 at a time: 0 0.5 1 1.5 2 3 4 6 are 0000 3F00 3F80 3FC0 4000 4040 4080 40C0.
__device__ __forceinline__ void e2m1x8_bf16(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t odd = w & 0x80808080u, even = (w << 4) & 0x80808080u;  // signs
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sel = (w >> (16 * h)) & 0x7777u;
    const uint32_t sign = __byte_perm(even, odd, h == 0 ? 0x5140 : 0x7362);
    const uint32_t top = __byte_perm(0x3F3F3F00u, 0x40404040u, sel) | sign, low = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    o[2 * h] = __byte_perm(low, top, 0x5140);
    o[2 * h + 1] = __byte_perm(low, top, 0x7362);
  }
}

// Thread (token, piece of 16 values of a row of K and of V); a CTA is one head of a stretch of tokens, whose
// codes and scales lie next to each other.
template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheReadArgs a) {
  constexpr int PPR = D / 16;
  constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;
  constexpr int PER = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
  if (blockIdx.x == 0)  // every entry is checked, whether or not a row of it is met below
    for (int b = threadIdx.x; b < a.batch; b += kCacheThreads) seq_span(a.cu, b, a.max_seqlen, a.total, a.status);
  const uint32_t block = blockIdx.x / a.c.hkv, g = blockIdx.x - block * a.c.hkv;
  const uint32_t at = block * (kCacheThreads / PPR) + threadIdx.x / PPR;  // (the last stretch may pass 2^31 tokens)
  if (at >= static_cast<uint32_t>(a.total)) return;
  const int t = static_cast<int>(at), c = threadIdx.x % PPR;
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
      if constexpr (FMT == BSA_CACHE_E4M3) {
        const float s = pow2i(static_cast<int>(scales[off]) - 127);
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(codes + 16 * c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = e4m3x2_f32(w[e]), q = e4m3x2_f32(w[e] >> 16);
          o[2 * e] = ptx::pack_bf16x2(p.x * s, p.y * s);
          o[2 * e + 1] = ptx::pack_bf16x2(q.x * s, q.y * s);
        }
      } else {
        // in bf16: a code times the group scale has at most six significant bits and is exact; the row's
        // power of two comes last, so that a row near bf16's smallest values is rounded once
        const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(codes + 8 * c));
        const float gs = e4m3x2_f32(scales[a.c.page + off * PPR + c]).x;
        const uint32_t g2 = __byte_perm(__float_as_uint(gs), 0u, 0x3232), s2 = scales[off] * 0x00800080u;
        uint32_t v[4];
        e2m1x8_bf16(u.x, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = mul_bf16x2(mul_bf16x2(v[e], g2), s2);
        e2m1x8_bf16(u.y, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 + e] = mul_bf16x2(mul_bf16x2(v[e], g2), s2);
      }
    }
    __stcs(out, make_uint4(o[0], o[1], o[2], o[3]));
    __stcs(out + 1, make_uint4(o[4], o[5], o[6], o[7]));
  }
}

template <int D, int FMT>
cudaError_t read_t(const CacheReadArgs &a, cudaStream_t stream) {
  cache_read_kernel<D, FMT><<<static_cast<unsigned>(cache_ctas(a.c, a.total)), kCacheThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// A CTA for every head of a stretch of tokens, the heads of a stretch next to each other.
int64_t cache_ctas(const CacheDims &c, int tokens) {
  const int per_cta = kCacheThreads / (c.d / 16);
  return (static_cast<int64_t>(tokens) + per_cta - 1) / per_cta * c.hkv;
}

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
