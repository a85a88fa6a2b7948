// Per-head norm of queries and keys with the position rotation in the same pass.
//
//   y = x * w / sqrt(mean(x^2) + eps),  then pairs of y turn by p * f_i
//
// Every value is read once and written once, about ten operations each, so the
// kernel is bound by HBM.  A row (one head of one token) belongs to D / 8
// lanes, eight dimensions and one 16-byte access each; the sum of squares is a
// butterfly over those lanes.  A warp takes whole tokens, one after another, and
// walks the heads of a token, all of which turn by the same angles: a lane
// computes the cosines and sines of its own dimensions once per token.  With
// few tokens the heads of a token are spread over warps instead, so that the
// step is one round of loads.
//
// The angle p * f is taken modulo one turn before any rounding: f / 2 pi as a
// 64-bit fraction of a turn times the integer p wraps modulo 2^64, which is
// exact, and its top 32 bits give the angle to 2^-32 of a turn at any
// position.  The product p * f in fp32 would be off by 2^-24 p radians.
//
// 131072 tokens x 36 heads of 128 out of the rows of a fused projection: 386 us, 6.3 TB/s.  The arithmetic is done on
// pairs of fp32 values: with single ones the instructions, not the loads, set the time (396 us).
// Six steps in flight on 24 warps per SM (4 to 12 bytes spill in the norm's forms): four on 32 warps spill more
// (399), four on 24 do not cover the loads (416), eight on 16 leave too few warps (451).  Heads of a token spread
// over two warps repeat the angles: 431.

#include <cuda_bf16.h>
#include <stdint.h>

#include "bsa_cache.h"
#include "sm103_ptx.cuh"

namespace bsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 3;  // resident per SM: up to 85 registers a thread

__device__ __forceinline__ float lo_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// f / 2 pi modulo one turn, in units of 2^-64 turns: f = m * 2^e with an integer m of 24 bits, times
// 2^64 / 2 pi as an integer of 62 bits, shifted.  Integer arithmetic: the double-precision pipe of this part
// is slow enough to show in a step.  For |f| < 2^16 the result is within 1 + |f| units (the shift drops up to one,
// the 62-bit constant is half a unit off), which the largest position takes to 2^-33 (1 + |f|) turns.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(f);
  const int ex = static_cast<int>((u >> 23) & 0xFFu);
  const uint64_t m = (u & 0x7FFFFFu) | (ex != 0 ? 0x800000u : 0u);
  const int right = 150 - (ex != 0 ? ex : 1);  // f = m * 2^-right
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  uint64_t r;
  if (right <= 0) r = right > -64 ? lo << -right : 0;
  else if (right < 64) r = (lo >> right) | (hi << (64 - right));
  else r = right < 128 ? hi >> (right - 64) : 0;
  return (u >> 31) ? 0 - r : r;
}

// cos and sin of p times the fraction.  The reduced angle lies in [-pi, pi), where the fast sine
// and cosine are within 2^-20; the bf16 result holds 2^-9.
__device__ __forceinline__ void rotation(int p, uint64_t frac, float &c, float &s) {
  const uint64_t turns = static_cast<uint64_t>(p) * frac;
  const float a = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  c = __cosf(a);
  s = __sinf(a);
}

// One warp: the heads [h0, h1) of a token, R = 32 / (D / 8) at a time; head h < hq is q's, the
// others are k's.  A lane's eight dimensions are two groups of four that turn with each other:
// half-split pairs (i, i + rotary / 2) put both in one lane, so nothing crosses lanes but the sum of
// squares, and a lane needs four angles.  Lane c of a row holds dimensions 4c .. and rotary / 2 + 4c ..
// while 8c < rotary, and its own eight past them; adjacent pairs are eight dimensions in a row anyway.
template <int D, bool PAIRS, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeArgs a, int heads_per_warp,
                                                                       int warps_per_token) {
  constexpr int LPR = D / 8;      // lanes per row
  constexpr int R = 32 / LPR;     // rows per warp step
  constexpr int U = 6;            // warp steps whose loads are in flight together
  const int lane = threadIdx.x & 31;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * (kRopeThreads / 32);
  int64_t w = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t items = static_cast<int64_t>(a.tokens) * warps_per_token;
  if (w >= items) return;
  const int heads = a.hq + a.hkv;
  const int sub = lane / LPR, c = lane % LPR;  // row of the step, lane of the row
  const bool rot = 8 * c < a.rotary;
  const int da = !PAIRS && rot ? 4 * c : 8 * c;
  const int db = !PAIRS && rot ? 4 * c + a.rotary / 2 : 8 * c + 4;
  auto load = [&](const uint16_t *p) -> uint4 {
    if constexpr (PAIRS) return __ldcs(reinterpret_cast<const uint4 *>(p + da));
    const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(p + da));
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p + db));
    return make_uint4(u.x, u.y, v.x, v.y);
  };
  uint64_t frac[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) frac[e] = rot ? turn_fraction(__ldg(a.inv_freq + 4 * c + e)) : 0;
  // eight values as pairs (xi, xj) that turn with each other
  auto unpack = [](const uint4 &u, uint64_t (&xi)[2], uint64_t (&xj)[2]) {
    if constexpr (PAIRS) {
      xi[0] = ptx::f32x2(lo_bf16(u.x), lo_bf16(u.y)), xj[0] = ptx::f32x2(hi_bf16(u.x), hi_bf16(u.y));
      xi[1] = ptx::f32x2(lo_bf16(u.z), lo_bf16(u.w)), xj[1] = ptx::f32x2(hi_bf16(u.z), hi_bf16(u.w));
    } else {
      xi[0] = ptx::f32x2(lo_bf16(u.x), hi_bf16(u.x)), xi[1] = ptx::f32x2(lo_bf16(u.y), hi_bf16(u.y));
      xj[0] = ptx::f32x2(lo_bf16(u.z), hi_bf16(u.z)), xj[1] = ptx::f32x2(lo_bf16(u.w), hi_bf16(u.w));
    }
  };
  uint64_t wi[2], wj[2];  // the norm's weights of q's or of k's heads
  int weights_of = -1;

  for (; w < items; w += n_warps) {
    const int64_t t = w / warps_per_token;
    const int h0 = static_cast<int>(w - t * warps_per_token) * heads_per_warp;
    const int h1 = min(heads, h0 + heads_per_warp);
    const uint16_t *qrow = a.q + t * a.q_stride, *krow = a.k + t * a.k_stride;
    uint16_t *qo = a.q_out + t * a.q_out_stride, *ko = a.k_out + t * a.k_out_stride;
    const int pos = __ldg(a.positions + t);
    if (pos < 0) continue;
    uint64_t cs[2], sn[2], minus_sn[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float c0, s0, c1, s1;
      rotation(pos, frac[2 * e], c0, s0);
      rotation(pos, frac[2 * e + 1], c1, s1);
      cs[e] = ptx::f32x2(c0, c1);
      sn[e] = ptx::f32x2(s0, s1);
      minus_sn[e] = ptx::f32x2(-s0, -s1);
    }
    for (int hb = h0; hb < h1; hb += R * U) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * R + sub;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < h1)
          raw[u] = load(h < a.hq ? qrow + static_cast<int64_t>(h) * D : krow + static_cast<int64_t>(h - a.hq) * D);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * R + sub;
        if (hb + u * R >= h1) break;  // warp-uniform
        const bool is_q = h < a.hq;
        uint64_t xi[2], xj[2];
        unpack(raw[u], xi, xj);
        if constexpr (NORM) {
          uint64_t s2 = mul_f32x2(xi[0], xi[0]);
          s2 = ptx::fma_f32x2(xi[1], xi[1], s2);
          s2 = ptx::fma_f32x2(xj[0], xj[0], s2);
          s2 = ptx::fma_f32x2(xj[1], xj[1], s2);
          float sa, sc;
          ptx::f32x2_split(s2, sa, sc);
          float ss = sa + sc;
#pragma unroll
          for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
          if (weights_of != static_cast<int>(is_q)) {  // twice a token
            weights_of = static_cast<int>(is_q);
            const uint16_t *wp = is_q ? a.q_weight : a.k_weight;
            unpack(wp != nullptr ? load(wp) : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), wi, wj);
          }
          const uint64_t inv2 = ptx::f32x2(inv, inv);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            xi[e] = mul_f32x2(mul_f32x2(xi[e], inv2), wi[e]);
            xj[e] = mul_f32x2(mul_f32x2(xj[e], inv2), wj[e]);
          }
        }
        if (rot) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t i = xi[e], j = xj[e];
            xi[e] = ptx::fma_f32x2(j, minus_sn[e], mul_f32x2(i, cs[e]));
            xj[e] = ptx::fma_f32x2(i, sn[e], mul_f32x2(j, cs[e]));
          }
        }
        if (h < h1) {
          uint16_t *out = is_q ? qo + static_cast<int64_t>(h) * D : ko + static_cast<int64_t>(h - a.hq) * D;
          float i[4], j[4];
          ptx::f32x2_split(xi[0], i[0], i[1]);
          ptx::f32x2_split(xi[1], i[2], i[3]);
          ptx::f32x2_split(xj[0], j[0], j[1]);
          ptx::f32x2_split(xj[1], j[2], j[3]);
          if constexpr (PAIRS) {
            __stcs(reinterpret_cast<uint4 *>(out + da),
                   make_uint4(ptx::pack_bf16x2(i[0], j[0]), ptx::pack_bf16x2(i[1], j[1]), ptx::pack_bf16x2(i[2], j[2]),
                              ptx::pack_bf16x2(i[3], j[3])));
          } else {
            __stcs(reinterpret_cast<uint2 *>(out + da), make_uint2(ptx::pack_bf16x2(i[0], i[1]), ptx::pack_bf16x2(i[2], i[3])));
            __stcs(reinterpret_cast<uint2 *>(out + db), make_uint2(ptx::pack_bf16x2(j[0], j[1]), ptx::pack_bf16x2(j[2], j[3])));
          }
        }
      }
    }
  }
}

template <int D, bool PAIRS>
cudaError_t launch_norm(const RopeArgs &a, bool norm, cudaStream_t stream) {
  constexpr int R = 32 / (D / 8);
  const int heads = a.hq + a.hkv;
  // A warp that keeps a token computes its angles once for all heads.  Below about two warps per
  // scheduler that leaves the GPU idle, so each warp takes one step of R heads.
  const bool spread = static_cast<int64_t>(a.tokens) < 152 * 8;
  const int per = spread ? R : heads;
  const int wpt = (heads + per - 1) / per;
  const int64_t warps = static_cast<int64_t>(a.tokens) * wpt;
  const int64_t most = 152 * kRopeCtas;
  const int64_t ctas = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const int64_t grid = ctas < most ? ctas : most;
  if (norm) rope_kernel<D, PAIRS, true><<<static_cast<unsigned>(grid), kRopeThreads, 0, stream>>>(a, per, wpt);
  else rope_kernel<D, PAIRS, false><<<static_cast<unsigned>(grid), kRopeThreads, 0, stream>>>(a, per, wpt);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int head_dim, bool pairs, bool norm, cudaStream_t stream) {
  if (head_dim == 64) return pairs ? launch_norm<64, true>(a, norm, stream) : launch_norm<64, false>(a, norm, stream);
  return pairs ? launch_norm<128, true>(a, norm, stream) : launch_norm<128, false>(a, norm, stream);
}

}  // namespace bsa
