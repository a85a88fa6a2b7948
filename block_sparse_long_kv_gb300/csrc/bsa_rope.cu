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

#include <cuda_bf16.h>
#include <stdint.h>

#include "bsa_cache.h"
#include "sm103_ptx.cuh"

namespace bsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 4;  // resident per SM

__device__ __forceinline__ float lo_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = lo_bf16(w[e]);
    f[2 * e + 1] = hi_bf16(w[e]);
  }
}

// f / 2 pi modulo one turn, in units of 2^-64 turns: f = m * 2^e with an integer m of 24 bits, times
// 2^64 / 2 pi as an integer of 62 bits, shifted.  Integer arithmetic: the double-precision pipe of this part
// is slow enough to show in a step.  For |f| < 2^16 the result is within |f| units.
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
  constexpr int U = 4;            // warp steps whose loads are in flight together
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
  const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  uint4 wq = ones, wk = ones;
  if constexpr (NORM) {
    if (a.q_weight != nullptr) wq = load(a.q_weight);
    if (a.k_weight != nullptr) wk = load(a.k_weight);
  }

  for (; w < items; w += n_warps) {
    const int64_t t = w / warps_per_token;
    const int h0 = static_cast<int>(w - t * warps_per_token) * heads_per_warp;
    const int h1 = min(heads, h0 + heads_per_warp);
    const uint16_t *qrow = a.q + t * a.q_stride, *krow = a.k + t * a.k_stride;
    uint16_t *qo = a.q_out + t * a.q_out_stride, *ko = a.k_out + t * a.k_out_stride;
    const int pos = __ldg(a.positions + t);
    if (pos < 0) continue;
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) rotation(pos, frac[e], cs[e], sn[e]);
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
        float x[8];
        unpack8(raw[u], x);
        if constexpr (NORM) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
          float wf[8];
          unpack8(is_q ? wq : wk, wf);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wf[e];
        }
        if (rot) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = PAIRS ? 2 * e : e, j = PAIRS ? 2 * e + 1 : e + 4;
            const float xi = x[i], xj = x[j];
            x[i] = xi * cs[e] - xj * sn[e];
            x[j] = xj * cs[e] + xi * sn[e];
          }
        }
        if (h < h1) {
          uint16_t *out = is_q ? qo + static_cast<int64_t>(h) * D : ko + static_cast<int64_t>(h - a.hq) * D;
          const uint2 u0 = make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
          const uint2 u1 = make_uint2(ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
          if constexpr (PAIRS) {
            __stcs(reinterpret_cast<uint4 *>(out + da), make_uint4(u0.x, u0.y, u1.x, u1.y));
          } else {
            __stcs(reinterpret_cast<uint2 *>(out + da), u0);
            __stcs(reinterpret_cast<uint2 *>(out + db), u1);
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
