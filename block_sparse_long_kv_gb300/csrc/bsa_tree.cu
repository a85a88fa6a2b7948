// Attention of drafted tokens over the paged cache, split over the keys.
//
// Rows.  The drafted tokens of a sequence times the G heads of a KV group are
// query rows that share every key: row r is token r / G, head r % G.  There are
// at most sixteen, one tile, the M of one m16n8k16 MMA.  A group's keys are laid
// out in units of 64: the 64-key chunks of the kept pages, then the (at most
// sixteen) drafted tokens.  The units of all groups are laid end to end and cut
// into equal runs, one per CTA, so that a short batch and a ragged one load every
// SM alike.
//
// One CTA streams its run through a cp.async ring; each of its four warps owns
// 16 keys of a chunk and keeps its own online softmax.  With few rows the
// kernel is bound by the cache's bytes, so codes go from shared memory to MMA
// fragments without a bf16 copy in between:
//   - K: thread tq of a key's four lanes takes a quarter of its dimensions, in
//     order; Q's fragments are loaded in the same order, since a dot product
//     does not care.  Codes become f16 (exact: at most six significant bits
//     between 2^-10 and 2688); the row's power of two multiplies the logit.
//   - V: lane group gq takes an eighth of the dimensions of four keys and
//     interleaves pairs of keys by byte permutes; O's columns come out in that
//     order.  The row's power of two multiplies P instead (below).
// Q of an 8- or 4-bit cache becomes f16 after a power of two per row that
// brings its largest element to [2^14, 2^15): bf16's eight bits fit f16's eleven
// and what lies 2^28 below the largest element loses bits.
//
// The softmax reference m of a row moves only when its maximum has grown by more
// than 2^TH, so that O is rarely rescaled; p <= 2^TH.
//
// P of an 8- or 4-bit cache is P' = p * 2^(e - eref + SHIFT) in f16, e the exponent
// of the key's V row and eref the largest seen, O held in units of 2^(eref - SHIFT):
// SHIFT = 15 - TH keeps P' within f16 and leaves 25 powers of two below the largest
// product at f16's full 2^-11, 10 more with fewer bits.  (The lag TH costs four of
// those; without it O is rescaled in most steps.)  P of a bf16 cache and of the drafted
// tokens is bf16, 2^-8 relative at any size: one token over 131072 is 0.0023 off in
// relative norm where fp32 weights would leave 0.0016, the rounding of the result.
// Sums and statistics are fp32 from unrounded p.
//
// One token over 131072 cached, 32 / 4 heads of 128: bf16 55 us (269 MB: 4.9 TB/s; about 15 us of it are the
// plan, the first chunk and the combine), e4m3 43, e2m1 44.  Over codes no unit is saturated: 42 to 49 %
// of the issue slots and 39 to 44 % of the integer pipe are taken, at three warps a scheduler, which do not cover
// the latencies.
//
// Groups that one CTA holds whole are written by it; of the others every CTA
// leaves an unnormalised part (O, max, sum), which tree_combine_kernel merges in
// a fixed order, so the result does not depend on timing.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "bsa_cache.h"
#include "bsa_internal.h"
#include "bsa_tree.cuh"
#include "sm103_ptx.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;        // rows of a tile
constexpr int kKeys = 64;        // keys of a unit
constexpr int kBatch = kThreads; // units resolved at a time
constexpr int kSms = 152;
constexpr int kMaxCtas = 3 * kSms;

template <int D, int FMT>
struct Cfg {
  static constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;  // bytes of a row
  static constexpr int PER = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
  static constexpr int CODE = kKeys * RB;
  static constexpr int SCALE = kKeys * PER;
  static constexpr int STAGE = 2 * (CODE + SCALE);
  // resident CTAs per SM (the register limit allows three) and ring stages that fill the 227 KB
  static constexpr int CTAS = FMT == BSA_CACHE_BF16 && D == 128 ? 2 : 3;
  static constexpr int STAGES = STAGE > 12000 ? 3 : 4;
  static constexpr int TH = FMT == BSA_CACHE_BF16 ? 8 : 4;
  static constexpr int SHIFT = FMT == BSA_CACHE_BF16 ? 0 : 15 - TH;
  static constexpr int UNIT1 = 127 + SHIFT;  // the exponent reference at which O's unit is 1
  static constexpr int NKS = D / 16;  // k-steps of S
  static constexpr int NNT = D / 8;   // n-tiles of O
  static constexpr int TB = RB / 4;   // bytes of a key row per thread
  static constexpr int VB = RB / 8;   // bytes of a value row per lane group
  static constexpr int LDO = D + 8;   // row of the merge buffer, in floats (the pad spreads the rows over the banks)
  static constexpr int OFF_O = STAGES * STAGE;
  static constexpr int OFF_ML = OFF_O + kRows * LDO * 4;            // [2][warps][16] floats
  static constexpr int OFF_MASK = OFF_ML + 2 * kWarps * kRows * 4;  // [16] the drafted tokens that a row sees
  static constexpr int OFF_UNIT = OFF_MASK + kRows * 4;             // [2][kBatch] int4
  static constexpr int OFF_PRE = OFF_UNIT + 2 * kBatch * 16;        // [groups + 1] first unit
  static size_t smem(int groups) { return OFF_PRE + static_cast<size_t>(groups + 1) * 4; }
};

// 16-byte chunk permutations of the staged rows (an XOR of the chunk index), such that the eight
// lanes of a phase of the loads below meet eight different chunks of the 128-byte bank line.
template <int RB>
__device__ __forceinline__ int k_swizzle(int row) {
  return RB == 256 ? (row & 1) << 2 : RB == 128 ? row & 7 : 0;
}
template <int RB>
__device__ __forceinline__ int v_swizzle(int row) {
  return RB == 256 ? ((row >> 1) & 1) | (row & 4) : RB == 128 ? row & 7 : RB == 64 ? row & 2 : 0;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool live) {
  const int n = live ? 16 : 0;  // 0: zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first of the two adjacent dimensions in word `which` of k-step ks of thread tq.
template <int D, int FMT>
__device__ __forceinline__ int frag_dim(int ks, int tq, int which) {
  if (FMT == BSA_CACHE_BF16 && D == 128) return (4 * (ks >> 1) + tq) * 8 + (ks & 1) * 4 + which * 2;
  return tq * (D / 4) + ks * 4 + which * 2;
}

// Exclusive prefix sum over the CTA's threads in thread order; *total gets the sum.
__device__ __forceinline__ int cta_scan(int c, int *total, int *wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int off = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    off += w < warp ? wsum[w] : 0;
    tot += wsum[w];
  }
  __syncthreads();
  *total = tot;
  return off + inc - c;
}

// A unit: .x the group (b * hkv + g), .y the cache tile (page * hkv + g; -1: drafted tokens, or nothing), .z its
// keys, .w its 64-key chunk of the page.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, Cfg<D, FMT>::CTAS) tree_attn_kernel(const TreeArgs a, float *part_o, float *part_ml,
                                                                        TreeRun *runs) {
  using C = Cfg<D, FMT>;
  constexpr bool Q16 = FMT != BSA_CACHE_BF16;  // f16 fragments
  extern __shared__ __align__(16) unsigned char smem[];
  float *obuf = reinterpret_cast<float *>(smem + C::OFF_O);
  float(*wm)[kRows] = reinterpret_cast<float(*)[kRows]>(smem + C::OFF_ML);
  float(*wl)[kRows] = wm + kWarps;
  uint32_t *dmask = reinterpret_cast<uint32_t *>(smem + C::OFF_MASK);
  int4 *unit = reinterpret_cast<int4 *>(smem + C::OFF_UNIT);
  int *pre = reinterpret_cast<int *>(smem + C::OFF_PRE);
  const int groups = a.batch * a.c.hkv;
  __shared__ int wsum[kWarps];
  __shared__ int not_finite_flag;  // drafted values of the group held Inf or NaN
  volatile int *not_finite_v = &not_finite_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const int cta = blockIdx.x, G = a.group;
  const int cpp = a.c.page / kKeys;

  // ---- the plan: first unit of every group
  {
    const int each = (groups + kThreads - 1) / kThreads;
    const int g0 = min(groups, tid * each), g1 = min(groups, g0 + each);
    int local = 0;
    for (int x = g0; x < g1; ++x) {
      const int b = x / a.c.hkv;
      const int listed = a.kv_cnt == nullptr ? INT32_MAX : __ldg(a.kv_cnt + x);  // (the loads in one round)
      const int n = cached_of(a, b);
      const Drafts dr = drafts_of(a, b);
      const int pages = (n + a.c.page - 1) >> a.c.page_shift;
      const int kept = max(0, min(listed, pages));
      // without a list the chunks past the last token are not units at all
      const int ku = a.kv_cnt == nullptr ? (n + kKeys - 1) / kKeys : kept * cpp;
      pre[x] = dr.len > 0 ? ku + 1 : 0;
      local += pre[x];
    }
    int n;
    int run = cta_scan(local, &n, wsum);
    for (int x = g0; x < g1; ++x) {
      const int c = pre[x];
      pre[x] = run;
      run += c;
    }
    if (tid == 0) {
      pre[groups] = n;
      *not_finite_v = 0;
    }
    __syncthreads();
  }
  const int n_all = pre[groups];
  const int W = (n_all + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int x0 = min(n_all, cta * W), x1 = min(n_all, x0 + W);
  if (x0 >= x1) {  // CTA-uniform
    if (tid == 0) runs[cta].group = -1;
    return;
  }
  const int nu = x1 - x0;

  auto resolve = [&](int first) {  // units first .. first + kBatch - 1 of the run, one per thread
    const int u = first + tid;
    if (u >= nu) return;
    const int x = x0 + u;
    int lo = 0, hi = groups - 1;
    while (lo < hi) {  // the last group with pre <= x (empty groups have none of their own)
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo / a.c.hkv, k = x - pre[lo];
    const int n = cached_of(a, b);
    int4 d = make_int4(lo, -1, 0, 0);
    if (k == pre[lo + 1] - pre[lo] - 1) {
      d.z = drafts_of(a, b).len;
    } else {
      const int e = k >> (a.c.page_shift - 6), sub = k & (cpp - 1);
      const int j = a.kv_idx == nullptr ? e : __ldg(a.kv_idx + static_cast<size_t>(lo) * a.table_stride + e);
      if (j >= 0 && j < (n + a.c.page - 1) >> a.c.page_shift) {
        const int pg = __ldg(a.table + static_cast<size_t>(b) * a.table_stride + j);
        if (pg >= 0 && pg < a.c.pages) {
          d.y = pg * a.c.hkv + (lo - b * a.c.hkv);
          d.z = max(0, min(kKeys, n - j * a.c.page - sub * kKeys));
          d.w = sub;
        } else if (a.status != nullptr) {
          atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
        }
      } else if (j < 0 && a.status != nullptr) {
        atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
      }
    }
    unit[u % (2 * kBatch)] = d;
  };

  // A thread copies the same 16-byte column of rows a fixed step apart (a multiple of eight, or of the
  // swizzles' period), so every address is one of a few bases plus a constant.
  constexpr int PR = C::RB / 16, STEP = kThreads / PR, COPIES = kKeys / STEP;
  const int crow = tid / PR, ccol = tid % PR;
  const uint32_t k_dst = ptx::smem_addr(smem) + crow * C::RB + (ccol ^ k_swizzle<C::RB>(crow)) * 16;
  const uint32_t v_dst = ptx::smem_addr(smem) + C::CODE + crow * C::RB + (ccol ^ v_swizzle<C::RB>(crow)) * 16;
  auto issue = [&](int u) {
    if (u < nu) {
      const int4 d = unit[u % (2 * kBatch)];
      const int n = d.z;
      if (d.y >= 0 && n > 0) {
        const uint32_t st = static_cast<uint32_t>(u % C::STAGES) * C::STAGE;
        const int sub = d.w;
        const size_t at = (static_cast<size_t>(d.y) * a.c.page + sub * kKeys) * C::RB + tid * 16;
        const uint8_t *ks = a.k_codes + at, *vs = a.v_codes + at;
        if (n == kKeys) {
#pragma unroll
          for (int i = 0; i < COPIES; ++i) {
            cp16(k_dst + st + i * STEP * C::RB, ks + i * kThreads * 16);
            cp16(v_dst + st + i * STEP * C::RB, vs + i * kThreads * 16);
          }
        } else {
#pragma unroll
          for (int i = 0; i < COPIES; ++i) {
            const bool live = crow + i * STEP < n;
            cp16_or_zero(k_dst + st + i * STEP * C::RB, ks + i * kThreads * 16, live);
            cp16_or_zero(v_dst + st + i * STEP * C::RB, vs + i * kThreads * 16, live);
          }
        }
        if constexpr (C::PER > 0) {
          // the exponents of the chunk's 64 rows, then their group scales
          const size_t sc = static_cast<size_t>(d.y) * a.c.page * C::PER;
          constexpr int PS = kKeys * C::PER / 16;
          if (tid < PS) {
            const size_t from = tid < kKeys / 16 ? sc + sub * kKeys + tid * 16
                                                 : sc + a.c.page + static_cast<size_t>(sub) * kKeys * (C::PER - 1) +
                                                       (tid - kKeys / 16) * 16;
            const uint32_t to = ptx::smem_addr(smem) + st + 2 * C::CODE + tid * 16;
            cp16(to, a.k_scales + from);
            cp16(to + C::SCALE, a.v_scales + from);
          }
        }
      }
    }
    cp_commit();  // one group per unit, empty for drafted tokens and past the run
  };

  uint32_t qa[C::NKS][4];
  float o[C::NNT][4];
  float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
  float sc_lo = a.scale_log2, sc_hi = a.scale_log2;  // logit scales of the rows gq and gq + 8
  int eref = 0;  // O is in units of 2^(eref - UNIT1); 0: nothing yet
  int arow_g = -1;
  Drafts adr{0, 0};

  // row r of q; null past the drafts
  auto q_row = [&](int r) -> const uint16_t * {
    const int t = r / G;
    if (t >= adr.len) return nullptr;
    const int g = arow_g % a.c.hkv;
    return a.q + (static_cast<size_t>(adr.start + t) * a.hq + g * G + r % G) * D;
  };

  auto start_group = [&](int grp) {
    arow_g = grp;
    adr = drafts_of(a, grp / a.c.hkv);
    const uint16_t *qlo = q_row(gq), *qhi = q_row(gq + 8);
    float am_lo = 0.f, am_hi = 0.f;
#pragma unroll
    for (int ks = 0; ks < C::NKS; ++ks)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int dim = frag_dim<D, FMT>(ks, tq, w);
        const uint32_t u = qlo != nullptr ? *reinterpret_cast<const uint32_t *>(qlo + dim) : 0u;
        const uint32_t v = qhi != nullptr ? *reinterpret_cast<const uint32_t *>(qhi + dim) : 0u;
        qa[ks][2 * w] = u;
        qa[ks][2 * w + 1] = v;
        if constexpr (Q16) {
          am_lo = fmaxf(am_lo, fmaxf(fabsf(__uint_as_float(u << 16)), fabsf(__uint_as_float(u & 0xFFFF0000u))));
          am_hi = fmaxf(am_hi, fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xFFFF0000u))));
        }
      }
    if constexpr (Q16) {
#pragma unroll
      for (int off = 1; off <= 2; off <<= 1) {
        am_lo = fmaxf(am_lo, __shfl_xor_sync(0xffffffffu, am_lo, off));
        am_hi = fmaxf(am_hi, __shfl_xor_sync(0xffffffffu, am_hi, off));
      }
      // the biased exponent of 2^-(e - 14), e the exponent of the largest element, kept normal
      const int e_lo = max(1, min(253, 268 - (__float_as_int(am_lo) >> 23)));
      const int e_hi = max(1, min(253, 268 - (__float_as_int(am_hi) >> 23)));
      const float f_lo = pow2_biased(e_lo), f_hi = pow2_biased(e_hi);
      sc_lo = a.scale_log2 * pow2_biased(254 - e_lo);
      sc_hi = a.scale_log2 * pow2_biased(254 - e_hi);
#pragma unroll
      for (int ks = 0; ks < C::NKS; ++ks)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = (w & 1) ? f_hi : f_lo;
          const uint32_t u = qa[ks][w];
          qa[ks][w] = pack_f16x2(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xFFFF0000u) * f);
        }
    }
#pragma unroll
    for (int nt = 0; nt < C::NNT; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
    m_lo = m_hi = -INFINITY;
    l_lo = l_hi = 0.f;
    eref = 0;
  };

  // Merges the four warps' O, max and sum of the group, and writes the rows or the part.
  auto flush = [&]() {
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      l_lo += __shfl_xor_sync(0xffffffffu, l_lo, off);
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, off);
    }
    m_lo = ptx::part_max(m_lo, l_lo);
    m_hi = ptx::part_max(m_hi, l_hi);
    if (tq == 0) {
      wm[warp][gq] = m_lo;
      wm[warp][gq + 8] = m_hi;
      wl[warp][gq] = l_lo;
      wl[warp][gq + 8] = l_hi;
    }
    __syncthreads();
    float mlo = -INFINITY, mhi = -INFINITY;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      mlo = ptx::max_nan(mlo, wm[x][gq]);
      mhi = ptx::max_nan(mhi, wm[x][gq + 8]);
    }
    const float unit_f = Q16 && eref != 0 ? exp2f(static_cast<float>(eref - C::UNIT1)) : 1.f;
    const float slo = m_lo == -INFINITY ? 0.f : ptx::ex2_approx(m_lo - mlo) * unit_f;
    const float shi = m_hi == -INFINITY ? 0.f : ptx::ex2_approx(m_hi - mhi) * unit_f;
    // One warp after another: a fixed order of the sums.  Element [row][8 nt + c] is dimension c (D / 8) + nt.
    // (One copy of the code: a flush runs once or twice per CTA, from a cold instruction cache.)
#pragma unroll 1
    for (int x = 0; x < kWarps; ++x) {
      if (warp == x) {
        float *rlo = obuf + gq * C::LDO + 2 * tq, *rhi = rlo + 8 * C::LDO;
#pragma unroll
        for (int nt = 0; nt < C::NNT; ++nt) {
          float2 u = make_float2(0.f, 0.f), v = u;
          if (x > 0) {
            u = *reinterpret_cast<const float2 *>(rlo + 8 * nt);
            v = *reinterpret_cast<const float2 *>(rhi + 8 * nt);
          }
          *reinterpret_cast<float2 *>(rlo + 8 * nt) = make_float2(fmaf(o[nt][0], slo, u.x), fmaf(o[nt][1], slo, u.y));
          *reinterpret_cast<float2 *>(rhi + 8 * nt) = make_float2(fmaf(o[nt][2], shi, v.x), fmaf(o[nt][3], shi, v.y));
        }
      }
      __syncthreads();
    }
    const int rs = pre[arow_g], re = pre[arow_g + 1];
    const bool whole = rs >= x0 && re <= x1;
    const size_t slot = 2 * static_cast<size_t>(cta) + (rs <= x0 ? 0 : 1);
    const bool lost = *not_finite_v != 0;
    constexpr int PIECES = D / 4;
#pragma unroll 1
    for (int e = tid; e < kRows * PIECES; e += kThreads) {
      const int r = e / PIECES, d4 = 4 * (e % PIECES);
      const int t = r / G;
      if (t >= adr.len) continue;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) m = ptx::max_nan(m, wm[x][r]);
#pragma unroll
      for (int x = 0; x < kWarps; ++x)
        if (wm[x][r] != -INFINITY) l = fmaf(ptx::ex2_approx(wm[x][r] - m), wl[x][r], l);
      const float *from = obuf + r * C::LDO + d4 / (D / 8) + 8 * (d4 % (D / 8));
      float4 v = make_float4(from[0], from[8], from[16], from[24]);
      if (lost) {  // Inf and NaN of the drafted values the row sees
        const uint16_t *vn = a.v_new + (static_cast<size_t>(adr.start) * a.c.hkv + arow_g % a.c.hkv) * D + d4;
        for (int p = t; p >= 0; p = parent_of(a, adr.start, p)) {
          const uint2 u = *reinterpret_cast<const uint2 *>(vn + static_cast<size_t>(p) * a.c.hkv * D);
          v.x += not_finite(u.x);
          v.y += not_finite(u.x >> 16);
          v.z += not_finite(u.y);
          v.w += not_finite(u.y >> 16);
        }
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // (NaN where the sum is)
        const size_t at = static_cast<size_t>(adr.start + t) * a.hq + (arow_g % a.c.hkv) * G + r % G;
        *reinterpret_cast<uint2 *>(a.o + at * D + d4) =
            make_uint2(ptx::pack_bf16x2(v.x * inv, v.y * inv), ptx::pack_bf16x2(v.z * inv, v.w * inv));
        if (a.lse != nullptr && d4 == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float4 *>(part_o + (slot * kRows + r) * D + d4) = v;
        if (d4 == 0) *reinterpret_cast<float2 *>(part_ml + (slot * kRows + r) * 2) = make_float2(m, l);
      }
    }
    __syncthreads();  // obuf and wm are free again
    if (tid == 0) *not_finite_v = 0;
  };

  // The softmax step of a 16-key slice: x holds the logits (log2 units, -inf where masked), and on
  // return p; the row references, sums and O move on where they have to.  `fo` further scales O.
  auto softmax = [&](float (&x)[2][4], float fo) {
    float mx_lo = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
    float mx_hi = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, off));
      mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, off));
    }
    const bool up_lo = mx_lo > m_lo + static_cast<float>(C::TH), up_hi = mx_hi > m_hi + static_cast<float>(C::TH);
    if (__any_sync(0xffffffffu, up_lo || up_hi || fo != 1.f)) {
      float f_lo = 1.f, f_hi = 1.f;
      if (up_lo) {
        f_lo = m_lo == -INFINITY ? 0.f : ptx::ex2_approx(m_lo - mx_lo);
        m_lo = mx_lo;
      }
      if (up_hi) {
        f_hi = m_hi == -INFINITY ? 0.f : ptx::ex2_approx(m_hi - mx_hi);
        m_hi = mx_hi;
      }
      l_lo *= f_lo;
      l_hi *= f_hi;
      f_lo *= fo;
      f_hi *= fo;
#pragma unroll
      for (int nt = 0; nt < C::NNT; ++nt) {
        o[nt][0] *= f_lo;
        o[nt][1] *= f_lo;
        o[nt][2] *= f_hi;
        o[nt][3] *= f_hi;
      }
    }
    // (a row without any key so far has only -inf here, and p = 0)
    const float r_lo = m_lo == -INFINITY ? 0.f : m_lo, r_hi = m_hi == -INFINITY ? 0.f : m_hi;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = ptx::ex2_approx(x[nt][e] - (e < 2 ? r_lo : r_hi));
    l_lo += (x[0][0] + x[0][1]) + (x[1][0] + x[1][1]);
    l_hi += (x[0][2] + x[0][3]) + (x[1][2] + x[1][3]);
  };

  // One 64-key chunk of the cache; n keys of it are there.
  auto cached_chunk = [&](const unsigned char *st, int n) {
    const int k0 = warp * 16;
    if (k0 >= n) return;  // warp-uniform
    float s[2][4], s2[2][4];  // even and odd k-steps: two chains of MMAs per n-tile
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
    const unsigned char *ksc = st + 2 * C::CODE, *vsc = ksc + C::SCALE;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int key = k0 + nt * 8 + gq;
      const unsigned char *row = st + key * C::RB;
      constexpr int NW = C::TB / 4;  // words of the thread's quarter
      uint32_t w[NW];
      if constexpr (C::TB >= 16) {
#pragma unroll
        for (int j = 0; j < C::TB / 16; ++j) {
          const int c = C::RB == 256 ? 4 * j + tq : tq * (C::TB / 16) + j;
          const uint4 u = *reinterpret_cast<const uint4 *>(row + (c ^ k_swizzle<C::RB>(key)) * 16);
          w[4 * j] = u.x;
          w[4 * j + 1] = u.y;
          w[4 * j + 2] = u.z;
          w[4 * j + 3] = u.w;
        }
      } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(row + tq * 8);
        w[0] = u.x;
        w[1] = u.y;
      }
      if constexpr (FMT == BSA_CACHE_BF16) {
#pragma unroll
        for (int ks = 0; ks < C::NKS; ++ks) mma<true>(ks & 1 ? s2[nt] : s[nt], qa[ks], w[2 * ks], w[2 * ks + 1]);
      } else if constexpr (FMT == BSA_CACHE_E4M3) {
#pragma unroll
        for (int ks = 0; ks < C::NKS; ++ks)
          mma<false>(ks & 1 ? s2[nt] : s[nt], qa[ks], e4m3x2_f16(w[ks]), e4m3x2_f16(w[ks] >> 16));
      } else {
        // the thread's quarter is whole groups of 16 dimensions: four k-steps each
        constexpr int NG = D / 64;
        const unsigned char *gs = ksc + kKeys + key * (D / 16) + tq * NG;
        uint32_t g2[NG];
        if constexpr (NG == 2) {
          const uint32_t both = e4m3x2_f16(*reinterpret_cast<const uint16_t *>(gs));
          g2[0] = __byte_perm(both, both, 0x1010);
          g2[1] = __byte_perm(both, both, 0x3232);
        } else {
          const uint32_t one = e4m3x2_f16(*gs);
          g2[0] = __byte_perm(one, one, 0x1010);
        }
#pragma unroll
        for (int ks = 0; ks < C::NKS; ++ks) {
          const uint32_t h = w[ks / 2] >> (16 * (ks & 1));
          mma<false>(ks & 1 ? s2[nt] : s[nt], qa[ks], mul_f16x2(e2m1x2_f16(h), g2[ks / 4]),
                     mul_f16x2(e2m1x2_f16(h >> 8), g2[ks / 4]));
        }
      }
    }
    // logits, and for 8- and 4-bit caches the scales of P
    float fo = 1.f;
    float vs[2][2];
    int ev[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int key = k0 + nt * 8 + 2 * tq;
      float kf[2] = {1.f, 1.f};
      if constexpr (Q16) {
        const uint32_t ek = *reinterpret_cast<const uint16_t *>(ksc + key);
        const uint32_t e2 = *reinterpret_cast<const uint16_t *>(vsc + key);
        kf[0] = __int_as_float((ek & 0xFF) << 23);
        kf[1] = __int_as_float((ek >> 8) << 23);
        ev[nt][0] = key < n ? e2 & 0xFF : 0;
        ev[nt][1] = key + 1 < n ? e2 >> 8 : 0;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = Q16 ? (e < 2 ? sc_lo : sc_hi) * kf[e & 1] : a.scale_log2;
        s[nt][e] = (s[nt][e] + s2[nt][e]) * f;
      }
      if (n < k0 + 16) {  // warp-uniform: the slice is not whole
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key + (e & 1) >= n) s[nt][e] = -INFINITY;
      }
    }
    if constexpr (Q16) {
      int top = max(max(ev[0][0], ev[0][1]), max(ev[1][0], ev[1][1]));
#pragma unroll
      for (int off = 1; off <= 2; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
      if (top > eref) {
        fo = pow2_biased(127 + eref - top);
        eref = top;
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        vs[nt][0] = pow2_biased(ev[nt][0] - eref + C::UNIT1);
        vs[nt][1] = pow2_biased(ev[nt][1] - eref + C::UNIT1);
      }
    }
    softmax(s, fo);
    uint32_t pa[4];
    if constexpr (Q16) {
      pa[0] = pack_f16x2(s[0][0] * vs[0][0], s[0][1] * vs[0][1]);
      pa[1] = pack_f16x2(s[0][2] * vs[0][0], s[0][3] * vs[0][1]);
      pa[2] = pack_f16x2(s[1][0] * vs[1][0], s[1][1] * vs[1][1]);
      pa[3] = pack_f16x2(s[1][2] * vs[1][0], s[1][3] * vs[1][1]);
    } else {
      pa[0] = ptx::pack_bf16x2(s[0][0], s[0][1]);
      pa[1] = ptx::pack_bf16x2(s[0][2], s[0][3]);
      pa[2] = ptx::pack_bf16x2(s[1][0], s[1][1]);
      pa[3] = ptx::pack_bf16x2(s[1][2], s[1][3]);
    }
    // O += P V: the lane group's eighth of the dimensions, keys 2 tq, + 1, + 8, + 9
    constexpr int NV = C::VB / 4;
    uint32_t v[4][NV];
    uint32_t g01 = 0u, g23 = 0u;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int key = k0 + 2 * tq + (x & 1) + 8 * (x >> 1);
      const unsigned char *row = st + C::CODE + key * C::RB;
      if constexpr (C::VB >= 16) {
#pragma unroll
        for (int j = 0; j < C::VB / 16; ++j) {
          const uint4 u =
              *reinterpret_cast<const uint4 *>(row + ((gq * (C::VB / 16) + j) ^ v_swizzle<C::RB>(key)) * 16);
          v[x][4 * j] = u.x;
          v[x][4 * j + 1] = u.y;
          v[x][4 * j + 2] = u.z;
          v[x][4 * j + 3] = u.w;
        }
      } else if constexpr (C::VB == 8) {
        const uint2 u = *reinterpret_cast<const uint2 *>(row + ((gq >> 1) ^ v_swizzle<C::RB>(key)) * 16 + (gq & 1) * 8);
        v[x][0] = u.x;
        v[x][1] = u.y;
      } else {
        v[x][0] = *reinterpret_cast<const uint32_t *>(row + gq * 4);
      }
      if constexpr (FMT == BSA_CACHE_E2M1) {
        // (rows past the last key hold zero codes beside scale bytes that nobody wrote)
        const uint32_t g = key < n ? vsc[kKeys + key * (D / 16) + gq * (D / 8) / 16] : 0u;
        if (x < 2) g01 |= g << (8 * x);
        else g23 |= g << (8 * (x - 2));
      }
    }
    if constexpr (FMT == BSA_CACHE_BF16) {
#pragma unroll
      for (int w = 0; w < NV; ++w) {
        mma<true>(o[2 * w], pa, __byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x5410));
        mma<true>(o[2 * w + 1], pa, __byte_perm(v[0][w], v[1][w], 0x7632), __byte_perm(v[2][w], v[3][w], 0x7632));
      }
    } else if constexpr (FMT == BSA_CACHE_E4M3) {
#pragma unroll
      for (int w = 0; w < NV; ++w) {
        const uint32_t p0 = __byte_perm(v[0][w], v[1][w], 0x5140), p1 = __byte_perm(v[2][w], v[3][w], 0x5140);
        const uint32_t q0 = __byte_perm(v[0][w], v[1][w], 0x7362), q1 = __byte_perm(v[2][w], v[3][w], 0x7362);
        mma<false>(o[4 * w], pa, e4m3x2_f16(p0), e4m3x2_f16(p1));
        mma<false>(o[4 * w + 1], pa, e4m3x2_f16(p0 >> 16), e4m3x2_f16(p1 >> 16));
        mma<false>(o[4 * w + 2], pa, e4m3x2_f16(q0), e4m3x2_f16(q1));
        mma<false>(o[4 * w + 3], pa, e4m3x2_f16(q0 >> 16), e4m3x2_f16(q1 >> 16));
      }
    } else {
      const uint32_t s01 = e4m3x2_f16(g01), s23 = e4m3x2_f16(g23);
      constexpr uint32_t LOW = 0x0F0F0F0Fu;
#pragma unroll
      for (int w = 0; w < NV; ++w) {
        // bytes of (key, next key) pairs: even dimensions from the low nibbles, odd from the high
        const uint32_t e0 = (v[0][w] & LOW) | ((v[1][w] << 4) & ~LOW), e1 = (v[2][w] & LOW) | ((v[3][w] << 4) & ~LOW);
        const uint32_t d0 = ((v[0][w] >> 4) & LOW) | (v[1][w] & ~LOW), d1 = ((v[2][w] >> 4) & LOW) | (v[3][w] & ~LOW);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma<false>(o[8 * w + 2 * j], pa, mul_f16x2(e2m1x2_f16(e0 >> (8 * j)), s01),
                     mul_f16x2(e2m1x2_f16(e1 >> (8 * j)), s23));
          mma<false>(o[8 * w + 2 * j + 1], pa, mul_f16x2(e2m1x2_f16(d0 >> (8 * j)), s01),
                     mul_f16x2(e2m1x2_f16(d1 >> (8 * j)), s23));
        }
      }
    }
  };

  // The n <= 16 drafted tokens: bf16 straight from global memory, by the first warp.
  auto drafted_chunk = [&](int n) {
    if (warp == 0) {
      if (lane < kRows) {
        const int t = lane / G;
        uint32_t bits = 0u;
        if (t < adr.len)
          for (int p = t; p >= 0; p = parent_of(a, adr.start, p)) bits |= 1u << p;
        dmask[lane] = bits;
      }
      __syncwarp();
      const int g = arow_g % a.c.hkv;
      auto row_of = [&](const uint16_t *base, int key) -> const uint16_t * {
        return key < n ? base + (static_cast<size_t>(adr.start + key) * a.c.hkv + g) * D : nullptr;
      };
      const uint16_t *qlo = q_row(gq), *qhi = q_row(gq + 8);
      const uint16_t *kr[2] = {row_of(a.k_new, gq), row_of(a.k_new, 8 + gq)};
      auto word = [](const uint16_t *row, int dim) -> uint32_t {
        return row != nullptr ? *reinterpret_cast<const uint32_t *>(row + dim) : 0u;
      };
      float s[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll 4
      for (int ks = 0; ks < C::NKS; ++ks) {
        const int da = frag_dim<D, FMT>(ks, tq, 0), db = frag_dim<D, FMT>(ks, tq, 1);
        const uint32_t qf[4] = {word(qlo, da), word(qhi, da), word(qlo, db), word(qhi, db)};
        mma<true>(s[0], qf, word(kr[0], da), word(kr[0], db));
        mma<true>(s[1], qf, word(kr[1], da), word(kr[1], db));
      }
      const uint32_t b_lo = dmask[gq], b_hi = dmask[gq + 8];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = nt * 8 + 2 * tq + (e & 1);
          s[nt][e] = ((e < 2 ? b_lo : b_hi) >> key) & 1u ? s[nt][e] * a.scale_log2 : -INFINITY;
        }
      float fo = 1.f;
      if constexpr (Q16) {  // O to units of 1
        if (eref != 0) fo = exp2f(static_cast<float>(eref - C::UNIT1));
        eref = C::UNIT1;
      }
      softmax(s, fo);
      const uint32_t pa[4] = {ptx::pack_bf16x2(s[0][0], s[0][1]), ptx::pack_bf16x2(s[0][2], s[0][3]),
                              ptx::pack_bf16x2(s[1][0], s[1][1]), ptx::pack_bf16x2(s[1][2], s[1][3])};
      const uint16_t *vr[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) vr[x] = row_of(a.v_new, 2 * tq + (x & 1) + 8 * (x >> 1));
      uint32_t lost = 0u;  // not 0: Inf or NaN among the values
#pragma unroll
      for (int w = 0; w < C::NNT / 2; ++w) {
        const int dim = gq * (D / 8) + 2 * w;
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = finite_bf16x2(word(vr[e], dim), lost);
        mma<true>(o[2 * w], pa, __byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
        mma<true>(o[2 * w + 1], pa, __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
      }
      if (__any_sync(0xffffffffu, lost != 0u) && lane == 0) *not_finite_v = 1;  // (flush reads it behind a barrier)
    }
  };

  resolve(0);
  __syncthreads();
  if (tid == 0) {  // the run's first group, for the combine
    const int grp = unit[0].x;
    const Drafts dr = drafts_of(a, grp / a.c.hkv);
    runs[cta] = TreeRun{grp, 0, pre[grp], pre[grp + 1], W, dr.start, dr.len, 0};
  }
#pragma unroll
  for (int x = 0; x < C::STAGES - 1; ++x) issue(x);
  for (int u = 0; u < nu; ++u) {
    if ((u + C::STAGES - 1) % kBatch == 0) resolve(u + C::STAGES - 1);  // its buffer's units are all behind u
    const int4 d = unit[u % (2 * kBatch)];
    if (d.x != arow_g) {  // (Q's loads beside the unit's)
      if (arow_g >= 0) flush();
      start_group(d.x);
    }
    cp_wait<C::STAGES - 2>();  // unit u has landed
    __syncthreads();           // for every thread; and unit u - 1's stage and a resolved batch are free to use
    issue(u + C::STAGES - 1);
    if (d.z > 0) {
      if (d.y >= 0) cached_chunk(smem + (u % C::STAGES) * C::STAGE, d.z);
      else drafted_chunk(d.z);
    }
  }
  cp_wait<0>();  // only empty groups can remain
  flush();
}

// The groups that several CTAs share.  CTA x takes the x-th of them in the order of their first CTA: it
// begins in the run of CTA c - 1 and goes on in CTA c's, which has recorded it.  Row r:
// O = sum w_p O_p / sum w_p l_p over its parts p = c - 1 .., w_p = 2^(m_p - max m).  Warp w sums the parts
// w, w + 8, .. against its own maximum, and the eight sums are added in order.
constexpr int kCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const TreeArgs a, const float *part_o,
                                                                         const float *part_ml, const TreeRun *runs,
                                                                         int ctas) {
  constexpr int VL = D / 32;
  constexpr int U = 4;  // parts of a warp in flight
  after_previous_kernel();
  __shared__ float red_o[kCombineWarps][D];
  __shared__ float red_m[kCombineWarps], red_l[kCombineWarps];
  const int r = blockIdx.y;
  TreeRun run;
  const int c = shared_tile(runs, ctas, blockIdx.x, &run);
  if (c < 0) return;
  const int t = r / a.group;
  if (t >= run.drafts) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p0 = c - 1, np = (run.last - 1) / run.run - p0 + 1;
  // every part after the first begins its CTA's run; the first may be that CTA's last group
  auto at = [&](int p) {
    return (2 * static_cast<size_t>(p0 + p) + (p > 0 || run.first == p0 * run.run ? 0 : 1)) * kRows + r;
  };
  // each warp with its own running maximum
  float m = -INFINITY, l = 0.f, acc[VL];
#pragma unroll
  for (int x = 0; x < VL; ++x) acc[x] = 0.f;
  for (int pb = warp; pb < np; pb += U * kCombineWarps) {
    float2 ml[U];
    float v[U][VL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = pb + u * kCombineWarps;
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int x = 0; x < VL; ++x) v[u][x] = 0.f;
      if (p < np) {
        ml[u] = *reinterpret_cast<const float2 *>(part_ml + at(p) * 2);
        const float *src = part_o + at(p) * D + lane * VL;
        if constexpr (VL == 4) {
          const float4 q = *reinterpret_cast<const float4 *>(src);
          v[u][0] = q.x; v[u][1] = q.y; v[u][2] = q.z; v[u][3] = q.w;
        } else {
          const float2 q = *reinterpret_cast<const float2 *>(src);
          v[u][0] = q.x; v[u][1] = q.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ml[u].x == -INFINITY) continue;
      const float mn = ptx::max_nan(m, ml[u].x);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), wgt = exp2f(ml[u].x - mn);
      m = mn;
      l = fmaf(ml[u].y, wgt, l * f);
#pragma unroll
      for (int x = 0; x < VL; ++x) acc[x] = fmaf(v[u][x], wgt, acc[x] * f);
    }
  }
#pragma unroll
  for (int x = 0; x < VL; ++x) red_o[warp][lane * VL + x] = acc[x];
  if (lane == 0) {
    red_m[warp] = m;
    red_l[warp] = l;
  }
  __syncthreads();
  float mm = -INFINITY, fw[kCombineWarps];
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) mm = ptx::max_nan(mm, red_m[w]);
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) fw[w] = red_m[w] == -INFINITY ? 0.f : exp2f(red_m[w] - mm);
  const size_t out = static_cast<size_t>(run.draft0 + t) * a.hq + (run.group % a.c.hkv) * a.group + r % a.group;
  for (int d = threadIdx.x; d < D; d += kCombineWarps * 32) {
    float s = 0.f, ls = 0.f;
#pragma unroll
    for (int w = 0; w < kCombineWarps; ++w) {
      s = fmaf(red_o[w][d], fw[w], s);
      ls = fmaf(red_l[w], fw[w], ls);
    }
    const __nv_bfloat16 v = __float2bfloat16_rn(ls == 0.f ? 0.f : s / ls);
    a.o[out * D + d] = *reinterpret_cast<const uint16_t *>(&v);
    if (a.lse != nullptr && d == 0) a.lse[out] = ls == 0.f ? -INFINITY : (mm + log2f(ls)) * 0.69314718055994531f;
  }
}

struct Workspace {
  size_t part_o, part_ml, runs, total;
};
Workspace workspace_layout(int d) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Workspace w;
  w.part_o = 0;
  w.part_ml = up(2ull * kMaxCtas * kRows * d * 4);
  w.runs = w.part_ml + up(2ull * kMaxCtas * kRows * 2 * 4);
  w.total = w.runs + up(kMaxCtas * sizeof(TreeRun));
  return w;
}

template <int D, int FMT>
cudaError_t launch_t(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  using C = Cfg<D, FMT>;
  const Workspace ws = workspace_layout(D);
  char *base = static_cast<char *>(workspace);
  float *part_o = reinterpret_cast<float *>(base + ws.part_o), *part_ml = reinterpret_cast<float *>(base + ws.part_ml);
  TreeRun *runs = reinterpret_cast<TreeRun *>(base + ws.runs);
  auto kern = tree_attn_kernel<D, FMT>;
  const size_t smem = C::smem(a.batch * a.c.hkv);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_up(kern, C::smem(kMaxDecodeRows), 0, done);
  if (e != cudaSuccess) return e;
  kern<<<kSms * C::CTAS, kThreads, smem, stream>>>(a, part_o, part_ml, runs);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int ctas = kSms * C::CTAS, groups = a.batch * a.c.hkv;
  const int shared = groups < ctas - 1 ? groups : ctas - 1;  // at most: a run boundary each
  return launch_after(tree_combine_kernel<D>, dim3(shared, a.max_draft * a.group), kCombineWarps * 32, stream, a,
                      static_cast<const float *>(part_o), static_cast<const float *>(part_ml),
                      static_cast<const TreeRun *>(runs), ctas);
}

}  // namespace

size_t tree_workspace_bytes(const CacheDims &c, int batch, int hq, int max_draft) {
  return max_draft * (hq / c.hkv) > kRows ? tree_mma_workspace_bytes(c) : workspace_layout(c.d).total;
}

bsa_status launch_tree(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  // More rows than one tile would read the cache once for each here.  8 x 32768 cached tokens, 32 / 4 heads of 128,
  // bf16 / e4m3 / e2m1: 16 rows take 78 / 57 / 60 us here, so 32 would take about twice that; 87 / 109 / 103 on
  // tcgen05.  (A form with several row tiles took 15.5 us for 32 rows over one sequence of 2048, tcgen05 15 to 17.)
  if (a.max_draft * a.group > kRows) return launch_tree_mma(a, workspace, stream);
  cudaError_t e;
  const bool wide = a.c.d == 128;
  switch (a.c.format) {
    case BSA_CACHE_E4M3:
      e = wide ? launch_t<128, BSA_CACHE_E4M3>(a, workspace, stream) : launch_t<64, BSA_CACHE_E4M3>(a, workspace, stream);
      break;
    case BSA_CACHE_E2M1:
      e = wide ? launch_t<128, BSA_CACHE_E2M1>(a, workspace, stream) : launch_t<64, BSA_CACHE_E2M1>(a, workspace, stream);
      break;
    default:
      e = wide ? launch_t<128, BSA_CACHE_BF16>(a, workspace, stream) : launch_t<64, BSA_CACHE_BF16>(a, workspace, stream);
      break;
  }
  return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace bsa
