// Attention of drafted tokens over the paged cache on tcgen05 tensor cores, for
// the many query rows of a tree (drafted tokens x heads of a KV group).
//
// Rows.  Query row r of a (sequence, KV head) is drafted token r / G, head r % G.
// 128 rows are one MMA tile.  Keys come in units of 128: pairs of the 64-key
// chunks of the kept pages, then the drafted tokens.  The units of all row tiles
// are laid end to end and cut into equal runs, one per CTA (one CTA per SM); a
// run crosses from one row tile into the next (segments).
//
// Two softmax lanes share the CTA's tensor core so that one lane's exponentials
// run under the other's MMAs:
//   PAIR   (more than 128 rows)  the lanes hold two row tiles and the same keys
//   !PAIR  (at most 128 rows)    the lanes hold the same rows and take alternate
//          units; their results are merged when the segment ends
// Warps:  0      TMEM owner; one thread issues S_t = Q_t K^T (both operands in
//                shared memory) and O_t += P_t V (P from TMEM, over S_t)
//         1      looks up the units (page of every chunk, keys there), 32 at a time and a batch ahead
//         4-7    loaders of K, 8-11 of V: bf16 pages by TMA; 8- and 4-bit codes by
//                cp.async into a ring of each thread's own pieces, from there into
//                f16 tiles with the 128-byte swizzle; partial chunks and drafted
//                tokens by hand
//         12-15, 16-19  the softmax lanes, one thread per query row; a lane also brings in its
//                rows of Q, the next segment's before it writes out the last one's result
//
// An 8- or 4-bit cache is computed in f16.  With e the exponent of a key's row and
// kref the largest of the unit, K' = code * 2^(e - kref + SHV) is exact down to
// e = kref - 21 (E4M3) or kref - 18 (E2M1, whose least value is half of 2^-9), and below
// that off by at most 2^-36 of the largest row's largest element (group scale and
// product are each half of 2^-24 off, in units of 2^-SHV); 2^(kref - 127 - SHV) joins the
// logit scale.  V likewise against oref, the largest exponent of the segment so far
// (drafted rows count too, and are held against it), O being held
// in units of 2^(oref - 127 - SHV - SHIFT).  Q rows become f16 after a power of
// two that brings their largest element to [2^14, 2^15), drafted K and V after one
// per unit.  P' = 2^(x - m + SHIFT) with the reference m at most 2^TH below the true
// maximum, so P' <= 2^15.  Row sums are fp32 from unrounded values.
//
// What bounds it: with two row tiles a unit is 32 MMAs of 64 cycles, 2048 cycles.  8 sequences of up to
// 32768 cached tokens, 64 drafted tokens, 32 / 4 heads of 128 (84 units a CTA): bf16 207 us, e4m3 243, e2m1
// 256 (0.93, 0.80 and 0.76 PFLOP/s; the MMAs alone 109).  From its logits to the last of P a lane takes 2400
// cycles, of which the other lane's products cover two thirds; keys are hardly ever waited for.  The lanes have a
// thousand instructions a unit and share the schedulers with the conversion, and the instruction cache shows: a
// warp waits for its code as long as it issues.  So code is kept short: logits are taken in two halves (the
// second is read from TMEM again), which also frees the registers for eight loader warps instead of four (e2m1
// 327 -> 268); and the loaders' handling of drafted rows, which is rare, keeps few loads in flight, or the codec beside
// it spills (e4m3 243 -> 278).  The issuing thread looks at both halves of P, V and the next K before its products: a look between
// them left the tensor core idle (e4m3 with P in quarters 256).
// Measured and not kept: two threads a row (297), the conversion or the halves unrolled (355, 260), all 128 logits
// in registers with four loader warps (bf16 190, e4m3 250, e2m1 293), running pointers in the loaders (257),
// deeper rings (no change), waits that poll instead of parking (+4 %).
// Every mbarrier wait is bounded, as in the prefill kernel.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "bsa_cache.h"
#include "bsa_internal.h"
#include "bsa_mma.cuh"
#include "bsa_tree.cuh"
#include "bsa_wait.cuh"
#include "sm103_ptx.cuh"

namespace bsa {
namespace {

using wait::Ctl;
using wait::drain_bar;
using namespace mma;

constexpr int kSms = 152;
constexpr size_t kMaxSmem = 227 * 1024;  // a CTA may have
constexpr int kThreads = 640;
constexpr int kLaunchRegs = 96;  // per thread
constexpr int kRows = 128;     // rows of a tile
constexpr int kUnit = 128;     // keys of a unit
constexpr int kChunk = 64;     // keys of a page chunk
constexpr int kBatch = 32;     // units looked up at a time, one per lane
constexpr int kLists = 3;      // batches kept
constexpr int kInfo = 8;       // units whose scales are kept
constexpr int kRegMma = 56, kRegLoad = 80, kRegSoft = 128;
static_assert(128 * (kRegMma + 2 * kRegLoad + 2 * kRegSoft) <= kThreads * kLaunchRegs, "register split exceeds the launch");

template <int D, int FMT, bool PAIR>
struct Cfg {
  static constexpr bool Q16 = FMT != BSA_CACHE_BF16;
  static constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;
  static constexpr int PER = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
  static constexpr int PP = Q16 ? RB / 16 : 1;     // 16-byte pieces of a code row
  static constexpr int NP = Q16 ? PP : 1;          // pieces of a unit per loader thread
  static constexpr int SHV = FMT == BSA_CACHE_E4M3 ? 6 : 4;  // 448 * 2^6 and 2688 * 2^4 stay below 2^16
  static constexpr int TH = Q16 ? 4 : 8;           // log2 of how far the reference may lag the maximum
  static constexpr int SHIFT = Q16 ? 15 - TH : 0;
  static constexpr int NTQ = PAIR ? 2 : 1;
  static constexpr int NCH = D / 64;               // 128-byte swizzle chunks per row
  static constexpr uint32_t TILE = 128u * D * 2;
  static constexpr uint32_t CHUNK = 128u * 128;    // one swizzle chunk column of a tile
  static constexpr int KS = 2, VS = PAIR || Q16 ? 2 : 3;
  static constexpr int GRP = 2;                    // pieces of a cp.async group
  static constexpr int NG = Q16 ? NP / GRP : 1;    // groups of a unit
  static constexpr int RING = 3;                   // groups in flight per thread
  static constexpr uint32_t CODES = Q16 ? 256u * RING * GRP * 16 : 0;  // of the eight loader warps
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + NTQ * TILE;
  static constexpr uint32_t OFF_V = OFF_K + KS * TILE;
  static constexpr uint32_t OFF_CODE = OFF_V + VS * TILE;
  static constexpr uint32_t OFF_BAR = OFF_CODE + CODES;
  static constexpr int NPC = 2;                    // P released in halves of 64 keys
  static constexpr int B_QF = 0, B_QE = 2, B_KF = 3, B_KE = B_KF + KS, B_VF = B_KE + KS, B_VE = B_VF + VS,
                       B_SF = B_VE + VS, B_PR = B_SF + 2, B_OD = B_PR + 2 * NPC, B_OE = B_OD + 2, B_UN = B_OE + 2,
                       B_UG = B_UN + kLists, B_IK = B_UG + 1, B_IV = B_IK + kInfo, B_RS = B_IV + kInfo, B_LK = B_RS + 2,
                       B_LV = B_LK + 1, B_LA = B_LV + 1, B_LB = B_LA + 1, B_FIN = B_LB + 1, NBARS = B_FIN + 1;
  static constexpr uint32_t OFF_MISC = (OFF_BAR + NBARS * 8 + 15) / 16 * 16;  // TMEM address, abort flag, scan sums
  // [kInfo] K's scale, [kInfo] oref, [kInfo][4] whether a V loader warp met Inf or NaN in drafted rows
  static constexpr uint32_t OFF_INFO = OFF_MISC + 128;
  static constexpr uint32_t OFF_ROWS = OFF_INFO + kInfo * 12;                 // [2][NTQ * 128] row scales of Q
  static constexpr uint32_t OFF_RED = OFF_ROWS + 2 * NTQ * 128 * 4;           // [8] loader maxima
  static constexpr uint32_t OFF_UNIT = OFF_RED + 32;                          // [kLists][kBatch] {int4, int4}
  static constexpr uint32_t OFF_PRE = OFF_UNIT + kLists * kBatch * 32;        // [groups + 1] first unit
  static size_t smem(int groups) { return OFF_PRE + static_cast<size_t>(groups + 1) * 4 + 1024; }
  static constexpr uint32_t IDESC_S = Q16 ? ptx::idesc_bf16_f32(128, 128, false) & ~((1u << 7) | (1u << 10))
                                          : ptx::idesc_bf16_f32(128, 128, false);
  static constexpr uint32_t IDESC_O = Q16 ? ptx::idesc_bf16_f32(128, D, true) & ~((1u << 7) | (1u << 10))
                                          : ptx::idesc_bf16_f32(128, D, true);
  static constexpr int TM_O = 256;                 // S_0, S_1, O_0, O_1
  static_assert(PER >= 0 && NCH >= 1 && B_FIN < 64, "");
};

// Units of one row tile of group x, its row tiles, and the 64-key chunks of its kept pages.
struct GroupPlan {
  int per, tiles, chunks;
};
template <int NTQ>
__device__ __forceinline__ GroupPlan plan_of(const TreeArgs &a, int x) {
  const int b = x / a.c.hkv;
  const int listed = a.kv_cnt == nullptr ? 0 : __ldg(a.kv_cnt + x);  // (the loads in one round)
  const int n = cached_of(a, b);
  const Drafts dr = drafts_of(a, b);
  GroupPlan p;
  if (a.kv_cnt == nullptr) {
    p.chunks = (n + kChunk - 1) / kChunk;
  } else {
    const int pages = (n + a.c.page - 1) >> a.c.page_shift;
    p.chunks = max(0, min(listed, pages)) * (a.c.page / kChunk);
  }
  p.per = (p.chunks + 1) / 2 + (dr.len + kUnit - 1) / kUnit;
  p.tiles = (dr.len * a.group + kRows * NTQ - 1) / (kRows * NTQ);
  return p;
}

// A stretch of a CTA's run inside one row tile.
struct Segment {
  int grp, rt, first, units;  // group, row tile, first unit (of the whole plan) and units in this run
  int rs, re;                 // the row tile's units
};
template <int NTQ>
__device__ __forceinline__ Segment segment_at(const TreeArgs &a, const int *pre, int groups, int x, int x1) {
  int lo = 0, hi = groups - 1;
  while (lo < hi) {  // the last group with pre <= x
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  const int len = drafts_of(a, lo / a.c.hkv).len;
  const int tiles = (len * a.group + kRows * NTQ - 1) / (kRows * NTQ);
  const int per = (pre[lo + 1] - pre[lo]) / tiles;
  Segment s;
  s.grp = lo;
  s.rt = (x - pre[lo]) / per;
  s.rs = pre[lo] + s.rt * per;
  s.re = s.rs + per;
  s.first = x;
  s.units = min(s.re, x1) - x;
  return s;
}

template <int D, int FMT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    tree_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const TreeArgs a, float *part_o, float *part_ml, float *lane_o, TreeRun *runs) {
  using C = Cfg<D, FMT, PAIR>;
  constexpr bool Q16 = C::Q16;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char *sb = smem_raw + (base - raw);
  const uint32_t bar0 = base + C::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sb + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sb + C::OFF_MISC + 4);
  int *scan = reinterpret_cast<int *>(sb + C::OFF_MISC + 16);  // [16]
  float *info_k = reinterpret_cast<float *>(sb + C::OFF_INFO);
  int *info_v = reinterpret_cast<int *>(info_k + kInfo);
  uint32_t *lost_v = reinterpret_cast<uint32_t *>(info_v + kInfo);
  float *row_scale = reinterpret_cast<float *>(sb + C::OFF_ROWS);
  float *red = reinterpret_cast<float *>(sb + C::OFF_RED);
  int4 *unit = reinterpret_cast<int4 *>(sb + C::OFF_UNIT);
  int *pre = reinterpret_cast<int *>(sb + C::OFF_PRE);
  // waits watch this CTA's own flag only: *status also carries reports about the arguments
  const Ctl ctl{abort_flag, nullptr};
  auto put16 = [&](uint32_t at, uint4 v) { *reinterpret_cast<uint4 *>(sb + at) = v; };
  // a whole warp waits, and goes on or gives up together
  auto wait_warp = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait_parked(bar(i), parity, ctl)) != 0; };
  auto arrive_warp = [&](int i) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar(i));
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, G = a.group, groups = a.batch * a.c.hkv;

  if (tid == 0) {
    for (int x = 0; x < C::NBARS; ++x) {
      // arrivals: 1 of a commit or the lookup warp, 2 of a commit and the thread that issues it (what it has seen is
      // then seen behind the barrier), 4 of the K or the V loaders' warps or a softmax lane, 8 of both lanes
      uint32_t count = 1;
      if (x >= C::B_OD && x < C::B_OE)
        count = 2;
      else if (x >= C::B_RS && x < C::B_LK)
        count = 8;
      else if (x < C::B_QE || (x >= C::B_KF && x < C::B_KE) || (x >= C::B_VF && x < C::B_VE) ||
               (x >= C::B_PR && x < C::B_OD) || (x >= C::B_OE && x < C::B_UN) || (x >= C::B_UG && x < C::B_FIN))
        count = 4;
      ptx::mbar_init(bar(x), count);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
    ptx::tmem_relinquish();
  }

  // ---- the plan: first unit of every group
  {
    const int each = (groups + kThreads - 1) / kThreads;
    const int g0 = min(groups, tid * each), g1 = min(groups, g0 + each);
    int local = 0;
    for (int x = g0; x < g1; ++x) {
      const GroupPlan p = plan_of<C::NTQ>(a, x);
      pre[x] = p.per * p.tiles;
      local += pre[x];
    }
    int inc = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int run = inc - local, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) run += scan[w];
      total += scan[w];
    }
    for (int x = g0; x < g1; ++x) {
      const int c = pre[x];
      pre[x] = run;
      run += c;
    }
    if (tid == 0) pre[groups] = total;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_all = pre[groups];
  const int W = (n_all + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int x0 = min(n_all, cta * W), x1 = min(n_all, x0 + W);
  if (tid == 0) {  // the run's first row tile, for the combine
    if (x0 < x1) {
      const Segment s = segment_at<C::NTQ>(a, pre, groups, x0, x1);
      const Drafts dr = drafts_of(a, s.grp / a.c.hkv);
      runs[cta] = TreeRun{s.grp, s.rt, s.rs, s.re, W, dr.start, dr.len, 0};
    } else {
      runs[cta].group = -1;
    }
  }

  if (warp < 4) {
    ptx::setmaxnreg_dec<kRegMma>();
    if (warp == 0 && lane == 0 && x0 < x1) {
      // ================================================================ MMA issuer
      const uint64_t dq0 = ptx::sdesc_sw128(base + C::OFF_Q, 16, 1024);
      const uint64_t dk0 = ptx::sdesc_sw128(base + C::OFF_K, 16, 1024);
      const uint64_t dv0 = ptx::sdesc_sw128(base + C::OFF_V, C::CHUNK, 1024);
      auto issue_s = [&](int t, int ks) {
        const uint64_t dq = dq0 + static_cast<uint64_t>(PAIR ? t : 0) * (C::TILE >> 4);
        const uint64_t dk = dk0 + static_cast<uint64_t>(ks) * (C::TILE >> 4);
        const uint32_t dst = tmem + t * 128;
        constexpr int NEXT = C::CHUNK >> 4;  // 16 dimensions are 32 bytes, four steps a swizzle chunk
        mma_ss_at<0, 0, true>(dst, dq, dk, C::IDESC_S);
        mma_ss_at<2, 2, false>(dst, dq, dk, C::IDESC_S);
        mma_ss_at<4, 4, false>(dst, dq, dk, C::IDESC_S);
        mma_ss_at<6, 6, false>(dst, dq, dk, C::IDESC_S);
        if constexpr (D == 128) {
          mma_ss_at<NEXT, NEXT, false>(dst, dq, dk, C::IDESC_S);
          mma_ss_at<NEXT + 2, NEXT + 2, false>(dst, dq, dk, C::IDESC_S);
          mma_ss_at<NEXT + 4, NEXT + 4, false>(dst, dq, dk, C::IDESC_S);
          mma_ss_at<NEXT + 6, NEXT + 6, false>(dst, dq, dk, C::IDESC_S);
        }
        ptx::mma_commit(bar(C::B_SF + t));
      };
      uint32_t pv_count[2] = {0, 0};  // P V products issued for each lane
      // (nv: the unit whose V is waited for first, or -1)
      auto issue_pv = [&](int t, int vs, bool accumulate, int nv) -> bool {
        const uint64_t dv = dv0 + static_cast<uint64_t>(vs) * (C::TILE >> 4);
        const uint32_t dst = tmem + C::TM_O + t * 128, src = tmem + t * 128;
        const uint32_t parity = pv_count[t] & 1;
        auto chunk = [&](auto at, uint32_t acc) {  // 32 keys: two MMAs of 16
          constexpr int c = decltype(at)::value;
          mma_ts_at<16 * c, 256 * c>(dst, src, dv, C::IDESC_O, acc);
          mma_ts_at<16 * c + 8, 256 * c + 128>(dst, src, dv, C::IDESC_O, 1u);
        };
        // both halves are looked at before the first product: mostly both are there, and a look between the
        // products would leave the tensor core idle
        const uint32_t p0 = bar(C::B_PR + t * C::NPC), p1 = p0 + 8;
        const uint32_t vf = bar(C::B_VF + vs), v_parity = (static_cast<uint32_t>(nv) / C::VS) & 1;
        const bool there = nv < 0 || is_complete(vf, v_parity);
        const bool first = is_complete(p0, parity), second = is_complete(p1, parity);
        if (!there && !wait_parked(vf, v_parity, ctl)) return false;
        if (!first && !wait_parked(p0, parity, ctl)) return false;
        ptx::tc_fence_after();
        chunk(Int<0>{}, accumulate ? 1u : 0u);
        chunk(Int<1>{}, 1u);
        if (!second) {
          if (!wait_parked(p1, parity, ctl)) return false;
          ptx::tc_fence_after();
        }
        chunk(Int<2>{}, 1u);
        chunk(Int<3>{}, 1u);
        ++pv_count[t];
        return true;
      };
      auto done_with = [&](int t) {  // lane t's O of the segment
        ptx::mma_commit(bar(C::B_OD + t));
        ptx::mbar_arrive(bar(C::B_OD + t));
      };
      bool ok = true;
      bool k_there = false;  // K of the next unit was seen to be there
      uint32_t n = 0, n_seg = 0;
      uint32_t lane_segs[2] = {0, 0};  // segments in which the lane had a unit
      // the lane's first P V of a segment overwrites O: the last segment's must have been read
      auto o_free = [&](int t) -> bool {
        const uint32_t k = lane_segs[t]++;
        return k == 0 || wait_parked(bar(C::B_OE + t), (k - 1) & 1, ctl);
      };
      for (int x = x0; ok && x < x1;) {
        const Segment s = segment_at<C::NTQ>(a, pre, groups, x, x1);
        x += s.units;
        if (!(ok = wait_parked(bar(C::B_QF), n_seg & 1, ctl))) break;
        if (!PAIR && !(ok = wait_parked(bar(C::B_QF + 1), n_seg & 1, ctl))) break;
        for (int i = 0; i < s.units; ++i, ++n) {
          const uint32_t ks = n % C::KS, vs = n % C::VS;
          const bool last = i == s.units - 1;
          if (!k_there && !(ok = wait_parked(bar(C::B_KF + ks), (n / C::KS) & 1, ctl))) break;
          k_there = false;
          ptx::tc_fence_after();
          if constexpr (PAIR) {
            issue_s(0, ks);
            if (i > 0) {
              const uint32_t pvs = (n - 1) % C::VS;
              if (i == 1 && !(ok = o_free(1))) break;
              if (!(ok = issue_pv(1, pvs, i > 1, -1))) break;
              ptx::mma_commit(bar(C::B_VE + pvs));
            }
            if (i == 0) {
              if (!(ok = wait_parked(bar(C::B_QF + 1), n_seg & 1, ctl))) break;
              ptx::tc_fence_after();
            }
            issue_s(1, ks);
            ptx::mma_commit(bar(C::B_KE + ks));
            if (!last) k_there = is_complete(bar(C::B_KF + (n + 1) % C::KS), ((n + 1) / C::KS) & 1);
            // V(n) has two stages only and is refilled late: it is waited for as late as possible
            if (i == 0 && !(ok = o_free(0))) break;
            if (!(ok = issue_pv(0, vs, i > 0, static_cast<int>(n)))) break;
            if (last) {
              done_with(0);
              if (i == 0 && !(ok = o_free(1))) break;
              if (!(ok = issue_pv(1, vs, i > 0, -1))) break;
              ptx::mma_commit(bar(C::B_VE + vs));
              done_with(1);
            }
          } else {
            issue_s(i & 1, ks);
            ptx::mma_commit(bar(C::B_KE + ks));
            if (last) ptx::mma_commit(bar(C::B_QE));
            for (int j = i > 0 ? i - 1 : i; j <= i; ++j) {  // unit i - 1, and the last unit itself
              if (j == i && !last) break;
              const uint32_t nj = n - static_cast<uint32_t>(i - j), pvs = nj % C::VS;
              const int t = j & 1;
              if (j == t && !(ok = o_free(t))) break;
              if (!(ok = issue_pv(t, pvs, j >= 2, static_cast<int>(nj)))) break;
              ptx::mma_commit(bar(C::B_VE + pvs));
              if (j + 2 >= s.units) done_with(t);
            }
            if (!ok) break;
          }
        }
        ++n_seg;
      }
      if (!ok) {
        // every MMA issued so far must finish before TMEM is released
        ptx::mma_commit(bar(C::B_FIN));
        drain_bar(bar(C::B_FIN), 0);
      }
    }
    if (warp == 1) {
      // ================================================================ lookups
      // Per unit: {group, row tile, 1 for drafted tokens, KV head} and the page and (keys | chunk of the page <<
      // 16) of both chunks.  Batch f replaces batch f - 3, which everyone has left once the K loaders have begun
      // batch f - 1: the other warps are at most four units behind them.
      const int nu = x1 - x0;
      for (int f = 0; f * kBatch < nu; ++f) {
        if (f >= 2 && !wait_warp(C::B_UG, f & 1)) break;
        const int u = f * kBatch + lane;
        if (u < nu) {
          const int x = x0 + u;
          int lo = 0, hi = groups - 1;
          while (lo < hi) {  // the last group with pre <= x
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= x) lo = mid;
            else hi = mid - 1;
          }
          const int b = lo / a.c.hkv;
          // three rounds of memory: these three together, the list's entries, the table's
          const int listed = a.kv_cnt == nullptr ? INT32_MAX : __ldg(a.kv_cnt + lo);
          const int n = cached_of(a, b);
          const Drafts dr = drafts_of(a, b);
          const int pages = (n + a.c.page - 1) >> a.c.page_shift;
          const int cpp = a.c.page / kChunk, kept = max(0, min(listed, pages));
          const int chunks = a.kv_cnt == nullptr ? (n + kChunk - 1) / kChunk : kept * cpp;
          const int cu = (chunks + 1) / 2, per = cu + (dr.len + kUnit - 1) / kUnit;
          const int rt = (x - pre[lo]) / per, k = x - pre[lo] - rt * per;
          int page[2] = {0, 0}, w[2] = {0, 0};
          const int draft = k >= cu ? 1 : 0;
          if (draft) {
#pragma unroll
            for (int h = 0; h < 2; ++h) w[h] = max(0, min(kChunk, dr.len - (k - cu) * kUnit - h * kChunk)) | (k - cu) << 16;
          } else {
            int j[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = (2 * k + h) >> (a.c.page_shift - 6);
              j[h] = e >= kept ? INT32_MAX : a.kv_idx == nullptr ? e : __ldg(a.kv_idx + static_cast<size_t>(lo) * a.table_stride + e);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (j[h] >= 0 && j[h] < pages) {
                const int sub = (2 * k + h) & (cpp - 1);
                const int pg = __ldg(a.table + static_cast<size_t>(b) * a.table_stride + j[h]);
                if (pg >= 0 && pg < a.c.pages) {
                  page[h] = pg;
                  w[h] = max(0, min(kChunk, n - j[h] * a.c.page - sub * kChunk)) | sub << 16;
                } else if (a.status != nullptr) {
                  atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
                }
              } else if (j[h] < 0 && a.status != nullptr) {
                atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
              }
            }
          }
          int4 *rec = unit + 2 * (u % (kLists * kBatch));
          rec[0] = make_int4(lo, rt, draft, lo - b * a.c.hkv);
          rec[1] = make_int4(page[0], w[0], page[1], w[1]);
        }
        arrive_warp(C::B_UN + f % kLists);
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    // ================================================================ loaders
    ptx::setmaxnreg_dec<kRegLoad>();
    const int kv = (warp - 4) >> 2;       // 0: K, 1: V
    const int lt = (tid - 128) & 127;     // thread of the four warps
    const int lw = warp - 4;
    const int nu = x1 - x0;
    const uint8_t *codes = kv == 0 ? a.k_codes : a.v_codes, *scales = kv == 0 ? a.k_scales : a.v_scales;
    uint32_t four_phase = 0;
    auto sync_four = [&]() -> bool {  // the four warps; bounded, unlike a named barrier
      arrive_warp(C::B_LK + kv);
      return wait_warp(C::B_LK + kv, four_phase++ & 1);
    };

    // ---- codes of a unit: thread (p, r0) of the four warps takes piece p of the rows r0 + STEP * i, those of a
    // chunk together, in groups of two pieces.  A thread reads back only what it has copied itself.
    constexpr int NP = C::NP, STEP = Q16 ? 128 / NP : 1, GRP = C::GRP, NG = C::NG;
    // (the group scales sit in registers, which wants constant indices)
    constexpr int UNROLL = FMT == BSA_CACHE_E2M1 ? NG : 1;
    const int p = lt % C::PP, r0 = lt / C::PP;
    const uint32_t ring = C::OFF_CODE + static_cast<uint32_t>(tid - 128) * 16;  // slots of 256 pieces
    struct {             // the group to be copied next
      int unit, group;   // its unit and place there
      const uint8_t *code[2];  // the thread's first piece of both chunks of the unit
      int n[2];          // keys of the chunks
    } next;
    next.unit = 0;
    next.group = 0;
    next.code[0] = next.code[1] = codes;
    next.n[0] = next.n[1] = 0;
    // Copies the next group of the run into ring slot `slot` (zeros for absent rows), as one cp.async group.
    auto copy_group = [&](int slot) {
      if constexpr (Q16) {
        if (next.unit < nu) {
          if (next.group == 0) {
            const int4 d0 = unit[2 * (next.unit % (kLists * kBatch))], d1 = unit[2 * (next.unit % (kLists * kBatch)) + 1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int pg = h == 0 ? d1.x : d1.z, w = h == 0 ? d1.y : d1.w;
              next.n[h] = d0.z ? -1 : w & 0xFFFF;
              next.code[h] = codes + ((static_cast<size_t>(pg) * a.c.hkv + d0.w) * a.c.page + (w >> 16) * kChunk + r0) *
                                         C::RB + p * 16;
            }
          }
          if (next.n[0] >= 0) {  // (drafted tokens have no codes)
#pragma unroll
            for (int e = 0; e < GRP; ++e) {
              // a group of an NG > 1 unit lies in one chunk, one of an NG == 1 unit in both
              const int h = NG > 1 ? (next.group >= NG / 2 ? 1 : 0) : (e >= GRP / 2 ? 1 : 0);
              const int i = NG > 1 ? (next.group % (NG > 1 ? NG / 2 : 1)) * GRP + e : e % (GRP / 2);
              const uint8_t *from = (h == 0 ? next.code[0] : next.code[1]) + i * (STEP * C::RB);
              const int live = r0 + STEP * i < (h == 0 ? next.n[0] : next.n[1]) ? 16 : 0;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + ring + (slot * GRP + e) * 4096u),
                           "l"(from), "r"(live)
                           : "memory");
            }
          }
          if (++next.group == NG) next.group = 0, ++next.unit;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
    };
    // exponents of the rows 4 lane .. + 3 of this unit and the next; of the next also which bytes are there
    // (applied only when they are used: it would wait for the load)
    uint32_t ew = 0u, ew_next = 0u, ew_mask = 0u;
    uint16_t gw[FMT == BSA_CACHE_E2M1 ? NP : 1], gw_next[FMT == BSA_CACHE_E2M1 ? NP : 1];  // group scales of the pieces
    auto fetch_scales = [&](int u) {
      if constexpr (Q16) {
        const int4 d0 = unit[2 * (u % (kLists * kBatch))], d1 = unit[2 * (u % (kLists * kBatch)) + 1];
        {
          const int pg = lane < 16 ? d1.x : d1.z, w = lane < 16 ? d1.y : d1.w;
          const int rr = 4 * (lane & 15), live = (d0.z ? 0 : w & 0xFFFF) - rr;
          const uint8_t *sc = scales + (static_cast<size_t>(pg) * a.c.hkv + d0.w) * a.c.page * C::PER;
          ew_mask = live >= 4 ? 0xffffffffu : live <= 0 ? 0u : (1u << (8 * live)) - 1u;
          ew_next = 0u;
          if (live > 0) ew_next = __ldg(reinterpret_cast<const uint32_t *>(sc + (w >> 16) * kChunk + rr));
        }
        if constexpr (FMT == BSA_CACHE_E2M1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pg = h == 0 ? d1.x : d1.z, w = h == 0 ? d1.y : d1.w;
            const int row = (w >> 16) * kChunk, n = d0.z ? 0 : w & 0xFFFF;
            const uint8_t *sc = scales + (static_cast<size_t>(pg) * a.c.hkv + d0.w) * a.c.page * C::PER;
#pragma unroll
            for (int i = 0; i < NP / 2; ++i) {
              const int rr = r0 + STEP * i;
              gw_next[h * (NP / 2) + i] =
                  rr < n ? __ldg(reinterpret_cast<const uint16_t *>(sc + a.c.page + (row + rr) * (D / 16) + 2 * p)) : 0;
            }
          }
        }
      }
    };
    auto top_byte = [&](uint32_t w) -> int {
      const uint32_t m = __vmaxu4(w, w >> 16);
      return static_cast<int>(__reduce_max_sync(0xffffffffu, max(m & 0xFFu, (m >> 8) & 0xFFu)));
    };
    int slot = 0;  // ring slot of the group to be read next
    // The unit's codes into the f16 tile at offset `dst`, rows scaled against `ref`; refills the ring.
    auto convert = [&](uint32_t dst, int ref) {
      if constexpr (Q16) {
        // f16 factors of this lane's rows 4 lane .. + 3 (an absent row has exponent 0 and zero codes)
        auto factor = [&](int x) { return pow2_f16x2(static_cast<int>((ew >> (8 * x)) & 0xFFu) - ref + C::SHV); };
        const uint32_t f01 = __byte_perm(factor(0), factor(1), 0x5410), f23 = __byte_perm(factor(2), factor(3), 0x5410);
        const bool upper = (r0 & 2) != 0;                      // STEP is a multiple of 8: the same for every i
        const uint32_t pick = (r0 & 1) ? 0x3232u : 0x1010u;
#pragma unroll(UNROLL)
        for (int gr = 0; gr < NG; ++gr) {
          asm volatile("cp.async.wait_group %0;" ::"n"(C::RING - 1) : "memory");
          uint4 cw[GRP];
          uint32_t fs[GRP];
#pragma unroll
          for (int e = 0; e < GRP; ++e) {
            cw[e] = *reinterpret_cast<const uint4 *>(sb + ring + (slot * GRP + e) * 4096);
            const int from = ((r0 + STEP * (gr * GRP + e)) >> 2) & 31;
            const uint32_t fa = __shfl_sync(0xffffffffu, f01, from), fb = __shfl_sync(0xffffffffu, f23, from);
            fs[e] = __byte_perm(upper ? fb : fa, 0u, pick);
          }
#pragma unroll
          for (int e = 0; e < GRP; ++e) {
            const uint32_t w[4] = {cw[e].x, cw[e].y, cw[e].z, cw[e].w};
            const uint32_t at = dst + static_cast<uint32_t>(r0 + STEP * (gr * GRP + e)) * 128;
            auto put = [&](int c, int u, uint4 v) {  // unit u of swizzle chunk c
              put16(at + static_cast<uint32_t>(c) * C::CHUNK + static_cast<uint32_t>((u ^ (r0 & 7)) * 16), v);
            };
            if constexpr (FMT == BSA_CACHE_E4M3) {
              uint32_t h[8];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                h[2 * x] = mul_f16x2(e4m3x2_f16(w[x]), fs[e]);
                h[2 * x + 1] = mul_f16x2(e4m3x2_f16(w[x] >> 16), fs[e]);
              }
              const uint4 s0 = make_uint4(h[0], h[1], h[2], h[3]), s1 = make_uint4(h[4], h[5], h[6], h[7]);
              // the upper pieces store their halves in the other order: no two lanes meet in a bank
              const int u = 2 * (p & 3), sw = (p >> 2) & 1;
              put(p >> 2, u + sw, sw ? s1 : s0);
              put(p >> 2, u + 1 - sw, sw ? s0 : s1);
            } else {
              const uint32_t g2 = mul_f16x2(e4m3x2_f16(gw[gr * GRP + e]), fs[e]);
              const uint32_t ga = __byte_perm(g2, g2, 0x1010), gb = __byte_perm(g2, g2, 0x3232);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t gs = x < 2 ? ga : gb;
                put(p >> 1, 4 * (p & 1) + x,
                    make_uint4(mul_f16x2(e2m1x2_f16(w[x]), gs), mul_f16x2(e2m1x2_f16(w[x] >> 8), gs),
                               mul_f16x2(e2m1x2_f16(w[x] >> 16), gs), mul_f16x2(e2m1x2_f16(w[x] >> 24), gs)));
              }
            }
          }
          copy_group(slot);
          slot = slot == C::RING - 1 ? 0 : slot + 1;
        }
      }
    };
    // bf16 rows by hand: `n` keys of chunk h, from `from` (row stride in elements); zeros past n, and with `clean`
    // in place of Inf and NaN.  Not 0 if there were any.  (Four pieces in flight: eight leave the codec
    // spilling, 278 against 243 us for 64 drafts over e4m3.)
    auto store_rows = [&](uint32_t dst, int h, const uint16_t *from, size_t stride, int n, float f, bool clean) -> uint32_t {
      uint32_t lost = 0u;
      constexpr int PR = D / 8, TOTAL = kChunk * PR / 128, U = 4;
#pragma unroll 1
      for (int b = 0; b < TOTAL; b += U) {
        uint4 v[U];
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int x = (b + e) * 128 + lt;
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (x / PR < n) v[e] = __ldg(reinterpret_cast<const uint4 *>(from + (x / PR) * stride + (x % PR) * 8));
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int x = (b + e) * 128 + lt;
          if (clean) v[e] = finite_bf16x8(v[e], lost);
          if constexpr (Q16) {
            uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = pack_f16x2(__uint_as_float(w[q] << 16) * f, __uint_as_float(w[q] & 0xFFFF0000u) * f);
            v[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          put16(swizzled(dst, (x % PR) >> 3, h * kChunk + x / PR, x % PR & 7), v[e]);
        }
      }
      return lost;
    };
    // the exponent reference of a unit of drafted rows: its largest finite element lands in [2^14, 2^15)
    auto draft_ref = [&](const uint16_t *from, size_t stride, int n, bool &ok) -> int {
      constexpr int PR = D / 8;
      float am = 0.f;
      uint32_t lost = 0u;
#pragma unroll 2
      for (int x = lt; x < n * PR; x += 128)
        am = fmaxf(am, amax8(finite_bf16x8(__ldg(reinterpret_cast<const uint4 *>(from + (x / PR) * stride + (x % PR) * 8)), lost)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      if (lane == 0) red[lw] = am;
      if (!(ok = sync_four())) return 8;
      am = fmaxf(fmaxf(red[4 * kv], red[4 * kv + 1]), fmaxf(red[4 * kv + 2], red[4 * kv + 3]));
      ok = sync_four();
      return max(8, (__float_as_int(am) >> 23) + C::SHV - 14);
    };

    // the records of the batch that begins with unit u
    auto looked_up = [&](int u) -> bool { return wait_warp(C::B_UN + u / kBatch % kLists, (u / kBatch / kLists) & 1); };
    bool ok = nu == 0 || looked_up(0);
    if (Q16 && ok && nu > 0) {
      for (int x = 0; x < C::RING; ++x) copy_group(x);
      fetch_scales(0);
    }
    constexpr int AHEAD = Q16 ? (NG - 1 + C::RING) / NG : 1;  // the furthest unit met while one is filled
    int seg_group = -1, seg_tile = -1, oref = 0;
    uint32_t copies = 0;  // units whose TMA copies were issued
    const int stages = kv == 0 ? C::KS : C::VS;
    int st = -1, round = -1;  // stage of the unit, and times the stage was filled before
    for (int n = 0; ok && n < nu; ++n) {
      const int4 d0 = unit[2 * (n % (kLists * kBatch))], d1 = unit[2 * (n % (kLists * kBatch)) + 1];
      const int g = d0.w;
      if (d0.x != seg_group || d0.y != seg_tile) seg_group = d0.x, seg_tile = d0.y, oref = 0;  // a new segment
      if (kv == 0 && n > 0 && n % kBatch == 0) arrive_warp(C::B_UG);
      if ((n + AHEAD) % kBatch == 0 && n + AHEAD < nu && !(ok = looked_up(n + AHEAD))) break;

      // ---- the unit's scales
      const size_t dstride = static_cast<size_t>(a.c.hkv) * D;
      const int n0 = d1.y & 0xFFFF, n1 = d1.w & 0xFFFF;
      const uint16_t *drafted = kv == 0 ? a.k_new : a.v_new;
      if (d0.z) drafted += ((static_cast<size_t>(drafts_of(a, d0.x / a.c.hkv).start) + (d1.y >> 16) * kUnit) * a.c.hkv + g) * D;
      int ref = 0;
      if constexpr (Q16) {
        ew = ew_next & ew_mask;
        if constexpr (FMT == BSA_CACHE_E2M1) {
#pragma unroll
          for (int i = 0; i < NP; ++i) gw[i] = gw_next[i];
        }
        if (d0.z) {
          ref = draft_ref(drafted, dstride, n0 + n1, ok);
          if (!ok) break;
        } else {
          ref = top_byte(ew);
        }
        if (kv == 0) {
          if (lt == 0) info_k[n % kInfo] = exp2f(static_cast<float>(ref - C::SHV - 127));
        } else {
          ref = oref = max(oref, ref);
          if (lt == 0) info_v[n % kInfo] = oref;
        }
        if (n + 1 < nu) fetch_scales(n + 1);
      }
      arrive_warp((kv == 0 ? C::B_IK : C::B_IV) + n % kInfo);

      // ---- wait for the stage and fill it
      if (st + 1 == stages || st < 0) st = 0, ++round;
      else ++st;
      const int full = (kv == 0 ? C::B_KF : C::B_VF) + st, empty = (kv == 0 ? C::B_KE : C::B_VE) + st;
      const uint32_t tile = (kv == 0 ? C::OFF_K : C::OFF_V) + st * C::TILE;
      if (round > 0 && !(ok = wait_warp(empty, (round - 1) & 1))) break;
      // bf16: whole chunks by TMA, at once (one box of 128 rows where a page holds both chunks); a chunk with
      // absent rows by hand below, with zeros for them
      uint32_t by_tma = 0;  // bit h: chunk h
      if constexpr (!Q16) {
        if (!d0.z) by_tma = (n0 == kChunk ? 1u : 0u) | (n1 == kChunk ? 2u : 0u);
        if (a.c.page >= kUnit && by_tma != 3) by_tma = 0;
        if ((lw & 3) == 0 && by_tma != 0) {
          // (announced without arriving: this warp may still have rows of the other chunk to write)
          if (lane == 0) mbar_expect_tx(bar(full), (by_tma == 3 ? 2u : 1u) * (C::TILE / 2));
          __syncwarp();
          const int c = lane >> 1, h = lane & 1;  // a lane for every copy
          const bool mine = c < C::NCH && (by_tma >> h & 1) && (h == 0 || a.c.page < kUnit);
          if (mine)
            tma_load_3d(base + tile + c * C::CHUNK + h * (kChunk * 128), kv == 0 ? &tm_k : &tm_v, bar(full), c * 64,
                        ((h == 0 ? d1.y : d1.w) >> 16) * kChunk, (h == 0 ? d1.x : d1.z) * a.c.hkv + g);
          __syncwarp();
          copies = n + 1;
        }
      }
      if (d0.z) {
        const float f = Q16 ? pow2_biased(254 + C::SHV - ref) : 1.f;
        uint32_t lost = store_rows(tile, 0, drafted, dstride, n0, f, kv == 1);
        lost |= store_rows(tile, 1, drafted + kChunk * dstride, dstride, n1, f, kv == 1);
        if (kv == 1) {
          // read behind B_OD, whose issuing thread has waited for this stage of V
          const bool any = __any_sync(0xffffffffu, lost != 0u);
          if (lane == 0) reinterpret_cast<uint8_t *>(lost_v + n % kInfo)[lw & 3] = any;
        }
        for (int gr = 0; Q16 && gr < NG; ++gr) {  // the unit's empty groups
          copy_group(slot);
          slot = slot == C::RING - 1 ? 0 : slot + 1;
        }
      } else if constexpr (Q16) {
        convert(tile, ref);
      } else {
        if (by_tma != 3) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (by_tma >> h & 1) continue;
            const int nh = h == 0 ? n0 : n1, pg = h == 0 ? d1.x : d1.z, sub = (h == 0 ? d1.y : d1.w) >> 16;
            const size_t row = (static_cast<size_t>(pg) * a.c.hkv + g) * a.c.page + sub * kChunk;
            store_rows(tile, h, reinterpret_cast<const uint16_t *>(codes) + row * D, D, nh, 1.f, false);
          }
        }
      }
      if (by_tma != 3) ptx::fence_proxy_async_smem();  // what was written by hand
      arrive_warp(full);
    }
    if (Q16) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!Q16 && *abort_flag && (lw & 3) == 0 && lane == 0) {
      // let copies in flight land before the CTA's shared memory is released
      const uint32_t last = static_cast<uint32_t>(stages);
      for (uint32_t n = copies > last ? copies - last : 0; n < copies; ++n)
        drain_bar(bar((kv == 0 ? C::B_KF : C::B_VF) + n % last), (n / last) & 1);
    }
    __syncwarp();
  } else {
    // ================================================================ softmax lanes
    ptx::setmaxnreg_inc<kRegSoft>();
    const int t = (warp - 12) >> 2;
    const int sub = warp & 3;
    const int r = (sub << 5) + lane;  // query row = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(sub << 5) << 16;
    const uint32_t tS = tmem + lane_off + t * 128, tO = tmem + lane_off + C::TM_O + t * 128;
    // A segment's rows of Q, this warp's part of them: its own rows, or half of them where both lanes have the
    // same rows.  The lane has seen the last S of the segment before (of both lanes: B_QE).
    auto load_q = [&](const Segment &s, uint32_t seg) {
      constexpr int LPR = D / 8, R = 32 / LPR, ROWS = PAIR ? 32 : 16;  // lanes of a row, rows of a step, of the warp
      constexpr int U = ROWS / R < 8 ? ROWS / R : 8;                   // steps in flight
      const Drafts dr = drafts_of(a, s.grp / a.c.hkv);
      const int q = lane % LPR, first = PAIR ? t * kRows + sub * 32 : sub * 32 + t * 16, g = s.grp % a.c.hkv;
#pragma unroll 1
      for (int r = first; r < first + ROWS; r += R * U) {
        uint4 v[U];
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int row = s.rt * C::NTQ * kRows + r + e * R + lane / LPR, tok = row / G;
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (tok < dr.len)
            v[e] = __ldg(reinterpret_cast<const uint4 *>(
                a.q + (static_cast<size_t>(dr.start + tok) * a.hq + g * G + row % G) * D + q * 8));
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int rr = r + e * R + lane / LPR;
          if constexpr (Q16) {
            float am = amax8(v[e]);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            const int ex = max(1, min(253, 268 - (__float_as_int(am) >> 23)));
            const float f = pow2_biased(ex);
            if (q == 0) row_scale[(seg & 1) * C::NTQ * 128 + rr] = pow2_biased(254 - ex);
            uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
            for (int x = 0; x < 4; ++x)
              w[x] = pack_f16x2(__uint_as_float(w[x] << 16) * f, __uint_as_float(w[x] & 0xFFFF0000u) * f);
            v[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          put16(swizzled(C::OFF_Q + (rr >> 7) * C::TILE, q >> 3, rr & 127, q & 7), v[e]);
        }
      }
      ptx::fence_proxy_async_smem();
      arrive_warp(C::B_QF + t);
      if constexpr (Q16 && !PAIR) arrive_warp(C::B_RS + (seg & 1));
    };
    bool ok = true;
    uint32_t n = 0, mine = 0, n_seg = 0, lane_segs = 0;  // units of the run, of this lane; segments
    Segment s{};
    if (x0 < x1) {
      s = segment_at<C::NTQ>(a, pre, groups, x0, x1);
      load_q(s, 0);
    }
    for (int x = x0; ok && x < x1; ++n_seg) {
      if (n_seg > 0) s = segment_at<C::NTQ>(a, pre, groups, x, x1);
      x += s.units;
      const Drafts dr = drafts_of(a, s.grp / a.c.hkv);
      const int row = (s.rt * C::NTQ + (PAIR ? t : 0)) * kRows + r, tok = row / G;
      const bool live = tok < dr.len;
      float rs = a.scale_log2;
      if constexpr (Q16) {
        if (!PAIR && !(ok = wait_warp(C::B_RS + (n_seg & 1), (n_seg >> 1) & 1))) break;
        rs *= row_scale[((n_seg & 1) * C::NTQ + (PAIR ? t : 0)) * 128 + r];
      }
      float m = -INFINITY, l = 0.f;
      int oref = 0;  // O's unit (8- and 4-bit caches)
      int done = 0;  // units of this lane in the segment
      for (int i = 0; i < s.units; ++i, ++n) {
        if (n % kBatch == 0 && !(ok = wait_warp(C::B_UN + n / kBatch % kLists, (n / kBatch / kLists) & 1))) break;
        if (!(ok = wait_warp(C::B_IK + n % kInfo, (n / kInfo) & 1))) break;
        if (!(ok = wait_warp(C::B_IV + n % kInfo, (n / kInfo) & 1))) break;
        if (!PAIR && (i & 1) != t) continue;
        const int4 d0 = unit[2 * (n % (kLists * kBatch))], d1 = unit[2 * (n % (kLists * kBatch)) + 1];
        const int n0 = d1.y & 0xFFFF, n1 = d1.w & 0xFFFF;
        float scl = rs;
        int oref_new = 0;
        if constexpr (Q16) {
          // never 0, so that a masked -inf stays one (the logits below it are 0 to any precision)
          scl = fmaxf(scl * info_k[n % kInfo], 1e-37f);
          oref_new = info_v[n % kInfo];
        }
        // which of the unit's keys the row sees
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        const bool partial = d0.z != 0 || n0 < kChunk || n1 < kChunk;
        if (partial) {
          if (d0.z) {
            const int first = (d1.y >> 16) * kUnit;
            vis[0] = vis[1] = vis[2] = vis[3] = 0u;
            if (live)
              for (int p = tok; p >= 0; p = parent_of(a, dr.start, p)) {
                const int k = p - first;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  if (k >> 5 == w) vis[w] |= 1u << (k & 31);
              }
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int k = (w < 2 ? n0 : n1) - 32 * (w & 1);
              vis[w] = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
            }
          }
        }
        if (!(ok = wait_warp(C::B_SF + t, mine & 1))) break;
        ptx::tc_fence_after();
        // the row's maximum first, keeping the first 64 logits only: what follows is a loop over halves, whose
        // code the instruction cache holds
        uint32_t sr[2][32];
        float pm[4];
        if (partial) {
          pm[1] = pm[2] = pm[3] = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            ptx::tmem_ld32(tS + c * 32, sr[0]);
            ptx::tmem_wait_ld();
            const uint32_t seen = c < 2 ? (c == 0 ? vis[0] : vis[1]) : (c == 2 ? vis[2] : vis[3]);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((seen >> e) & 1u) pm[1] = fmaxf(pm[1], __uint_as_float(sr[0][e]));
          }
        } else {
          ptx::tmem_ld32_max(tS + 64, sr[0], pm[2]);
          ptx::tmem_ld32_max(tS + 96, sr[1], pm[3]);
          ptx::tmem_wait_ld();
        }
        float first[2];
        ptx::tmem_ld32_max(tS, sr[0], first[0]);
        ptx::tmem_ld32_max(tS + 32, sr[1], first[1]);
        ptx::tmem_wait_ld();
        pm[0] = partial ? pm[1] : first[0];
        pm[1] = partial ? pm[1] : first[1];
        const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
        const float mt = mx == -INFINITY ? -INFINITY : mx * scl;
        // O moves to a new reference or a larger unit only when it has to
        float factor = 1.f;
        if (mt > m + static_cast<float>(C::TH)) {
          factor = m == -INFINITY ? 0.f : ptx::ex2_approx(m - mt);
          m = mt;
        }
        float of = factor;
        if constexpr (Q16) {
          if (oref_new != oref) {  // (the reference only grows)
            of *= pow2_biased(127 + oref - oref_new);
            oref = oref_new;
          }
        }
        const bool resc = done > 0 && of != 1.f;
        const float mb = m == -INFINITY ? 0.f : m;
        const float bias = static_cast<float>(C::SHIFT) - mb;
        uint64_t acc[2] = {0ull, 0ull};
        const uint64_t scl2 = ptx::f32x2(scl, scl), bias2 = ptx::f32x2(bias, bias);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (half == 1) ptx::tmem_wait_ld();
          if (partial) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t seen = half == 0 ? vis[c] : vis[2 + c];
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((seen >> e) & 1u)) sr[c][e] = 0xFF800000u;
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t y = ptx::fma_f32x2(
                  ptx::f32x2(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1])), scl2, bias2);
              float y0, y1;
              ptx::f32x2_split(y, y0, y1);
              const float p0 = ptx::ex2_approx(y0), p1 = ptx::ex2_approx(y1);
              acc[e & 1] = ptx::add_f32x2(acc[e & 1], ptx::f32x2(p0, p1));
              pk[e] = Q16 ? pack_f16x2(p0, p1) : ptx::pack_bf16x2(p0, p1);
            }
            ptx::tmem_st16(tS + half * 32 + c * 16, pk);  // over logits that have been read
            if (c == 0 && half == 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
              for (int q = 0; q < D / 8; ++q) {
                uint32_t ov[8];
                ptx::tmem_ld8(tO + q * 8, ov);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * of);
                ptx::tmem_st8(tO + q * 8, ov);
              }
            }
            if (half == 0) ptx::tmem_ld32(tS + 64 + c * 32, sr[c]);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          arrive_warp(C::B_PR + t * C::NPC + half);
        }
        float s4[4];
        ptx::f32x2_split(acc[0], s4[0], s4[1]);
        ptx::f32x2_split(acc[1], s4[2], s4[3]);
        constexpr float unshift = 1.f / (1 << C::SHIFT);
        l = fmaf((s4[0] + s4[1]) + (s4[2] + s4[3]), unshift, l * factor);
        ++mine;
        ++done;
      }
      if (!ok) break;
      if (x < x1) {  // the next segment's rows, so that its first products run beside what follows
        if (!PAIR && !(ok = wait_warp(C::B_QE, n_seg & 1))) break;
        load_q(segment_at<C::NTQ>(a, pre, groups, x, x1), n_seg + 1);
      }

      // ---- the segment's result of this lane: rows to the output, or a part for the combine
      if (done > 0) {
        if (!(ok = wait_warp(C::B_OD + t, lane_segs & 1))) break;
        ptx::tc_fence_after();
        ++lane_segs;
      }
      // whether the segment's drafted values (its last units, two at most) held Inf or NaN; kInfo units are kept
      bool lost = false;
      for (int i = max(0, s.units - 2); i < s.units; ++i) {
        const uint32_t u = n - static_cast<uint32_t>(s.units - i);
        if ((PAIR || (i & 1) == t) && unit[2 * (u % (kLists * kBatch))].z != 0) lost |= lost_v[u % kInfo] != 0u;
      }
      if (lost) {  // warp-uniform; those that the row sees, into O
        const uint16_t *vn = a.v_new + (static_cast<size_t>(dr.start) * a.c.hkv + s.grp % a.c.hkv) * D;
#pragma unroll 1
        for (int q = 0; q < D / 8; ++q) {
          uint32_t ov[8];
          ptx::tmem_ld8(tO + q * 8, ov);
          ptx::tmem_wait_ld();
          if (live)
            for (int p = tok; p >= 0; p = parent_of(a, dr.start, p)) {
              const uint4 u = __ldg(reinterpret_cast<const uint4 *>(vn + static_cast<size_t>(p) * a.c.hkv * D + q * 8));
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 8; ++e)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) + not_finite(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu));
            }
          __syncwarp();
          ptx::tmem_st8(tO + q * 8, ov);
        }
        ptx::tmem_wait_st();
      }
      m = ptx::part_max(m, l);
      const bool whole = s.rs >= x0 && s.re <= x1;
      const size_t slot = (2 * static_cast<size_t>(cta) + (s.rs <= x0 ? 0 : 1)) * C::NTQ + (PAIR ? t : 0);
      float unit_f = 1.f;
      if constexpr (Q16) unit_f = exp2f(static_cast<float>(oref - 127 - C::SHV - C::SHIFT));
      float4 *mine_o = reinterpret_cast<float4 *>(lane_o) + static_cast<size_t>(cta) * (D / 4 + 1) * kRows;
      float other_f = 0.f;
      if constexpr (!PAIR) {
        // lane 1 hands its rows to lane 0 through this CTA's scratch
        if (t == 1) {
          if (n_seg > 0 && !(ok = wait_warp(C::B_LB, (n_seg - 1) & 1))) break;  // the last one has been read
          if (done > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              ptx::tmem_ld32(tO + c * 32, ov);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                mine_o[(c * 8 + e) * kRows + r] =
                    make_float4(__uint_as_float(ov[4 * e]) * unit_f, __uint_as_float(ov[4 * e + 1]) * unit_f,
                                __uint_as_float(ov[4 * e + 2]) * unit_f, __uint_as_float(ov[4 * e + 3]) * unit_f);
            }
          }
          mine_o[D / 4 * kRows + r] = make_float4(m, l, done > 0 ? 1.f : 0.f, 0.f);
          ptx::tc_fence_before();
          if (done > 0) arrive_warp(C::B_OE + t);
          arrive_warp(C::B_LA);
          continue;
        }
        if (!(ok = wait_warp(C::B_LA, n_seg & 1))) break;
        const float4 ml = mine_o[D / 4 * kRows + r];
        if (ml.z != 0.f && ml.x != -INFINITY) {
          const float mm = ptx::max_nan(m, ml.x);
          const float f0 = m == -INFINITY ? 0.f : ptx::ex2_approx(m - mm);
          other_f = ptx::ex2_approx(ml.x - mm);
          l = l * f0 + ml.y * other_f;
          unit_f *= f0;
          m = mm;
        }
      }
      const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;  // (NaN where the sum is)
      const size_t out = static_cast<size_t>(dr.start + tok) * a.hq + (s.grp % a.c.hkv) * G + row % G;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        ptx::tmem_ld32(tO + c * 32, ov);
        ptx::tmem_wait_ld();
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(ov[e]) * unit_f;
        if constexpr (!PAIR) {
          if (other_f != 0.f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = mine_o[(c * 8 + e) * kRows + r];
              f[4 * e] = fmaf(v.x, other_f, f[4 * e]);
              f[4 * e + 1] = fmaf(v.y, other_f, f[4 * e + 1]);
              f[4 * e + 2] = fmaf(v.z, other_f, f[4 * e + 2]);
              f[4 * e + 3] = fmaf(v.w, other_f, f[4 * e + 3]);
            }
          }
        }
        if (whole) {
          if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4 *>(a.o + out * D + c * 32 + e * 8) =
                  make_uint4(ptx::pack_bf16x2(f[8 * e] * inv, f[8 * e + 1] * inv),
                             ptx::pack_bf16x2(f[8 * e + 2] * inv, f[8 * e + 3] * inv),
                             ptx::pack_bf16x2(f[8 * e + 4] * inv, f[8 * e + 5] * inv),
                             ptx::pack_bf16x2(f[8 * e + 6] * inv, f[8 * e + 7] * inv));
          }
        } else {
          float4 *po = reinterpret_cast<float4 *>(part_o) + slot * (D / 4) * kRows;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            po[(c * 8 + e) * kRows + r] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
        }
      }
      if (whole) {
        if (live && a.lse != nullptr) a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float2 *>(part_ml + (slot * kRows + r) * 2) = make_float2(m, l);
      }
      ptx::tc_fence_before();
      if (done > 0) arrive_warp(C::B_OE + t);
      if constexpr (!PAIR) arrive_warp(C::B_LB);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag && a.status != nullptr)
    atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_DEVICE_TIMEOUT));
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The row tiles that several CTAs share; CTA x takes the x-th of them (shared_tile), kCombineRows of its
// rows and kCombineDims dimensions.  Parts p = c - 1 .. are spread over the warps (warp w takes w, w + 8, ..),
// a lane is a row; O = sum w_p O_p / sum w_p l_p, w_p = 2^(m_p - max m), the eight sums added in order.
constexpr int kCombineRows = 32, kCombineDims = 16, kCombineWarps = 8;

template <int D, bool PAIR>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_mma_combine_kernel(const TreeArgs a, const float *part_o,
                                                                             const float *part_ml, const TreeRun *runs) {
  constexpr int NTQ = PAIR ? 2 : 1, NQ = kCombineDims / 4, U = 2;
  after_previous_kernel();
  __shared__ float red_m[kCombineWarps][32], red_l[kCombineWarps][32];
  __shared__ float4 red_o[kCombineWarps][NQ][32];
  TreeRun run;
  const int c = shared_tile(runs, kSms, blockIdx.x, &run);
  if (c < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int BLOCKS = kRows / kCombineRows;
  const int t = blockIdx.z / BLOCKS, r = (blockIdx.z % BLOCKS) * kCombineRows + lane, q0 = blockIdx.y * NQ;
  const int row = (run.tile * NTQ + t) * kRows + r, tok = row / a.group;
  if ((row - lane) / a.group >= run.drafts) return;  // no row of the block is there
  const int p0 = c - 1, np = (run.last - 1) / run.run - p0 + 1;
  // every part after the first begins its CTA's run; the first may be that CTA's last tile
  auto slot = [&](int p) { return (2 * static_cast<size_t>(p0 + p) + (p > 0 || run.first == p0 * run.run ? 0 : 1)) * NTQ + t; };
  // each warp with its own running maximum
  float m = -INFINITY, l = 0.f;
  float4 acc[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int pb = warp; pb < np; pb += U * kCombineWarps) {
    float2 ml[U];
    float4 v[U][NQ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = pb + u * kCombineWarps;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (p < np) {
        ml[u] = *reinterpret_cast<const float2 *>(part_ml + (slot(p) * kRows + r) * 2);
#pragma unroll
        for (int q = 0; q < NQ; ++q)
          v[u][q] = reinterpret_cast<const float4 *>(part_o)[(slot(p) * (D / 4) + q0 + q) * kRows + r];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ml[u].x == -INFINITY) continue;
      const float mn = ptx::max_nan(m, ml[u].x);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(ml[u].x - mn);
      m = mn;
      l = fmaf(ml[u].y, w, l * f);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        acc[q].x = fmaf(v[u][q].x, w, acc[q].x * f);
        acc[q].y = fmaf(v[u][q].y, w, acc[q].y * f);
        acc[q].z = fmaf(v[u][q].z, w, acc[q].z * f);
        acc[q].w = fmaf(v[u][q].w, w, acc[q].w * f);
      }
    }
  }
  red_m[warp][lane] = m;
  red_l[warp][lane] = l;
#pragma unroll
  for (int q = 0; q < NQ; ++q) red_o[warp][q][lane] = acc[q];
  __syncthreads();
  if (warp >= NQ) return;  // warp q finishes dimensions 4 (q0 + q) ..
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) mm = ptx::max_nan(mm, red_m[w][lane]);
  float ls = 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) {
    if (red_m[w][lane] == -INFINITY) continue;
    const float f = exp2f(red_m[w][lane] - mm);
    ls = fmaf(red_l[w][lane], f, ls);
    const float4 v = red_o[w][warp][lane];
    s.x = fmaf(v.x, f, s.x);
    s.y = fmaf(v.y, f, s.y);
    s.z = fmaf(v.z, f, s.z);
    s.w = fmaf(v.w, f, s.w);
  }
  if (tok >= run.drafts) return;
  const float inv = ls == 0.f ? 0.f : 1.f / ls;
  const size_t out = static_cast<size_t>(run.draft0 + tok) * a.hq + (run.group % a.c.hkv) * a.group + row % a.group;
  *reinterpret_cast<uint2 *>(a.o + out * D + 4 * (q0 + warp)) =
      make_uint2(ptx::pack_bf16x2(s.x * inv, s.y * inv), ptx::pack_bf16x2(s.z * inv, s.w * inv));
  if (a.lse != nullptr && q0 + warp == 0) a.lse[out] = ls == 0.f ? -INFINITY : (mm + log2f(ls)) * 0.69314718055994531f;
}

struct Workspace {
  size_t part_o, part_ml, lane_o, runs, total;
};
Workspace workspace_layout(int d) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Workspace w;
  w.part_o = 0;  // two parts per CTA, up to two row tiles each
  w.part_ml = up(4ull * kSms * kRows * d * 4);
  w.lane_o = w.part_ml + up(4ull * kSms * kRows * 2 * 4);
  w.runs = w.lane_o + up(static_cast<size_t>(kSms) * kRows * (d + 4) * 4);
  w.total = w.runs + up(kSms * sizeof(TreeRun));
  return w;
}

template <int D, int FMT, bool PAIR>
bsa_status launch_t(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  using C = Cfg<D, FMT, PAIR>;
  CUtensorMap mk{}, mv{};
  if (!C::Q16) {
    cudaError_t e = cudaSuccess;
    EncodeTiledFn fn = tensor_map_encoder(&e);
    if (fn == nullptr || e != cudaSuccess || !chunk_map(fn, &mk, a.k_codes, a.c) || !chunk_map(fn, &mv, a.v_codes, a.c))
      return BSA_ERR_CUDA;
  }
  const Workspace ws = workspace_layout(D);
  char *base = static_cast<char *>(workspace);
  float *part_o = reinterpret_cast<float *>(base + ws.part_o), *part_ml = reinterpret_cast<float *>(base + ws.part_ml);
  float *lane_o = reinterpret_cast<float *>(base + ws.lane_o);
  TreeRun *runs = reinterpret_cast<TreeRun *>(base + ws.runs);
  auto kern = tree_mma_kernel<D, FMT, PAIR>;
  // setmaxnreg.inc waits until the registers it asks for are free: the split is only safe if the
  // kernel really launches with that many registers per thread
  static std::atomic<uint64_t> done{0};
  const cudaError_t ready = set_up(kern, kMaxSmem, kLaunchRegs, done);
  if (ready != cudaSuccess) return ready == cudaErrorNotSupported ? BSA_ERR_UNSUPPORTED : BSA_ERR_CUDA;
  const size_t smem = C::smem(a.batch * a.c.hkv);
  kern<<<kSms, kThreads, smem, stream>>>(mk, mv, a, part_o, part_ml, lane_o, runs);
  if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  const int rows = a.max_draft * a.group;
  const long long tiles = static_cast<long long>(a.batch) * a.c.hkv * ((rows + kRows * C::NTQ - 1) / (kRows * C::NTQ));
  const int shared = static_cast<int>(tiles < kSms - 1 ? tiles : kSms - 1);  // at most: a run boundary each
  const int most = rows < kRows * C::NTQ ? rows : kRows * C::NTQ;
  const dim3 grid(shared, D / kCombineDims, (most + kCombineRows - 1) / kCombineRows);
  const cudaError_t e = launch_after(tree_mma_combine_kernel<D, PAIR>, grid, kCombineWarps * 32, 0, stream, a,
                                     static_cast<const float *>(part_o), static_cast<const float *>(part_ml),
                                     static_cast<const TreeRun *>(runs));
  return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <int D, int FMT>
bsa_status launch_fmt(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  // two row tiles per unit halve the reads and conversions of the cache; the plan of very large batches
  // does not fit beside them in shared memory
  const bool pair = a.max_draft * a.group > kRows && Cfg<D, FMT, true>::smem(a.batch * a.c.hkv) <= kMaxSmem;
  return pair ? launch_t<D, FMT, true>(a, workspace, stream) : launch_t<D, FMT, false>(a, workspace, stream);
}

}  // namespace

size_t tree_mma_workspace_bytes(const CacheDims &c) { return workspace_layout(c.d).total; }

bsa_status launch_tree_mma(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  const bool wide = a.c.d == 128;
  switch (a.c.format) {
    case BSA_CACHE_E4M3:
      return wide ? launch_fmt<128, BSA_CACHE_E4M3>(a, workspace, stream) : launch_fmt<64, BSA_CACHE_E4M3>(a, workspace, stream);
    case BSA_CACHE_E2M1:
      return wide ? launch_fmt<128, BSA_CACHE_E2M1>(a, workspace, stream) : launch_fmt<64, BSA_CACHE_E2M1>(a, workspace, stream);
    default:
      return wide ? launch_fmt<128, BSA_CACHE_BF16>(a, workspace, stream) : launch_fmt<64, BSA_CACHE_BF16>(a, workspace, stream);
  }
}

}  // namespace bsa
