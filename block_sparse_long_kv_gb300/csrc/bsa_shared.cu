// Attention of sequences that share the first pages of their tables, the shared pages read once for all.
//
// softmax over the union of two sets of keys splits: with m, l and O the maximum, the sum of 2^(x - m) and the
// weighted values over each set, the union's are those of the sets brought to the larger maximum and added.  So the
// rows of all sequences of a group (drafted tokens x heads of a KV group) meet the shared pages together, in
// shared_kernel; each sequence's rows meet its own keys in the drafted-token kernels, which start first and hand over
// the SMs as they finish; shared_combine_kernel adds the two.
//
// shared_kernel.  128 rows are a tile of tcgen05 MMAs, 128 keys a unit.  The units of all (group, KV head, row tile)
// are laid end to end and cut into equal runs, one per CTA (one CTA per SM); a run crosses from one row tile into the
// next (segments).  Two lanes of eight softmax warps share the tensor core, so that one lane's exponentials run under
// the other's MMAs:
//   PAIR   (more than 128 rows a group)  the lanes hold two row tiles and the same keys
//   !PAIR  the lanes hold the same rows and take alternate units; both leave their results
// Two threads share a row, each with the 64 keys of one chunk, which is there as a whole or not at all: shared pages
// are full.  The issuing order S_0(n), P_1 V(n-1), S_1(n), P_0 V(n) keeps one tile's products under the other's
// softmax.  P lies over the first half of its own S columns.
// Warps:  0      looks pages up, publishes segments, issues the copies (bf16: TMA tiles; codes: bulk copies)
//         1      TMEM owner; one thread issues the MMAs
//         4-19   the softmax lanes
//         20-23  (8- and 4-bit caches) Q and the codes into f16 tiles
//
// An 8- or 4-bit cache is computed in f16, with the scales of the drafted-token kernel: with e the exponent of a
// key's row and kref the largest of the unit, K' = code * 2^(e - kref + SHV) is exact down to e = kref - 21 (E4M3) or
// kref - 18 (E2M1); 2^(kref - 127 - SHV) joins the logit scale.  V likewise against oref, the largest exponent of the
// segment so far, O being held in units of 2^(oref - 127 - SHV - SHIFT).  P' = 2^(x - m + SHIFT) with the reference m
// at most 2^TH below the true maximum, so P' <= 2^15.  Row sums are fp32 from unrounded values.
//
// Every mbarrier wait is bounded, as in the prefill kernel.
#include "bsa_tree_mma.cuh"

namespace bsa {
namespace {

constexpr int kSoftWarp = 4, kLoadWarp = 20;
constexpr int kSegs = 8;   // segments published ahead
constexpr int kUnits = 8;  // units whose records are kept

template <int D, int FMT, bool PAIR>
struct Shared {
  static constexpr bool Q16 = FMT != BSA_CACHE_BF16;
  static constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;
  static constexpr int THREADS = Q16 ? 768 : 640;
  static constexpr int LAUNCH_REGS = Q16 ? 80 : 96;
  static constexpr int REG_LOW = Q16 ? 40 : 56, REG_SOFT = Q16 ? 88 : 104, REG_LOAD = 88;
  static_assert(128 * REG_LOW + 512 * REG_SOFT + (Q16 ? 128 * REG_LOAD : 0) <= THREADS * LAUNCH_REGS, "register split");
  static constexpr int SHV = FMT == BSA_CACHE_E4M3 ? 6 : 4;  // 448 * 2^6 and 2688 * 2^4 stay below 2^16
  static constexpr int TH = Q16 ? 4 : 8;                     // log2 of how far the reference may lag the maximum
  static constexpr int SHIFT = Q16 ? 15 - TH : 0;
  static constexpr int NTQ = PAIR ? 2 : 1;
  static constexpr int NCH = D / 64;                         // 128-byte swizzle chunks per row
  static constexpr uint32_t TILE = 128u * D * 2, CHUNK = 128u * 128;
  // K and V tiles, in turn, and staged code tiles: what fills the 227 KB at d = 128
  static constexpr int NS = FMT == BSA_CACHE_BF16 ? (PAIR ? 5 : 6) : FMT == BSA_CACHE_E4M3 ? 3 : PAIR ? 3 : 4;
  static constexpr int NG = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? (PAIR ? 3 : 5) : PAIR ? 4 : 6;
  static constexpr uint32_t CODES = 128u * RB;
  static constexpr uint32_t EXPS = CODES, GROUPS = EXPS + 128;    // of a stage: codes, row exponents, group scales
  static constexpr uint32_t STAGE = Q16 ? GROUPS + (FMT == BSA_CACHE_E2M1 ? 128u * (D / 16) : 0) : 0;
  static constexpr uint32_t OFF_Q = 0, OFF_T = NTQ * TILE, OFF_G = OFF_T + NS * TILE, OFF_BAR = OFF_G + NG * STAGE;
  static constexpr int B_QF = 0, B_QE = 1, B_F = 2, B_E = B_F + NS, B_GF = B_E + NS, B_GE = B_GF + NG, B_SF = B_GE + NG,
                       B_PR = B_SF + 2, B_OD = B_PR + 4, B_OE = B_OD + 2, B_IN = B_OE + 2, B_IK = B_IN + kUnits,
                       B_SG = B_IK + (Q16 ? kUnits : 0), B_SE = B_SG + kSegs, B_RS = B_SE + kSegs,
                       B_FIN = B_RS + (Q16 ? 2 : 0), NBARS = B_FIN + 1;
  static constexpr uint32_t OFF_MISC = OFF_BAR + (NBARS * 8 + 15) / 16 * 16;  // TMEM address, abort flag, run
  static constexpr uint32_t OFF_SEG = OFF_MISC + 32;                          // [kSegs] two int4
  static constexpr uint32_t OFF_INFO = OFF_SEG + kSegs * 32;                  // [kUnits] chunks there; K's scale; oref
  static constexpr uint32_t OFF_RED = OFF_INFO + kUnits * 12;                 // [2][2][128] halves' maxima, bf16
  static constexpr uint32_t OFF_ROWS = OFF_RED + 1024;                        // [2][NTQ * 128] row scales of Q
  static constexpr uint32_t SMEM = OFF_ROWS + (Q16 ? 2 * NTQ * 128 * 4 : 0) + 1024;
  static_assert(SMEM <= kMaxSmem, "shared memory");
  static constexpr uint32_t F16 = Q16 ? (1u << 7) | (1u << 10) : 0;
  static constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, 128, false) & ~F16;
  static constexpr uint32_t IDESC_O = ptx::idesc_bf16_f32(128, D, true) & ~F16;
  static constexpr int TM_O = 256;  // S_0, S_1, O_0, O_1
};

// The plan of group y over its shared pages: units of one row tile, and row tiles (of one KV head).
struct SharedPlan {
  int per, tiles;
};
__device__ __forceinline__ SharedPlan shared_plan(const TreeArgs &a, const SharedRows &r, int tile_rows) {
  const int chunks = r.pages << (a.c.page_shift - 6);
  return SharedPlan{(chunks + 1) / 2, (r.rows.len * a.group + tile_rows - 1) / tile_rows};
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

template <int D, int FMT, bool PAIR>
__global__ void __launch_bounds__(Shared<D, FMT, PAIR>::THREADS, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const TreeArgs a, float *part_o, float2 *part_ml,
                  const SharedOut so) {
  using C = Shared<D, FMT, PAIR>;
  constexpr bool Q16 = C::Q16;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char *sb = smem_raw + (base - raw);
  const uint32_t bar0 = base + C::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sb + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sb + C::OFF_MISC + 4);
  int *run_of = reinterpret_cast<int *>(sb + C::OFF_MISC + 8);  // first unit of the run, the one past its last, group, its first unit
  int4 *seg_rec = reinterpret_cast<int4 *>(sb + C::OFF_SEG);
  int *info_in = reinterpret_cast<int *>(sb + C::OFF_INFO);
  float *info_k = reinterpret_cast<float *>(info_in + kUnits);
  int *info_v = reinterpret_cast<int *>(info_k + kUnits);
  uint16_t *red = reinterpret_cast<uint16_t *>(sb + C::OFF_RED);
  float *row_scale = reinterpret_cast<float *>(sb + C::OFF_ROWS);
  const Ctl ctl{abort_flag, nullptr};
  auto wait_warp = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait_parked(bar(i), parity, ctl)) != 0; };
  auto arrive_warp = [&](int i) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar(i));
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, G = a.group;

  if (tid == 32) {
    for (int x = 0; x < C::NBARS; ++x) {
      // arrivals: 1 of a commit, the producer or a copy's announcement; 4 of the loader warps; 8 of a lane's warps; 16
      // of both lanes'
      uint32_t count = 1;
      if (Q16 && (x == C::B_QF || (x >= C::B_F && x < C::B_E) || (x >= C::B_GE && x < C::B_SF) ||
                  (x >= C::B_RS && x < C::B_FIN)))
        count = 4;
      else if ((x >= C::B_PR && x < C::B_OD) || (x >= C::B_OE && x < C::B_IN))
        count = 8;
      else if (x >= C::B_SE && x < C::B_RS)
        count = 16;
      ptx::mbar_init(bar(x), count);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  if (warp == 0) {
    // ---- the plan, a lane per group: all units, then where this CTA's run begins
    auto units_of = [&](int y) {
      if (y >= a.groups) return 0;
      const SharedPlan p = shared_plan(a, shared_rows(a, y), C::NTQ * kRows);
      return p.per * p.tiles * a.c.hkv;
    };
    int all = 0, mine = 0, inc = 0;
    for (int y0 = 0; y0 < a.groups; y0 += 32) {
      mine = units_of(y0 + lane);
      inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (cta == 0 && y0 + lane < a.groups) so.plan[y0 + lane] = all + inc - mine;
      all += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (cta == 0 && lane == 0) so.plan[a.groups] = all;
    const int W = (all + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const int x0 = min(all, cta * W), x1 = min(all, x0 + W);
    int y = 0, first = 0;
    if (x0 < x1) {
      int before = 0;
      for (int y0 = 0; y0 < a.groups; y0 += 32) {
        if (a.groups > 32) {
          mine = units_of(y0 + lane);
          inc = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
          }
        }
        const unsigned over = __ballot_sync(0xffffffffu, before + inc > x0);
        if (over != 0) {
          const int at = __ffs(over) - 1;
          y = y0 + at;
          first = before + __shfl_sync(0xffffffffu, inc - mine, at);
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    if (lane == 0) {
      run_of[0] = x0;
      run_of[1] = x1;
      run_of[2] = y;
      run_of[3] = first;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int x0 = run_of[0], x1 = run_of[1], nu = x1 - x0;

  if (warp < 4) {
    ptx::setmaxnreg_dec<C::REG_LOW>();
    if (warp == 0 && nu > 0) {
      // ================================================================ producer
      // A segment's record: {units, first token, tokens, KV head}, {row tile, 1 if the CTA has all of the row tile's
      // units | 2 if it does not begin the run, 0, 0}.
      bool ok = true;
      int y = run_of[2], first = run_of[3], n = 0, seg = 0;
      uint32_t tiles_sent = 0, stages_sent = 0;
      for (int x = x0; ok && x < x1; ++seg) {
        SharedRows r = shared_rows(a, y);
        SharedPlan p = shared_plan(a, r, C::NTQ * kRows);
        while (x >= first + p.per * p.tiles * a.c.hkv) {  // (the run is not at its end: there is a next group)
          first += p.per * p.tiles * a.c.hkv;
          r = shared_rows(a, ++y);
          p = shared_plan(a, r, C::NTQ * kRows);
        }
        const int tile = (x - first) / p.per, rs = first + tile * p.per, k0 = x - rs;
        const int g = tile / p.tiles, rt = tile - g * p.tiles, units = min(rs + p.per, x1) - x;
        const int32_t *table = a.table + static_cast<size_t>(r.seq) * a.table_stride;
        const int chunks = r.pages << (a.c.page_shift - 6), sub_mask = (1 << (a.c.page_shift - 6)) - 1;
        if (seg >= kSegs) ok = wait_warp(C::B_SE + seg % kSegs, (seg / kSegs - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          seg_rec[2 * (seg % kSegs)] = make_int4(units, r.rows.start, r.rows.len, g);
          seg_rec[2 * (seg % kSegs) + 1] =
              make_int4(rt, (rs >= x0 && rs + p.per <= x1 ? 1 : 0) | (rs <= x0 ? 0 : 2), 0, 0);
          ptx::mbar_arrive(bar(C::B_SG + seg % kSegs));
        }
        if constexpr (!Q16) {
          if (lane == 0) {
            if (seg > 0) ok = wait_parked(bar(C::B_QE), (seg - 1) & 1, ctl);
            if (ok) {
              ptx::mbar_arrive_expect_tx(bar(C::B_QF), C::NTQ * C::TILE);
              for (int t = 0; t < C::NTQ; ++t)
                for (int c = 0; c < C::NCH; ++c)
                  tma_load_3d(base + C::OFF_Q + t * C::TILE + c * C::CHUNK, &tm_q, bar(C::B_QF), c * 64, g * G,
                              r.rows.start + (rt * C::NTQ + t) * (kRows / G));
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
        }
        // pages of the segment's units, 32 at a time, one per lane and a batch ahead; -1: none
        auto look_up = [&](int i, int &p0, int &p1) {
          p0 = p1 = -1;
          if (i >= units) return;
          const int c = 2 * (k0 + i);
          p0 = __ldg(table + (c >> (a.c.page_shift - 6)));
          if (c + 1 < chunks) p1 = sub_mask == 0 ? __ldg(table + c + 1) : p0;
        };
        auto checked = [&](int &p) {
          if (p < -1 || p >= a.c.pages) p = -2;
        };
        int now0, now1, next0, next1;
        look_up(lane, now0, now1);
        for (int i = 0; ok && i < units; ++i, ++n) {
          if (i % 32 == 0) {
            if (i > 0) now0 = next0, now1 = next1;
            look_up(i + 32 + lane, next0, next1);
            // an entry that names no page
            checked(now0);
            checked(now1);
            if (i + lane < units && (now0 < 0 || now1 < -1 || (now1 < 0 && 2 * (k0 + i + lane) + 1 < chunks))) report_arg(a);
          }
          const int p0 = __shfl_sync(0xffffffffu, now0, i & 31), p1 = __shfl_sync(0xffffffffu, now1, i & 31);
          if (lane == 0) {
            const int sub = (2 * (k0 + i)) & sub_mask;
            const int there = (p0 >= 0 ? 1 : 0) | (p1 >= 0 ? 2 : 0);
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const uint32_t z = 2u * static_cast<uint32_t>(n) + kv;
              if constexpr (!Q16) {
                const uint32_t s = z % C::NS, round = z / C::NS;
                if (round > 0 && !(ok = wait_parked(bar(C::B_E + s), (round - 1) & 1, ctl))) break;
                if (kv == 0) {
                  info_in[n % kUnits] = there;
                  ptx::mbar_arrive(bar(C::B_IN + n % kUnits));
                }
                const CUtensorMap *map = kv == 0 ? &tm_k : &tm_v;
                const uint32_t dst = base + C::OFF_T + s * C::TILE, f = bar(C::B_F + s);
                ptx::mbar_arrive_expect_tx(f, C::TILE);
                // a chunk that is not there lies outside the tensor, and comes as zeros
                const int none = a.c.pages * a.c.hkv;
                const int row0 = p0 >= 0 ? p0 * a.c.hkv + g : none, row1 = p1 >= 0 ? p1 * a.c.hkv + g : none;
                if (sub_mask != 0) {
                  for (int c = 0; c < C::NCH; ++c) tma_load_3d(dst + c * C::CHUNK, map, f, c * 64, sub * kChunk, row0);
                } else {
                  for (int c = 0; c < C::NCH; ++c) {
                    tma_load_3d(dst + c * C::CHUNK, map, f, c * 64, 0, row0);
                    tma_load_3d(dst + c * C::CHUNK + kChunk * 128, map, f, c * 64, 0, row1);
                  }
                }
                tiles_sent = z + 1;
              } else {
                const uint32_t s = z % C::NG, round = z / C::NG;
                if (round > 0 && !(ok = wait_parked(bar(C::B_GE + s), (round - 1) & 1, ctl))) break;
                if (kv == 0) {
                  info_in[n % kUnits] = there;
                  ptx::mbar_arrive(bar(C::B_IN + n % kUnits));
                }
                constexpr int PER = FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
                const uint8_t *codes = kv == 0 ? a.k_codes : a.v_codes, *scales = kv == 0 ? a.k_scales : a.v_scales;
                const uint32_t dst = base + C::OFF_G + s * C::STAGE, f = bar(C::B_GF + s);
                const uint32_t half = C::STAGE / 2;  // of a chunk
                ptx::mbar_arrive_expect_tx(f, ((there & 1) + (there >> 1)) * half);
                for (int h = 0; h < 2; ++h) {
                  const int pg = h == 0 ? p0 : p1;
                  if (pg < 0) continue;
                  const size_t tile = static_cast<size_t>(pg) * a.c.hkv + g;
                  const int row = sub_mask == 0 ? 0 : (sub + h) * kChunk;
                  bulk_load(dst + h * (C::CODES / 2), codes + (tile * a.c.page + row) * C::RB, C::CODES / 2, f);
                  const uint8_t *sc = scales + tile * a.c.page * PER;
                  bulk_load(dst + C::EXPS + h * 64, sc + row, 64, f);
                  if constexpr (FMT == BSA_CACHE_E2M1)
                    bulk_load(dst + C::GROUPS + h * (64 * (D / 16)), sc + a.c.page + row * (D / 16), 64 * (D / 16), f);
                }
                stages_sent = z + 1;
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        x += units;
      }
      if (*abort_flag && lane == 0) {
        // let copies in flight land before the CTA's shared memory is released
        if constexpr (!Q16) {
          if (seg > 0) drain_bar(bar(C::B_QF), (seg - 1) & 1);
          for (uint32_t z = tiles_sent > C::NS ? tiles_sent - C::NS : 0; z < tiles_sent; ++z)
            drain_bar(bar(C::B_F + z % C::NS), (z / C::NS) & 1);
        } else {
          for (uint32_t z = stages_sent > C::NG ? stages_sent - C::NG : 0; z < stages_sent; ++z)
            drain_bar(bar(C::B_GF + z % (C::NG > 0 ? C::NG : 1)), (z / (C::NG > 0 ? C::NG : 1)) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 1 && lane == 0 && nu > 0) {
      // ================================================================ MMA issuer
      const uint64_t dq0 = ptx::sdesc_sw128(base + C::OFF_Q, 16, 1024);
      const uint64_t dk0 = ptx::sdesc_sw128(base + C::OFF_T, 16, 1024);
      const uint64_t dv0 = ptx::sdesc_sw128(base + C::OFF_T, C::CHUNK, 1024);
      auto issue_s = [&](int t, uint32_t slot) {
        const uint64_t dq = dq0 + static_cast<uint64_t>(PAIR ? t : 0) * (C::TILE >> 4);
        const uint64_t dk = dk0 + static_cast<uint64_t>(slot) * (C::TILE >> 4);
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
      uint32_t pv_count[2] = {0, 0}, lane_segs[2] = {0, 0};  // P V products of each lane, segments in which it had a unit
      auto issue_pv = [&](int t, uint32_t slot, bool accumulate) -> bool {
        const uint64_t dv = dv0 + static_cast<uint64_t>(slot) * (C::TILE >> 4);
        const uint32_t dst = tmem + C::TM_O + t * 128, src = tmem + t * 128, parity = pv_count[t]++ & 1;
        // 32 keys of each half: P of a half lies over the first of its columns
        if (!wait_parked(bar(C::B_PR + 2 * t), parity, ctl)) return false;
        ptx::tc_fence_after();
        mma_ts_at<0, 0>(dst, src, dv, C::IDESC_O, accumulate ? 1u : 0u);
        mma_ts_at<8, 128>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<64, 512>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<72, 640>(dst, src, dv, C::IDESC_O, 1u);
        if (!wait_parked(bar(C::B_PR + 2 * t + 1), parity, ctl)) return false;
        ptx::tc_fence_after();
        mma_ts_at<16, 256>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<24, 384>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<80, 768>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<88, 896>(dst, src, dv, C::IDESC_O, 1u);
        return true;
      };
      // the lane's first P V of a segment overwrites O: the last segment's must have been read
      auto o_free = [&](int t) -> bool {
        const uint32_t k = lane_segs[t]++;
        return k == 0 || wait_parked(bar(C::B_OE + t), (k - 1) & 1, ctl);
      };
      auto tile_there = [&](uint32_t z) -> bool {
        if (!wait_parked(bar(C::B_F + z % C::NS), (z / C::NS) & 1, ctl)) return false;
        ptx::tc_fence_after();
        return true;
      };
      bool ok = true;
      uint32_t n = 0;
      int seg = 0;
      for (int x = x0; ok && x < x1; ++seg) {
        if (!(ok = wait_parked(bar(C::B_SG + seg % kSegs), (seg / kSegs) & 1, ctl))) break;
        const int units = seg_rec[2 * (seg % kSegs)].x;
        x += units;
        if (!(ok = wait_parked(bar(C::B_QF), seg & 1, ctl))) break;
        ptx::tc_fence_after();
        for (int i = 0; i < units; ++i, ++n) {
          const uint32_t kz = 2 * n, vz = kz + 1;
          const bool last = i == units - 1;
          if (!(ok = tile_there(kz))) break;
          if constexpr (PAIR) {
            // S_0(n) overwrites what P_0 V(n - 1) reads: MMAs of one thread run in the order of issue
            issue_s(0, kz % C::NS);
            if (!(ok = tile_there(vz))) break;
            if (i > 0) {
              if (i == 1 && !(ok = o_free(1))) break;
              if (!(ok = issue_pv(1, (vz - 2) % C::NS, i > 1))) break;
              ptx::mma_commit(bar(C::B_E + (vz - 2) % C::NS));
            }
            issue_s(1, kz % C::NS);
            if (last) ptx::mma_commit(bar(C::B_QE));
            ptx::mma_commit(bar(C::B_E + kz % C::NS));
            if (i == 0 && !(ok = o_free(0))) break;
            if (!(ok = issue_pv(0, vz % C::NS, i > 0))) break;
            if (last) {
              ptx::mma_commit(bar(C::B_OD));
              if (i == 0 && !(ok = o_free(1))) break;
              if (!(ok = issue_pv(1, vz % C::NS, i > 0))) break;
              ptx::mma_commit(bar(C::B_E + vz % C::NS));
              ptx::mma_commit(bar(C::B_OD + 1));
            }
          } else {
            issue_s(i & 1, kz % C::NS);
            ptx::mma_commit(bar(C::B_E + kz % C::NS));
            if (last) ptx::mma_commit(bar(C::B_QE));
            for (int j = i > 0 ? i - 1 : i; j <= i; ++j) {  // unit i - 1, and the last unit itself
              if (j == i && !last) break;
              const uint32_t z = vz - 2 * static_cast<uint32_t>(i - j);
              const int t = j & 1;
              if (j < 2 && !(ok = o_free(t))) break;
              if (!(ok = tile_there(z) && issue_pv(t, z % C::NS, j >= 2))) break;
              ptx::mma_commit(bar(C::B_E + z % C::NS));
              if (j + 2 >= units) ptx::mma_commit(bar(C::B_OD + t));
            }
            if (!ok) break;
          }
        }
      }
      if (!ok) {
        // every MMA issued so far must finish before TMEM is released
        ptx::mma_commit(bar(C::B_FIN));
        drain_bar(bar(C::B_FIN), 0);
      }
    }
    __syncwarp();
  } else if (warp < kLoadWarp) {
    // ================================================================ softmax lanes
    ptx::setmaxnreg_inc<C::REG_SOFT>();
    const int t = (warp - kSoftWarp) >> 3, hf = ((warp - kSoftWarp) >> 2) & 1, sub = warp & 3;
    const int r = (sub << 5) + lane;  // query row = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(sub << 5) << 16;
    const uint32_t tS = tmem + lane_off + t * 128 + hf * 64;  // this thread's S columns, P over the first half
    const uint32_t tO = tmem + lane_off + C::TM_O + t * 128 + hf * (D / 2);
    uint16_t *mine_max = red + (t * 2 + hf) * 128 + r, *other_max = red + (t * 2 + 1 - hf) * 128 + r;
    const int pair_bar = 1 + t * 4 + sub;  // the two warps that share rows
    bool ok = true;
    uint32_t n = 0, mine = 0, lane_segs = 0;  // units of the run, of this lane; its segments
    int seg = 0;
    for (int x = x0; ok && x < x1; ++seg) {
      if (!(ok = wait_warp(C::B_SG + seg % kSegs, (seg / kSegs) & 1))) break;
      const int4 ra = seg_rec[2 * (seg % kSegs)], rb = seg_rec[2 * (seg % kSegs) + 1];
      const int units = ra.x;
      x += units;
      float rs = a.scale_log2;
      if constexpr (Q16) {
        if (PAIR || units > t) {
          if (!(ok = wait_warp(C::B_RS + (seg & 1), (seg >> 1) & 1))) break;
          rs *= row_scale[((seg & 1) * C::NTQ + (PAIR ? t : 0)) * 128 + r];
        }
      }
      float m = -INFINITY, l = 0.f;
      int oref = 0, done = 0;  // O's unit (8- and 4-bit caches); units of this lane in the segment
      for (int i = 0; i < units; ++i, ++n) {
        if (!PAIR && (i & 1) != t) continue;
        if (!(ok = wait_warp(C::B_IN + n % kUnits, (n / kUnits) & 1))) break;
        const bool there = (info_in[n % kUnits] >> hf & 1) != 0;
        float scl = rs;
        int oref_new = 0;
        if constexpr (Q16) {
          if (!(ok = wait_warp(C::B_IK + n % kUnits, (n / kUnits) & 1))) break;
          // never 0, so that logits below it are 0 to any precision and not NaN
          scl = fmaxf(scl * info_k[n % kUnits], 1e-37f);
          oref_new = info_v[n % kUnits];
        }
        if (!(ok = wait_warp(C::B_SF + t, mine & 1))) break;
        ptx::tc_fence_after();
        uint32_t sr[Q16 ? 32 : 64];
        float pm[2];
        if constexpr (Q16) {  // registers for half of the logits: the second half is read again
          uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
          ptx::tmem_ld32_max(tS + 32, s0, pm[1]);
          ptx::tmem_wait_ld();
          ptx::tmem_ld32_max(tS, s0, pm[0]);
        } else {
          ptx::tmem_ld32_max(tS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]), pm[0]);
          ptx::tmem_ld32_max(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[Q16 ? 0 : 32]), pm[1]);
        }
        ptx::tmem_wait_ld();
        // the row's maximum of both halves: each half's rounded up to bf16 (any upper bound is a valid reference, and
        // both halves then hold the same value).  The slot is written again only after the partner has released P,
        // which the lane's next S waits for.
        uint32_t u = there ? __float_as_uint(fmaxf(pm[0], pm[1])) : 0xFF800000u;
        if ((u & 0xFFFFu) != 0u && !(u >> 31)) u += 0x10000u;
        *mine_max = static_cast<uint16_t>(u >> 16);
        ptx::named_barrier(pair_bar, 64);
        const float mx = fmaxf(__uint_as_float(u & 0xFFFF0000u), __uint_as_float(static_cast<uint32_t>(*other_max) << 16));
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
        // a chunk that is not there: p = 0 whatever its columns hold
        const float bias = there ? static_cast<float>(C::SHIFT) - mb : -INFINITY;
        uint64_t acc[2] = {0ull, 0ull};
        const uint64_t scl2 = there ? ptx::f32x2(scl, scl) : 0ull, bias2 = ptx::f32x2(bias, bias);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          constexpr int STEP = Q16 ? 0 : 32;
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t y = ptx::fma_f32x2(
                ptx::f32x2(__uint_as_float(sr[c * STEP + 2 * e]), __uint_as_float(sr[c * STEP + 2 * e + 1])), scl2, bias2);
            float y0, y1;
            ptx::f32x2_split(y, y0, y1);
            const float p0 = ptx::ex2_approx(y0), p1 = ptx::ex2_approx(y1);
            acc[e & 1] = ptx::add_f32x2(acc[e & 1], ptx::f32x2(p0, p1));
            pk[e] = Q16 ? pack_f16x2(p0, p1) : ptx::pack_bf16x2(p0, p1);
          }
          ptx::tmem_st16(tS + c * 16, pk);
          if (c == 0) {
            if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t ov[8];
                ptx::tmem_ld8(tO + q * 8, ov);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * of);
                ptx::tmem_st8(tO + q * 8, ov);
              }
            }
            if constexpr (Q16) ptx::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          arrive_warp(C::B_PR + 2 * t + c);
          if (Q16 && c == 0) ptx::tmem_wait_ld();
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

      // ---- the segment's result of this lane: this thread's half of the dimensions and of the sum
      if (done > 0) {
        if (!(ok = wait_warp(C::B_OD + t, lane_segs & 1))) break;
        ptx::tc_fence_after();
        ++lane_segs;
      }
      m = ptx::part_max(m, l);
      const bool whole = (rb.y & 1) != 0;
      const int row = (rb.x * C::NTQ + (PAIR ? t : 0)) * kRows + r, tok = row / G;
      const size_t out = static_cast<size_t>(ra.y + tok) * a.hq + ra.w * G + row % G;
      const size_t slot = 2 * (2 * static_cast<size_t>(cta) + (rb.y >> 1)) + t;
      const bool live = tok < ra.z;
      float unit_f = 1.f;
      if constexpr (Q16) unit_f = exp2f(static_cast<float>(oref - 127 - C::SHV - C::SHIFT));
      if (done > 0) {
        float4 *po = reinterpret_cast<float4 *>(part_o) + (slot * (D / 4) + hf * (D / 8)) * kRows + r;
        float4 *ro = reinterpret_cast<float4 *>(so.row_o + ((PAIR ? 0 : t) * so.rows + out) * D) + hf * (D / 8);
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t ov[8];
          ptx::tmem_ld8(tO + q * 8, ov);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 v = make_float4(__uint_as_float(ov[4 * e]) * unit_f, __uint_as_float(ov[4 * e + 1]) * unit_f,
                                         __uint_as_float(ov[4 * e + 2]) * unit_f, __uint_as_float(ov[4 * e + 3]) * unit_f);
            if (!whole) po[(2 * q + e) * kRows] = v;
            else if (live) ro[2 * q + e] = v;
          }
        }
      }
      if (!whole) part_ml[(slot * 2 + hf) * kRows + r] = make_float2(m, l);
      else if (live) so.row_ml[((PAIR ? 0 : t) * 2 + hf) * so.rows + out] = make_float2(m, l);
      ptx::tc_fence_before();
      if (done > 0) arrive_warp(C::B_OE + t);
      arrive_warp(C::B_SE + seg % kSegs);
    }
  } else if constexpr (Q16) {
    // ================================================================ loaders
    ptx::setmaxnreg_inc<C::REG_LOAD>();
    const int lt = tid - kLoadWarp * 32;
    constexpr int PP = C::RB / 16, STEP = 128 / PP;  // pieces of a code row; a thread's rows are STEP apart
    const int p = lt % PP, r0 = lt / PP;
    bool ok = true;
    uint32_t n = 0;
    int seg = 0;
    for (int x = x0; ok && x < x1; ++seg) {
      if (!(ok = wait_warp(C::B_SG + seg % kSegs, (seg / kSegs) & 1))) break;
      const int4 ra = seg_rec[2 * (seg % kSegs)], rb = seg_rec[2 * (seg % kSegs) + 1];
      const int units = ra.x;
      x += units;
      // ---- Q: rows as f16, the largest element of each brought to [2^14, 2^15)
      if (seg > 0 && !(ok = wait_warp(C::B_QE, (seg - 1) & 1))) break;
      constexpr int LPR = D / 8, RS = 128 / LPR, U = 4;  // threads of a row, rows of a step, steps in flight
#pragma unroll 1
      for (int q0 = 0; q0 < C::NTQ * kRows; q0 += RS * U) {
        uint4 v[U];
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int row = rb.x * C::NTQ * kRows + q0 + e * RS + lt / LPR, tok = row / G;
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (tok < ra.z)
            v[e] = __ldg(reinterpret_cast<const uint4 *>(
                a.q + (static_cast<size_t>(ra.y + tok) * a.hq + ra.w * G + row % G) * D + lt % LPR * 8));
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int rr = q0 + e * RS + lt / LPR;
          float am = amax8(v[e]);
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
          const int ex = max(1, min(253, 268 - (__float_as_int(am) >> 23)));
          const float f = pow2_biased(ex);
          if (lt % LPR == 0) row_scale[(seg & 1) * C::NTQ * 128 + rr] = pow2_biased(254 - ex);
          uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            w[c] = pack_f16x2(__uint_as_float(w[c] << 16) * f, __uint_as_float(w[c] & 0xFFFF0000u) * f);
          *reinterpret_cast<uint4 *>(sb + swizzled(C::OFF_Q + (rr >> 7) * C::TILE, lt % LPR >> 3, rr & 127, lt % LPR & 7)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      ptx::fence_proxy_async_smem();
      arrive_warp(C::B_QF);
      arrive_warp(C::B_RS + (seg & 1));

      int oref = 0;
      for (int i = 0; ok && i < units; ++i, ++n) {
        // ---- the unit's scales, K's and V's
        if (!(ok = wait_warp(C::B_IN + n % kUnits, (n / kUnits) & 1))) break;
        const int there = info_in[n % kUnits];
        int ref[2];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t z = 2 * n + kv;
          if (!(ok = wait_warp(C::B_GF + z % C::NG, (z / C::NG) & 1))) break;
          const uint32_t w = *reinterpret_cast<const uint32_t *>(sb + C::OFF_G + (z % C::NG) * C::STAGE + C::EXPS + lane * 4);
          const uint32_t m = (there >> (lane >> 4) & 1) != 0 ? __vmaxu4(w, w >> 16) : 0u;
          ref[kv] = static_cast<int>(__reduce_max_sync(0xffffffffu, max(m & 0xFFu, (m >> 8) & 0xFFu)));
        }
        if (!ok) break;
        ref[1] = oref = max(oref, ref[1]);
        if (lt == 0) {
          info_k[n % kUnits] = exp2f(static_cast<float>(ref[0] - C::SHV - 127));
          info_v[n % kUnits] = oref;
          ptx::mbar_arrive(bar(C::B_IK + n % kUnits));
        }
        // ---- both tiles
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t z = 2 * n + kv, s = z % C::NS, round = z / C::NS;
          if (round > 0 && !(ok = wait_warp(C::B_E + s, (round - 1) & 1))) break;
          const unsigned char *stage = sb + C::OFF_G + (z % C::NG) * C::STAGE;
          const uint32_t dst = C::OFF_T + s * C::TILE;
          const int top = kv == 0 ? ref[0] : ref[1];
#pragma unroll 4
          for (int e = 0; e < PP; ++e) {
            const int row = r0 + e * STEP;
            const bool live = (there >> (row >> 6) & 1) != 0;
            const uint4 cw = live ? *reinterpret_cast<const uint4 *>(stage + row * C::RB + p * 16) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t f = live ? pow2_f16x2(static_cast<int>(stage[C::EXPS + row]) - top + C::SHV) : 0u;
            const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
            const uint32_t at = dst + static_cast<uint32_t>(row) * 128;
            auto put = [&](int c, int u, uint4 v) {  // unit u of swizzle chunk c
              *reinterpret_cast<uint4 *>(sb + at + static_cast<uint32_t>(c) * C::CHUNK +
                                         static_cast<uint32_t>((u ^ (row & 7)) * 16)) = v;
            };
            if constexpr (FMT == BSA_CACHE_E4M3) {
              uint32_t h[8];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                h[2 * c] = mul_f16x2(e4m3x2_f16(w[c]), f);
                h[2 * c + 1] = mul_f16x2(e4m3x2_f16(w[c] >> 16), f);
              }
              const uint4 s0 = make_uint4(h[0], h[1], h[2], h[3]), s1 = make_uint4(h[4], h[5], h[6], h[7]);
              // the upper pieces store their halves in the other order: no two lanes meet in a bank
              const int u = 2 * (p & 3), sw = (p >> 2) & 1;
              put(p >> 2, u + sw, sw ? s1 : s0);
              put(p >> 2, u + 1 - sw, sw ? s0 : s1);
            } else {
              const uint32_t g2 = mul_f16x2(
                  e4m3x2_f16(live ? *reinterpret_cast<const uint16_t *>(stage + C::GROUPS + row * (D / 16) + 2 * p) : 0u), f);
              const uint32_t ga = __byte_perm(g2, g2, 0x1010), gb = __byte_perm(g2, g2, 0x3232);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t gs = c < 2 ? ga : gb;
                put(p >> 1, 4 * (p & 1) + c,
                    make_uint4(mul_f16x2(e2m1x2_f16(w[c]), gs), mul_f16x2(e2m1x2_f16(w[c] >> 8), gs),
                               mul_f16x2(e2m1x2_f16(w[c] >> 16), gs), mul_f16x2(e2m1x2_f16(w[c] >> 24), gs)));
              }
            }
          }
          ptx::fence_proxy_async_smem();
          arrive_warp(C::B_F + s);
          arrive_warp(C::B_GE + z % C::NG);
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag && a.status != nullptr)
    atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_DEVICE_TIMEOUT));
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  // The kernel over the sequences' own keys may still run beside this one; the combine waits for this one alone.
  after_previous_kernel();
}

// The combine.  A block is up to kItems (row, four dimensions) of one token and KV head; its kSplit teams take parts
// i, i + kSplit, ..: the parts of the token's rows over the shared pages, then those over its own keys.  Sums are
// added in a fixed order.
constexpr int kItems = 64, kSplit = 8;

// Where the parts of a token's rows in one row tile are.
struct Parts {
  int count;  // 0: no keys
  bool whole;  // one part, left row by row
  int first_cta, tile_first, run, tile, row;
};
__device__ __forceinline__ Parts parts_of(int tile_first, int per, int row, int tile_rows, int run) {
  Parts p;
  p.tile_first = tile_first;
  p.first_cta = tile_first / run;
  p.count = (tile_first + per - 1) / run - p.first_cta + 1;
  p.whole = p.count == 1;
  p.run = run;
  p.tile = row % tile_rows / kRows;
  p.row = row % kRows;
  return p;
}

template <int D, bool PAIR>
__global__ void __launch_bounds__(kItems * kSplit)
    shared_combine_kernel(const TreeArgs a, const float *part_o, const float2 *part_ml, const float *own_o,
                          const float2 *own_ml, const SharedOut so, const int *own_plan, const OwnParts op) {
  constexpr int LANES = PAIR ? 1 : 2;  // results of a row and part over shared pages
  after_previous_kernel();
  __shared__ float red_m[kSplit][kItems], red_l[kSplit][kItems];
  __shared__ float4 red_o[kSplit][kItems];
  const int G = a.group, items = G * (D / 4), slices = (items + kItems - 1) / kItems;
  const int i = blockIdx.x / slices, g = blockIdx.y, b = blockIdx.z;
  const Drafts dr = drafts_of(a, b);
  if (i >= dr.len) return;
  const int y = group_of(a, b);
  Parts ps{}, po{};
  if (y >= 0) {
    constexpr int TILE_ROWS = PAIR ? 2 * kRows : kRows;
    const SharedRows all = shared_rows(a, y);
    const SharedPlan plan = shared_plan(a, all, TILE_ROWS);
    const int at = dr.start + i - all.rows.start, units = so.plan[a.groups];
    if (at >= 0 && at < all.rows.len && plan.per > 0)
      ps = parts_of(so.plan[y] + (g * plan.tiles + at * G / TILE_ROWS) * plan.per, plan.per, at * G, TILE_ROWS,
                    (units + kSms - 1) / kSms);
  }
  const int shared = ps.count * LANES;
  {
    const int x = b * a.c.hkv + g, u0 = own_plan[x], units = own_plan[x + 1] - u0, all = own_plan[a.batch * a.c.hkv];
    const int tiles = (dr.len * G + op.rows - 1) / op.rows, per = units / tiles;
    if (op.rows_first) {  // one row tile, whatever its rows
      po = parts_of(u0, units, i * G, kRows, (all + op.ctas - 1) / op.ctas);
    } else {
      po = parts_of(u0 + i * G / op.rows * per, per, i * G, op.rows, (all + op.ctas - 1) / op.ctas);
    }
  }

  const int item = threadIdx.x % kItems, team = threadIdx.x / kItems;
  const int it = blockIdx.x % slices * kItems + item, h = it % G, q = it / G;
  const size_t out = static_cast<size_t>(dr.start + i) * a.hq + g * G + h;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (it < items) {
    const int n = shared + po.count;
    constexpr int U = 2;  // parts in flight
    for (int base = team; base < n; base += U * kSplit) {
      float2 ml[U], ml2[U];
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = base + u * kSplit;
        ml[u] = ml2[u] = make_float2(-INFINITY, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < shared) {
          const int lane = PAIR ? 0 : x & 1;
          if (ps.whole) {
            ml[u] = so.row_ml[2 * lane * so.rows + out];
            ml2[u] = so.row_ml[(2 * lane + 1) * so.rows + out];
            v[u] = reinterpret_cast<const float4 *>(so.row_o)[(lane * so.rows + out) * (D / 4) + q];
          } else {
            const int cta = ps.first_cta + x / LANES;
            const size_t slot = 2 * (2 * static_cast<size_t>(cta) + (ps.tile_first <= cta * ps.run ? 0 : 1)) + (PAIR ? ps.tile : lane);
            ml[u] = part_ml[slot * 2 * kRows + ps.row + h];
            ml2[u] = part_ml[(slot * 2 + 1) * kRows + ps.row + h];
            v[u] = reinterpret_cast<const float4 *>(part_o)[(slot * (D / 4) + q) * kRows + ps.row + h];
          }
        } else if (x < n) {
          if (po.whole) {
            ml[u] = so.row_ml[4 * so.rows + out];
            v[u] = reinterpret_cast<const float4 *>(so.row_o)[(2 * so.rows + out) * (D / 4) + q];
          } else {
            const int cta = po.first_cta + x - shared;
            const size_t slot = 2 * static_cast<size_t>(cta) + (po.tile_first <= cta * po.run ? 0 : 1);
            if (op.rows_first) {
              ml[u] = own_ml[slot * op.rows + po.row + h];
              v[u] = reinterpret_cast<const float4 *>(own_o)[(slot * op.rows + po.row + h) * (D / 4) + q];
            } else {
              const size_t tile = slot * (op.rows / kRows) + po.tile;
              ml[u] = own_ml[tile * kRows + po.row + h];
              v[u] = reinterpret_cast<const float4 *>(own_o)[(tile * (D / 4) + q) * kRows + po.row + h];
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float pm = ptx::max_nan(ml[u].x, ml2[u].x);  // (the halves differ where one holds NaN alone)
        if (pm == -INFINITY) continue;
        const float mn = ptx::max_nan(m, pm);
        const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(pm - mn);
        m = mn;
        l = fmaf(ml[u].y + ml2[u].y, w, l * f);
        acc.x = fmaf(v[u].x, w, acc.x * f);
        acc.y = fmaf(v[u].y, w, acc.y * f);
        acc.z = fmaf(v[u].z, w, acc.z * f);
        acc.w = fmaf(v[u].w, w, acc.w * f);
      }
    }
  }
  red_m[team][item] = m;
  red_l[team][item] = l;
  red_o[team][item] = acc;
  __syncthreads();
  if (team != 0 || it >= items) return;
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < kSplit; ++w) mm = ptx::max_nan(mm, red_m[w][item]);
  float ls = 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kSplit; ++w) {
    if (red_m[w][item] == -INFINITY) continue;
    const float f = exp2f(red_m[w][item] - mm);
    ls = fmaf(red_l[w][item], f, ls);
    const float4 v = red_o[w][item];
    s.x = fmaf(v.x, f, s.x);
    s.y = fmaf(v.y, f, s.y);
    s.z = fmaf(v.z, f, s.z);
    s.w = fmaf(v.w, f, s.w);
  }
  const float inv = ls == 0.f ? 0.f : 1.f / ls;
  *reinterpret_cast<uint2 *>(a.o + out * D + 4 * q) =
      make_uint2(ptx::pack_bf16x2(s.x * inv, s.y * inv), ptx::pack_bf16x2(s.z * inv, s.w * inv));
  if (a.lse != nullptr && q == 0) a.lse[out] = ls == 0.f ? -INFINITY : (mm + log2f(ls)) * 0.69314718055994531f;
}

struct Workspace {
  size_t part_o, part_ml, own_o, own_ml, lane_o, row_o, row_ml, plan, own_plan, total;
};
Workspace workspace_layout(const CacheDims &c, int groups, int batch, size_t rows) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t d = c.d, parts = 4ull * kSms * kRows;  // two parts per CTA, up to two row tiles or lanes each
  const OwnParts few = own_few_parts(c);
  const size_t own = 2ull * few.ctas * few.rows > parts ? 2ull * few.ctas * few.rows : parts;
  Workspace w;
  w.part_o = 0;
  w.part_ml = up(parts * d * 4);
  w.own_o = w.part_ml + up(2 * parts * 8);
  w.own_ml = w.own_o + up(own * d * 4);
  w.lane_o = w.own_ml + up(own * 8);
  w.row_o = w.lane_o + up(static_cast<size_t>(kSms) * kRows * (d + 4) * 4);
  w.row_ml = w.row_o + up(3 * rows * d * 4);
  w.plan = w.row_ml + up(6 * rows * 8);
  w.own_plan = w.plan + up((static_cast<size_t>(groups) + 1) * 4);
  w.total = w.own_plan + up((static_cast<size_t>(batch) * c.hkv + 1) * 4);
  return w;
}

// Rows of q [total, hq, d]: box of 64 dimensions, the G heads of a KV group and 128 / G tokens; 128-byte swizzle.
bool query_map(EncodeTiledFn fn, CUtensorMap *map, const TreeArgs &a) {
  const cuuint64_t d = static_cast<cuuint64_t>(a.c.d);
  const cuuint64_t dims[3] = {d, static_cast<cuuint64_t>(a.hq), static_cast<cuuint64_t>(a.total)};
  const cuuint64_t strides[2] = {d * 2, d * 2 * static_cast<cuuint64_t>(a.hq)};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(a.group), static_cast<cuuint32_t>(kRows / a.group)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(a.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int FMT, bool PAIR>
bsa_status launch_t(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  using C = Shared<D, FMT, PAIR>;
  CUtensorMap mq{}, mk{}, mv{};
  if (!C::Q16) {
    cudaError_t e = cudaSuccess;
    EncodeTiledFn fn = tensor_map_encoder(&e);
    if (fn == nullptr || e != cudaSuccess || !query_map(fn, &mq, a) || !chunk_map(fn, &mk, a.k_codes, a.c) ||
        !chunk_map(fn, &mv, a.v_codes, a.c))
      return BSA_ERR_CUDA;
  }
  const size_t rows = static_cast<size_t>(a.total) * a.hq;
  const Workspace ws = workspace_layout(a.c, a.groups, a.batch, rows);
  char *base = static_cast<char *>(workspace);
  auto f32 = [&](size_t at) { return reinterpret_cast<float *>(base + at); };
  auto f32x2 = [&](size_t at) { return reinterpret_cast<float2 *>(base + at); };
  SharedOut so{f32(ws.row_o), f32x2(ws.row_ml), rows, reinterpret_cast<int *>(base + ws.own_plan)};
  int *own_plan = so.plan;
  auto kern = shared_kernel<D, FMT, PAIR>;
  // setmaxnreg.inc waits until the registers it asks for are free: the split is only safe if the
  // kernel really launches with that many registers per thread
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_up(kern, C::SMEM, C::LAUNCH_REGS, done);
  if (e != cudaSuccess) return e == cudaErrorNotSupported ? BSA_ERR_UNSUPPORTED : BSA_ERR_CUDA;
  const bool few = a.max_draft * a.group <= own_few_parts(a.c).rows;
  const OwnParts op = few ? own_few_parts(a.c) : own_many_parts(a);
  e = few ? launch_own_few(a, so, f32(ws.own_o), f32(ws.own_ml), stream)
          : launch_own_many(a, so, f32(ws.own_o), f32(ws.own_ml), f32(ws.lane_o), stream);
  if (e != cudaSuccess) return e == cudaErrorNotSupported ? BSA_ERR_UNSUPPORTED : BSA_ERR_CUDA;
  so.plan = reinterpret_cast<int *>(base + ws.plan);
  e = launch_after(kern, dim3(kSms), C::THREADS, C::SMEM, stream, mq, mk, mv, a, f32(ws.part_o), f32x2(ws.part_ml), so);
  if (e != cudaSuccess) return BSA_ERR_CUDA;
  const int slices = (a.group * (D / 4) + kItems - 1) / kItems;
  e = launch_after(shared_combine_kernel<D, PAIR>, dim3(a.max_draft * slices, a.c.hkv, a.batch), kItems * kSplit, 0, stream, a,
                   static_cast<const float *>(f32(ws.part_o)), static_cast<const float2 *>(f32x2(ws.part_ml)),
                   static_cast<const float *>(f32(ws.own_o)), static_cast<const float2 *>(f32x2(ws.own_ml)), so,
                   static_cast<const int *>(own_plan), op);
  return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <int D, int FMT>
bsa_status launch_fmt(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  // two row tiles per unit halve the reads and conversions of the shared pages where a group fills more than one
  const bool pair = static_cast<long long>(a.total) * a.group > static_cast<long long>(kRows) * a.groups;
  return pair ? launch_t<D, FMT, true>(a, workspace, stream) : launch_t<D, FMT, false>(a, workspace, stream);
}

}  // namespace

size_t shared_workspace_bytes(const CacheDims &c, int groups, int batch, int total, int, int hq) {
  return workspace_layout(c, groups, batch, static_cast<size_t>(total) * hq).total;
}

bsa_status launch_shared(const TreeArgs &a, void *workspace, cudaStream_t stream) {
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
