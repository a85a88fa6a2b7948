// Attention of sequences that share the first pages of their tables, the shared pages read once for all.
//
// The drafted tokens of all sequences of a group times the G heads of a KV group are the query rows; 128 are a tile of
// tcgen05 MMAs.  The keys of a row tile come in units of 128: the group's shared pages, which all rows see; then, of
// every sequence that has rows in the tile, the pages it does not share, which its rows alone see; then the tile's
// drafted tokens, of which a row sees its path.  A unit that few rows see costs as much as another, but needs no
// switch of rows, whose latencies would be several units long: a step of 32 answers over a prompt of 128K and 350
// tokens of their own each has 1024 shared units a head, 106 own and one of drafts.
// (Own keys in a kernel of their own, 16 rows at a time, took 23 us of that step and 36 us of trees of 5 drafts.)
//
// shared_plan_kernel lays the tiles out; the units of all (tile, KV head) are laid end to end and cut into equal
// runs, one per CTA (one CTA per SM) of shared_kernel; a run crosses from one tile into the next (segments).
// shared_combine_kernel merges what several CTAs have of a row.
//
// Two lanes of eight softmax warps share the tensor core, so that one lane's exponentials run under the other's MMAs:
//   PAIR   (more than 128 rows a group)  the lanes hold two row tiles and the same keys
//   !PAIR  the lanes hold the same rows and take alternate units; both leave their results
// Two threads share a row, each with the 64 keys of one page chunk.  The issuing order S_0(n), P_1 V(n-1), S_1(n),
// P_0 V(n) keeps one tile's products under the other's softmax.  P lies over the first half of its own S columns.
// Warps:  0      looks units up, publishes segments, issues the copies (bf16: TMA tiles; codes: bulk copies)
//         1      TMEM owner; one thread issues the MMAs
//         2      (PAIR) passes the arrival of V and the next K on
//         4-19   the softmax lanes; before they release P of a unit with masked places, (bf16) they clean its V
//         20-27  (8- and 4-bit caches) Q, then the codes and drafted rows of K (20-23) and V into f16 tiles
//
// An 8- or 4-bit cache is computed in f16, with the scales of the drafted-token kernel: with e the exponent of a
// key's row and kref the largest of the unit, K' = code * 2^(e - kref + SHV) is exact down to e = kref - 21 (E4M3) or
// kref - 18 (E2M1); 2^(kref - 127 - SHV) joins the logit scale.  V likewise against oref, the largest exponent of the
// segment so far, O being held in units of 2^(oref - 127 - SHV - SHIFT).  Q rows become f16 after a power of two that
// brings their largest element to [2^14, 2^15), drafted K and V after one per unit.  P' = 2^(x - m + SHIFT) with the
// reference m at most 2^TH below the true maximum, so P' <= 2^15.  Row sums are fp32 from unrounded values.
//
// Inf and NaN of a value that some rows of the tile do not see would reach them (p = 0, and 0 times them is not 0):
// they are taken out of the product, and the combine adds them to the rows that see them.
// Every mbarrier wait is bounded, as in the prefill kernel.
//
// Measured (32 / 4 heads of 128): 32 answers over 128K in bf16 78 us (295 MB, 3.8 TB/s, 0.88 PFLOP/s), 8 answers 67 (bf16),
// 74 (e4m3), 74 (e2m1); 16 x 16 drafts over 32K in bf16 126 us (1.05 PFLOP/s).  Of 78 us 10 pass before the first product
// (5 of plan, then look-ups and the first tile) and 10 after the last was issued (parts through the L2, combine); of 66 with
// four groups of e4m3 15 and 10.  bf16: 3300 cycles a unit and pair of row tiles, 2150 of them products; the thread that
// issues them sets the pace (P released in halves: 90 us, waits that spin: 82, four barriers a lane for S: 82).  Codes: a
// loader warp's chain (of 3700 cycles a unit 2300 converted) and instruction supply.
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
constexpr int kRows = 128, kUnit = 128, kChunk = 64;  // rows of a tile; keys of a unit, of a page chunk
constexpr int kSoftWarp = 4, kLoadWarp = 20, kLoadWarps = 8;
constexpr int kSegs = 8;   // segments published ahead
constexpr int kUnits = 8;  // units whose records are kept
enum Kind { kShared = 0, kOwn = 1, kDraft = 2 };

// ---------------------------------------------------------------- the plan

// A sequence: its drafts, the keys it does not share and their first page; the place of its rows among its group's
// tokens and the group's first tile.
struct alignas(16) SeqRecord {
  int start, len, keys, first_page, at, tile0, pad0, pad1;
};
// A row tile: its tokens, the sequences that have rows in it, its units over shared pages (and their chunks, and the
// sequence whose table names them), the first drafted token that its rows see; the first unit (of one KV head), the
// units and those over own keys, the first place.
struct alignas(16) TileRecord {
  int tok0, tokens, seq_a, seq_b, shared, chunks, table, draft0, first, units, own, place;
};
// What the calls leave in the workspace.  Parts: two per CTA and lane, O as [dimension / 4][128 rows] float4, two
// halves' (max, sum); row buffers for tiles that one CTA has whole, of lane 0 (PAIR: of both) and 1.
struct SharedWork {
  float *part_o, *row_o;
  float2 *part_ml, *row_ml;
  size_t rows;
  SeqRecord *seqs;
  TileRecord *tiles;
  int *own_before;    // [batch + 1] units over own keys before a sequence's
  int *token_start;   // [total] the first token of a token's sequence
  int *totals;        // units of one KV head, tiles, whether a drafted value held Inf or NaN, places of one KV head
  uint32_t *odd;      // [batch * hkv][13] whether own values held Inf or NaN, and where: +Inf, -Inf, NaN, a bit per dimension
  int max_tiles;
};
constexpr int kOdd = 13;

// Runs are cut where the units of all tiles and KV heads are laid end to end at places: a unit that few rows see takes
// 7/6 of one over shared pages (its V is cleaned, its keys come from anywhere), and a tile's drafts with the change of
// rows behind them kPad more.  32 answers over 128K, own keys on four CTAs a head: these take 63 us of the run's units
// where the others take 53 without that, 55 with it.
constexpr int kPad = 2;
__device__ __forceinline__ int place_of(int k, int shared) { return k + max(0, k - shared) / 6; }
__device__ __forceinline__ int unit_at(int place, int shared, int units) {  // the units before a place
  const int r = max(0, place - shared);
  return min(place - r / 7, units);
}
__device__ __forceinline__ int span_of(int shared, int units) { return place_of(units, shared) + kPad; }

__device__ __forceinline__ void report_arg(const TreeArgs &a) {
  if (a.status != nullptr) atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
}

// The sum of the values of the threads before this one; *total the whole sum.  `warps`: [33] of shared memory.
__device__ __forceinline__ int scan_block(int value, int *warps, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = value;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();  // the last sums have been read
  if (lane == 31) warps[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < (blockDim.x >> 5) ? warps[lane] : 0;
    int run = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    warps[lane] = run - w;
    if (lane == 31) warps[32] = run;
  }
  __syncthreads();
  *total = warps[32];
  return warps[warp] + inc - value;
}

// The last of the indexes lo .. hi - 1 whose value (ascending) is at most x; lo if none is.
template <typename Value>
__device__ __forceinline__ int last_at_most(int lo, int hi, int x, Value value) {
  --hi;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (value(mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One CTA; offsets, lengths and sums stay in shared memory, so that the caller's arrays are read in one round.
__global__ void __launch_bounds__(1024) shared_plan_kernel(const TreeArgs a, const SharedWork w, int tile_rows) {
  extern __shared__ int sm[];
  int *cu = sm, *own_before = cu + a.batch + 1, *cu_group = own_before + a.batch + 1;  // [batch + 1] twice, [groups + 1]
  int *pages_of = cu_group + a.groups + 1, *tile_of = pages_of + a.groups;             // [groups], [groups + 1]
  int4 *group = reinterpret_cast<int4 *>(tile_of + a.groups + 1 + (4 - (2 * a.batch + 3 * a.groups + 4) % 4) % 4);  // [groups]
  __shared__ int warps[33];
  const int threads = blockDim.x, tid = threadIdx.x, G = a.group, tile_tokens = tile_rows / G;
  launch_next();
  // (one round of reads for what `threads` hold: a read behind a store of another's result would wait for that)
  const int c0 = tid <= a.batch ? __ldg(a.cu + tid) : 0, g0 = tid <= a.groups ? __ldg(a.cu_group + tid) : 0;
  const int p0 = tid < a.groups ? __ldg(a.shared_pages + tid) : 0;
  const int n_first = tid < a.batch ? cached_of(a, tid) : 0;
  for (int b = tid; b <= a.batch; b += threads) cu[b] = b == tid ? c0 : __ldg(a.cu + b);
  for (int y = tid; y <= a.groups; y += threads) cu_group[y] = y == tid ? g0 : __ldg(a.cu_group + y);
  for (int y = tid; y < a.groups; y += threads) {
    int p = y == tid ? p0 : __ldg(a.shared_pages + y);
    if (p < 0 || p > a.max_cached >> a.c.page_shift) {
      report_arg(a);
      p = 0;
    }
    pages_of[y] = p;
  }
  for (int x = tid; x < a.batch * a.c.hkv * kOdd; x += threads) w.odd[x] = 0u;
  __syncthreads();
  // groups that do not divide the batch up, or sequences whose tokens do not follow one another: nothing is computed (the
  // host's bounds on the numbers of tiles and units hold for those that do)
  bool bad = false;
  for (int b = tid; b < a.batch; b += threads) bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > a.total;
  for (int y = tid; y < a.groups; y += threads)
    bad |= cu_group[y + 1] < cu_group[y] || (y == 0 && cu_group[y] != 0) || (y == a.groups - 1 && cu_group[y + 1] != a.batch);
  bad = __syncthreads_or(bad) != 0;
  if (bad && tid == 0) report_arg(a);

  // groups
  int carry = 0;
  for (int base = 0; base < a.groups; base += threads) {
    const int y = base + tid;
    int tiles = 0;
    int4 rec = make_int4(0, 0, 0, 0);  // first tile, first token, tokens, the sequence whose table counts
    if (y < a.groups && !bad) {
      const int first = cu_group[y], last = cu_group[y + 1], start = cu[first], end = cu[last];
      if (first < last) {
        int b = first;
        while (b + 1 < last && cu[b + 1] == start) ++b;
        rec = make_int4(0, start, end - start, b);
        tiles = (rec.z + tile_tokens - 1) / tile_tokens;
      }
    }
    int total;
    rec.x = carry + scan_block(tiles, warps, &total);
    if (y < a.groups) {
      group[y] = rec;
      tile_of[y] = rec.x;
    }
    carry += total;
  }
  const int tiles = min(carry, w.max_tiles);
  __syncthreads();

  // sequences
  carry = 0;
  for (int base = 0; base < a.batch; base += threads) {
    const int b = base + tid;
    int units = 0;
    if (b < a.batch) {
      SeqRecord r{0, 0, 0, 0, 0, 0, 0, 0};
      const int n = base == 0 ? n_first : cached_of(a, b);
      if (!bad) {
        const int y = last_at_most(0, a.groups, b, [&](int x) { return cu_group[x]; });
        const int4 g = group[y];
        const Drafts dr = drafts_of(a, b);
        r.start = dr.start;
        r.len = dr.len;
        r.first_page = pages_of[y];
        r.at = r.start - g.y;
        r.tile0 = g.x;
        r.keys = n - (r.first_page << a.c.page_shift);
        if (r.keys < 0) {  // its table does not hold the group's pages
          if (r.len > 0) report_arg(a);
          r.keys = 0;
        }
        if (r.len > 0) units = ((r.keys + kChunk - 1) / kChunk + 1) / 2;
        for (int t = 0; t < r.len; ++t) w.token_start[r.start + t] = r.start;
      }
      w.seqs[b] = r;
    }
    int total;
    const int before = carry + scan_block(units, warps, &total);
    if (b < a.batch) own_before[b] = w.own_before[b] = before;
    carry += total;
  }
  if (tid == 0) own_before[a.batch] = w.own_before[a.batch] = carry;
  __syncthreads();

  // row tiles
  carry = 0;
  int places = 0;
  for (int base = 0; base < tiles; base += threads) {
    const int e = base + tid;
    TileRecord r{};
    if (e < tiles) {
      const int y = last_at_most(0, a.groups, e, [&](int x) { return tile_of[x]; });
      const int4 g = group[y];
      r.tok0 = g.y + (e - g.x) * tile_tokens;
      r.tokens = max(0, min(tile_tokens, g.y + g.z - r.tok0));
      auto start_of = [&](int b) { return cu[b]; };
      r.seq_a = last_at_most(cu_group[y], cu_group[y + 1], r.tok0, start_of);
      r.seq_b = last_at_most(r.seq_a, cu_group[y + 1], r.tok0 + r.tokens - 1, start_of) + 1;
      r.chunks = pages_of[y] << (a.c.page_shift - 6);
      r.shared = (r.chunks + 1) / 2;
      r.table = g.w;
      r.draft0 = max(cu[r.seq_a], r.tok0 - a.max_draft + 1);  // (a longer sequence reads as none)
      r.own = own_before[r.seq_b] - own_before[r.seq_a];
      r.units = r.shared + r.own + (r.tok0 + r.tokens - r.draft0 + kUnit - 1) / kUnit;
    }
    int total;
    r.first = carry + scan_block(r.units, warps, &total);
    carry += total;
    r.place = places + scan_block(e < tiles ? span_of(r.shared, r.units) : 0, warps, &total);
    places += total;
    if (e < tiles) w.tiles[e] = r;
  }
  if (tid == 0) {
    w.totals[0] = carry;
    w.totals[1] = tiles;
    w.totals[2] = 0;
    w.totals[3] = places;
  }
}
size_t plan_smem(int batch, int groups) { return (2 * static_cast<size_t>(batch) + 3 * groups + 7) * 4 + groups * sizeof(int4); }

// ---------------------------------------------------------------- the attention

template <int D, int FMT, bool PAIR>
struct Shared {
  static constexpr bool Q16 = FMT != BSA_CACHE_BF16;
  static constexpr int RB = FMT == BSA_CACHE_BF16 ? 2 * D : FMT == BSA_CACHE_E4M3 ? D : D / 2;
  static constexpr int THREADS = Q16 ? 896 : 640;
  static constexpr int LAUNCH_REGS = Q16 ? 72 : 96;
  static constexpr int REG_LOW = 56, REG_SOFT = Q16 ? 80 : 104, REG_LOAD = 64;
  static_assert(128 * REG_LOW + 512 * REG_SOFT + (Q16 ? 256 * REG_LOAD : 0) <= THREADS * LAUNCH_REGS, "register split");
  static constexpr int SHV = FMT == BSA_CACHE_E4M3 ? 6 : 4;  // 448 * 2^6 and 2688 * 2^4 stay below 2^16
  static constexpr int TH = Q16 ? 4 : 8;                     // log2 of how far the reference may lag the maximum
  static constexpr int SHIFT = Q16 ? 15 - TH : 0;
  static constexpr int NTQ = PAIR ? 2 : 1;
  static constexpr int NCH = D / 64;                         // 128-byte swizzle chunks per row
  static constexpr uint32_t TILE = 128u * D * 2, CHUNK = 128u * 128;
  // K and V tiles, in turn, and staged code tiles: what fills the 227 KB at d = 128.  (8 answers over 128K with 3, 4 tiles
  // and 5, 3 stages of e4m3: 85, 78 us; with 4, 5 and 6, 3 of e2m1: 75, 82.)
  static constexpr int NS = FMT == BSA_CACHE_BF16 ? (PAIR ? 5 : 6) : PAIR ? 3 : 4;
  static constexpr int NG = FMT == BSA_CACHE_BF16 ? 0 : FMT == BSA_CACHE_E4M3 ? 3 : PAIR ? 4 : 6;
  static constexpr uint32_t CODES = 128u * RB;
  static constexpr uint32_t EXPS = CODES, GROUPS = EXPS + 128;    // of a stage: codes, row exponents, group scales
  static constexpr uint32_t STAGE = Q16 ? GROUPS + (FMT == BSA_CACHE_E2M1 ? 128u * (D / 16) : 0) : 0;
  static constexpr uint32_t OFF_Q = 0, OFF_T = NTQ * TILE, OFF_G = OFF_T + NS * TILE, OFF_BAR = OFF_G + NG * STAGE;
  // Q there; K, V of a unit there; V of a unit read (!PAIR); staged codes there, read; S there; P there; O done, read;
  // unit records; K's scale, V's; segment published, done; row scales; last MMA
  static constexpr int B_QF = 0, B_FK = 1, B_FV = B_FK + 4, B_EV = B_FV + 4, B_GF = B_EV + 4, B_GE = B_GF + NG,
                       B_SF = B_GE + NG, B_PR = B_SF + 4, B_OD = B_PR + 2, B_OE = B_OD + 2, B_IN = B_OE + 2,
                       B_IK = B_IN + (Q16 ? 0 : kUnits), B_IV = B_IK + (Q16 ? kUnits : 0), B_SG = B_IV + (Q16 ? kUnits : 0), B_SE = B_SG + kSegs, B_RS = B_SE + kSegs,
                       B_FIN = B_RS + (Q16 ? 2 : 0), NBARS = B_FIN + 1;
  static constexpr uint32_t OFF_MISC = OFF_BAR + (NBARS * 8 + 15) / 16 * 16;  // TMEM address, abort flag
  static constexpr uint32_t OFF_SEG = OFF_MISC + 16;                          // [kSegs] two int4
  static constexpr uint32_t OFF_INFO = OFF_SEG + kSegs * 32;                  // [kUnits] int4
  static constexpr uint32_t OFF_SCALE = OFF_INFO + kUnits * 16;                          // [kUnits] K's scale; oref
  static constexpr uint32_t OFF_RED = OFF_SCALE + (Q16 ? kUnits * 8 : 0);     // [2][2][128] halves' maxima, bf16
  static constexpr uint32_t OFF_ROWS = OFF_RED + 1024;                        // [2][NTQ * 128] row scales of Q
  static constexpr uint32_t OFF_FACTORS = OFF_ROWS + (Q16 ? 2 * NTQ * 128 * 4 : 0);  // [loader warps][128] f16 pairs
  static constexpr uint32_t SMEM = OFF_FACTORS + (Q16 ? kLoadWarps * 128 * 4 : 0) + 1024;
  static_assert(SMEM <= kMaxSmem, "shared memory");
  static constexpr uint32_t F16 = Q16 ? (1u << 7) | (1u << 10) : 0;
  static constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, 128, false) & ~F16;
  static constexpr uint32_t IDESC_O = ptx::idesc_bf16_f32(128, D, true) & ~F16;
  static constexpr int TM_O = 256;  // S_0, S_1, O_0, O_1
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// A run's unit, for the warps that compute: {keys of both chunks | kind << 16, own: first and one past the last of the
// tile's rows that see it | << 16, own: the sequence, drafts: their first token, 0}.
__device__ __forceinline__ int unit_keys(const int4 &u, int half) { return u.x >> (8 * half) & 0xFF; }
__device__ __forceinline__ int unit_kind(const int4 &u) { return u.x >> 16; }

// Takes out of a tile of bf16 values what must not reach rows that do not see it: Inf and NaN (p = 0 does for the rest,
// whatever lies behind the last key).  Of 256 threads `thread` takes every 256th piece of 16 bytes; `odd` gets where they stood (own values), *drafts_odd
// whether there were any (drafted ones).
template <int D>
__device__ __forceinline__ void clean_v(unsigned char *tile, int thread, const int4 &u, uint32_t *odd, int *drafts_odd) {
  constexpr int N = 128 * D * 2 / 16 / 256;
  const bool own = unit_kind(u) == kOwn;
  uint4 *piece = reinterpret_cast<uint4 *>(tile) + thread;  // eight pieces make a row of a swizzle chunk
  uint32_t lost = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) finite_bf16x8(piece[256 * i], lost);
  if (lost == 0u) return;
#pragma unroll 1
  for (int i = 0; i < N; ++i) {
    const uint4 w = piece[256 * i];
    uint32_t bad = 0u;
    const uint4 f = finite_bf16x8(w, bad);
    if (bad == 0u) continue;
    piece[256 * i] = f;
    const int row = (thread >> 3) + 32 * (i & 3);
    if (own && (row & 63) >= unit_keys(u, row >> 6)) continue;  // behind the last key: nobody's
    if (!own) {
      *drafts_odd = 1;
      continue;
    }
    odd[0] = 1u;
    const int dim = (i >> 2) * 64 + ((thread & 7) ^ (thread >> 3 & 7)) * 8;
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    for (int d = 0; d < 8; ++d) {
      const uint32_t b16 = words[d >> 1] >> (16 * (d & 1)) & 0xFFFFu;
      if ((b16 & 0x7F80u) != 0x7F80u) continue;
      const int which = (b16 & 0x7Fu) != 0u ? 2 : b16 >> 15;
      atomicOr(odd + 1 + which * 4 + (dim + d) / 32, 1u << ((dim + d) & 31));
    }
  }
  ptx::fence_proxy_async_smem();
}

// TMEM columns to and from registers.
__device__ __forceinline__ void tmem_ld_cols(uint32_t at, uint32_t (&r)[32]) { ptx::tmem_ld32(at, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t at, uint32_t (&r)[16]) { ptx::tmem_ld16(at, r); }
__device__ __forceinline__ void tmem_st_cols(uint32_t at, const uint32_t (&r)[16]) { ptx::tmem_st16(at, r); }
__device__ __forceinline__ void tmem_st_cols(uint32_t at, const uint32_t (&r)[8]) { ptx::tmem_st8(at, r); }

// The codes among four that are NaN (bit 7 of their bytes); and: marks the dimensions of those in `odd` (.. of +Inf, -Inf,
// NaN), `each` dimensions a code from `dim` on, and takes them out.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int dim, int each, uint32_t *odd) {
  const uint32_t bad = nan_codes(w);
  if (bad == 0u) return w;
  odd[0] = 1u;
#pragma unroll 1
  for (int c = 0; c < 4; ++c)
    if (bad >> (8 * c + 7) & 1u)
      atomicOr(odd + 9 + (dim + c * each) / 32, ((1u << each) - 1u) << ((dim + c * each) & 31));
  return w & ~((bad >> 7) * 0xFFu);
}

// The maps of a bf16 call: q, cached and drafted K and V.
struct SharedMaps {
  CUtensorMap q, k, v, kn, vn;
};

template <int D, int FMT, bool PAIR>
__global__ void __launch_bounds__(Shared<D, FMT, PAIR>::THREADS, 1)
    shared_kernel(const __grid_constant__ SharedMaps maps, const TreeArgs a, const SharedWork wk) {
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
  int4 *seg_rec = reinterpret_cast<int4 *>(sb + C::OFF_SEG);
  int4 *unit_rec = reinterpret_cast<int4 *>(sb + C::OFF_INFO);
  float *scale_k = reinterpret_cast<float *>(sb + C::OFF_SCALE);
  int *ref_v = reinterpret_cast<int *>(scale_k + kUnits);
  uint16_t *red = reinterpret_cast<uint16_t *>(sb + C::OFF_RED);
  float *row_scale = reinterpret_cast<float *>(sb + C::OFF_ROWS);
  // waits watch this CTA's own flag only: *status also carries reports about the arguments
  const Ctl ctl{abort_flag, nullptr};
  // a whole warp waits, and goes on or gives up together
  auto wait_warp = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait_parked(bar(i), parity, ctl)) != 0; };
  auto arrive_warp = [&](int i) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar(i));
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, G = a.group;

  if (tid == 0) {
    for (int x = 0; x < C::NBARS; ++x) {
      // arrivals: 1 of a commit, the producer or a copy's announcement; 4 of the loader warps of K or of V; 8 of all of
      // them or a lane's warps; 16 of both lanes'; P_0 has one more for V and the next K
      uint32_t count = 1;
      if (Q16 && (x == C::B_QF || (x >= C::B_RS && x < C::B_FIN)))
        count = kLoadWarps;
      else if (Q16 && ((x >= C::B_FK && x < C::B_EV) || (x >= C::B_GE && x < C::B_SF)))
        count = kLoadWarps / 2;
      else if ((x >= C::B_PR && x < C::B_OD) || (x >= C::B_OE && x < C::B_IN))
        count = PAIR && x == C::B_PR ? 9 : 8;
      else if (x >= C::B_SE && x < C::B_RS)
        count = 16;
      ptx::mbar_init(bar(x), count);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  if (!Q16 && tid == 64) {
    ptx::tma_prefetch_desc(&maps.q);
    ptx::tma_prefetch_desc(&maps.k);
    ptx::tma_prefetch_desc(&maps.v);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  after_previous_kernel();  // the plan
  launch_next();
  // This CTA's run
  const int units_all = wk.totals[0] * a.c.hkv, tiles_all = wk.totals[1], places = wk.totals[3] * a.c.hkv;
  const int W = (places + kSms - 1) / kSms;
  // the units before a place
  auto units_before = [&](int place) {
    if (place >= places) return units_all;
    int e = 0, hi = tiles_all;  // the last row tile that begins at or before it, 32 looked at at a time
    while (hi - e > 1) {
      const int step = (hi - e + 31) / 32, at = e + lane * step;
      const bool before = at < hi && wk.tiles[at].place * a.c.hkv <= place;
      const int k = __popc(__ballot_sync(0xffffffffu, before));
      hi = min(hi, e + k * step);
      e += (k - 1) * step;
    }
    const TileRecord t = wk.tiles[e];
    const int span = span_of(t.shared, t.units), off = place - t.place * a.c.hkv, g = off / span;
    return t.first * a.c.hkv + g * t.units + unit_at(off - g * span, t.shared, t.units);
  };
  const int x0 = tiles_all > 0 ? units_before(cta * W) : 0, x1 = tiles_all > 0 ? units_before(cta * W + W) : 0, nu = x1 - x0;

  // S of unit n (of lane t) is there.  It is also the sign that K of the unit is read, and, where both row tiles take
  // every unit, V of the unit before: the issuing thread has few cycles for signs of their own.
  auto s_bar = [&](int t, uint32_t n) { return C::B_SF + (PAIR ? 2 * t + static_cast<int>(n & 1) : static_cast<int>(n & 3)); };
  auto s_parity = [&](uint32_t n) { return (PAIR ? n >> 1 : n >> 2) & 1; };
  // The barrier and parity after which tile z may be written (z >= NS; tiles are K and V of the units in turn).
  auto free_bar = [&](uint32_t z, uint32_t &parity) {
    const uint32_t before = z - C::NS, m = before >> 1;
    if (!PAIR && (before & 1) != 0) {
      parity = (m >> 2) & 1;
      return C::B_EV + static_cast<int>(m & 3);
    }
    const uint32_t n = m + (PAIR ? before & 1 : 0);
    parity = s_parity(n);
    return s_bar(1, n);
  };
  // The barrier on which tile z is announced (in phase z >> 3).
  auto full_bar = [&](uint32_t z) { return ((z & 1) == 0 ? C::B_FK : C::B_FV) + static_cast<int>(z >> 1 & 3); };

  if (warp < 4) {
    ptx::setmaxnreg_dec<C::REG_LOW>();
    if (warp == 0 && nu > 0) {
      // ================================================================ producer
      // A segment's record: {units, first token, tokens, KV head}, {1 if the CTA has all of the row tile's units | 2 if
      // it does not begin the run, 0, 0, 0}.
      bool ok = true;
      int e = 0, n = 0, seg = 0;
      uint32_t tiles_sent = 0, stages_sent = 0;
      const int sub_mask = (1 << (a.c.page_shift - 6)) - 1;
      {  // the last row tile that begins at or before x0, 32 looked at at a time
        int hi = wk.totals[1];
        while (hi - e > 1) {
          const int step = (hi - e + 31) / 32, at = e + lane * step;
          const bool before = at < hi && wk.tiles[at].first * a.c.hkv <= x0;
          const int k = __popc(__ballot_sync(0xffffffffu, before));
          hi = min(hi, e + k * step);
          e += (k - 1) * step;
        }
      }
      // the run's units, 32 at a time, one per lane and a batch ahead
      struct Unit {
        int p0, p1, sub, keys, rows, what;  // pages of both chunks (-1: none); the record's fields
        int tok0, tokens, g, k, left;       // the tile's tokens; KV head; the unit's place, and how many there are from it on
      };
      auto look_up = [&](int i) {
        Unit u{-1, -1, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        const bool in = i < nu;
        const int x = x0 + min(i, nu - 1);
        const int e0 = e;
        TileRecord tr = wk.tiles[e];
        while (x >= (tr.first + tr.units) * a.c.hkv) tr = wk.tiles[++e];
        const int off = x - tr.first * a.c.hkv;
        u.g = off / tr.units;
        u.k = off - u.g * tr.units;
        u.left = tr.units - u.k;
        u.tok0 = tr.tok0;
        u.tokens = tr.tokens;
        const int own = u.k - tr.shared, seqs = tr.seq_b - tr.seq_a, own0 = wk.own_before[tr.seq_a];
        const bool is_own = own >= 0 && own < tr.own;
        // the sequence of an own unit: in one tile of few sequences a lane holds each one's units before it
        int b = tr.seq_a;
        if (__all_sync(0xffffffffu, e == e0 && seqs <= 32)) {
          const int before = wk.own_before[min(tr.seq_a + lane, tr.seq_b)] - own0;
          int at = 0;
#pragma unroll 1
          for (int step = 16; step > 0; step >>= 1) {
            const int there = __shfl_sync(0xffffffffu, before, min(at + step, 31));
            if (at + step < seqs && there <= own) at += step;
          }
          b += at;
        } else if (is_own) {
          b = last_at_most(tr.seq_a, tr.seq_b, own + own0, [&](int j) { return __ldg(wk.own_before + j); });
        }
        int seq = tr.table, c = 2 * u.k, first_page = 0;
        if (own < 0) {
          u.keys = kChunk | (c + 1 < tr.chunks ? kChunk << 8 : 0) | kShared << 16;
        } else if (is_own) {
          const SeqRecord r = wk.seqs[b];
          seq = b;
          first_page = r.first_page;
          c = 2 * (own - (wk.own_before[b] - own0));
          const int n0 = max(0, min(kChunk, r.keys - c * kChunk)), n1 = max(0, min(kChunk, r.keys - (c + 1) * kChunk));
          u.keys = n0 | n1 << 8 | kOwn << 16;
          const int t0 = max(r.start, tr.tok0) - tr.tok0, t1 = min(r.start + r.len, tr.tok0 + tr.tokens) - tr.tok0;
          u.rows = max(0, t0) * G | max(0, t1) * G << 16;
          u.what = b;
        } else {
          u.what = tr.draft0 + (own - tr.own) * kUnit;
          const int left = tr.tok0 + tr.tokens - u.what;
          u.keys = max(0, min(kChunk, left)) | max(0, min(kChunk, left - kChunk)) << 8 | kDraft << 16;
        }
        if (in && u.keys >> 16 != kDraft) {
          const int32_t *entry = a.table + static_cast<size_t>(seq) * a.table_stride + first_page + (c >> (a.c.page_shift - 6));
          u.sub = c & sub_mask;
          u.p0 = __ldg(entry);
          if ((u.keys >> 8 & 0xFF) != 0) u.p1 = sub_mask == 0 ? __ldg(entry + 1) : u.p0;
        }
        e = __shfl_sync(0xffffffffu, e, 31);
        return u;
      };
      // entries that name no page: their chunk has no keys
      auto checked = [&](Unit &u, bool in) {
        if (u.keys >> 16 == kDraft) return;
        const bool bad0 = (u.keys & 0xFF) != 0 && (u.p0 < 0 || u.p0 >= a.c.pages);
        const bool bad1 = (u.keys >> 8 & 0xFF) != 0 && (u.p1 < 0 || u.p1 >= a.c.pages);
        if (bad0) u.p0 = -1, u.keys &= ~0xFF;
        if (bad1) u.p1 = -1, u.keys &= ~0xFF00;
        if (in && (bad0 || bad1)) report_arg(a);
      };
      // With two row tiles and an odd ring, tiles of K and V of a unit j take the places of V(j - 3) and K(j - 2), which one
      // sign frees: S_1(j - 2).  V does not wait for it again: S_1(j), which needs K(j) alone, may by then have completed
      // that barrier once more, and the parity would be that of another phase.  V((NS - 1) / 2) is the first that needs a
      // place, and its K none: it takes S_1(0), or S_1(1) where that barrier has gone on (its own does so with the product
      // that needs this V).
      static_assert(Q16 || !PAIR || C::NS % 2 == 1, "V's place becomes free with K's");
      auto first_place = [&]() -> bool {
        const uint64_t t0 = ptx::globaltimer_ns();
        for (;;) {
          if (try_wait_parked(bar(s_bar(1, 0)), 0) || is_complete(bar(s_bar(1, 1)), 0)) return true;
          if (*ctl.abort_flag) return false;
          if (ptx::globaltimer_ns() - t0 > wait::kWaitTimeoutNs) {
            wait::report(ctl, BSA_ERR_DEVICE_TIMEOUT);
            return false;
          }
        }
      };
      Unit now = look_up(lane), next{};
      for (; ok && n < nu; ++n) {
        if (n % 32 == 0) {
          if (n > 0) now = next;
          if (n + 32 < nu) next = look_up(n + 32 + lane);
          checked(now, n + lane < nu);
        }
        const int from = n & 31;
        const int g = __shfl_sync(0xffffffffu, now.g, from), k = __shfl_sync(0xffffffffu, now.k, from);
        const bool begins = n == 0 || k == 0;  // a segment
        const int tok0 = __shfl_sync(0xffffffffu, now.tok0, from);
        if (begins) {
          const int tokens = __shfl_sync(0xffffffffu, now.tokens, from);
          const int left = __shfl_sync(0xffffffffu, now.left, from);
          if (seg >= kSegs && !(ok = wait_warp(C::B_SE + seg % kSegs, (seg / kSegs - 1) & 1))) break;
          if (lane == 0) {
            seg_rec[2 * (seg % kSegs)] = make_int4(min(left, nu - n), tok0, tokens, g);
            // (it begins the run: nothing lies before it; the CTA has all its units: nor does any of its own)
            seg_rec[2 * (seg % kSegs) + 1] = make_int4((k == 0 && left <= nu - n ? 1 : 0) | (n == 0 ? 0 : 2), 0, 0, 0);
            ptx::mbar_arrive(bar(C::B_SG + seg % kSegs));
          }
          ++seg;
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
        }
        {
          const int p0 = __shfl_sync(0xffffffffu, now.p0, from), p1 = __shfl_sync(0xffffffffu, now.p1, from);
          const int keys = __shfl_sync(0xffffffffu, now.keys, from), rows = __shfl_sync(0xffffffffu, now.rows, from);
          const int what = __shfl_sync(0xffffffffu, now.what, from), sub = __shfl_sync(0xffffffffu, now.sub, from);
          if (lane == 0) {
            const int kind = keys >> 16;
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const uint32_t z = 2u * static_cast<uint32_t>(n) + kv;
              if constexpr (!Q16) {
                const uint32_t s = z % C::NS;
                uint32_t parity = 0;
                if (PAIR && kv == 1) {  // (K has waited for the sign of both, but the first V to need a place)
                  if (z == C::NS && !(ok = first_place())) break;
                } else if (z >= C::NS) {
                  const int fb = free_bar(z, parity);
                  if (!(ok = wait_parked(bar(fb), parity, ctl))) break;
                }
                if (kv == 0) {
                  unit_rec[n % kUnits] = make_int4(keys, rows, what, 0);
                  ptx::mbar_arrive(bar(C::B_IN + n % kUnits));
                }
                const uint32_t dst = base + C::OFF_T + s * C::TILE, f = bar(full_bar(z));
                ptx::mbar_arrive_expect_tx(f, C::TILE);
                if (kind == kDraft) {
                  const CUtensorMap *map = kv == 0 ? &maps.kn : &maps.vn;
                  for (int c = 0; c < C::NCH; ++c) tma_load_3d(dst + c * C::CHUNK, map, f, c * 64, g, what);
                } else {
                  const CUtensorMap *map = kv == 0 ? &maps.k : &maps.v;
                  // a chunk that is not there lies outside the tensor, and comes as zeros
                  const int none = a.c.pages * a.c.hkv;
                  const int row0 = p0 >= 0 ? p0 * a.c.hkv + g : none, row1 = p1 >= 0 ? p1 * a.c.hkv + g : none;
                  for (int c = 0; c < C::NCH; ++c) {
                    tma_load_3d(dst + c * C::CHUNK, map, f, c * 64, sub * kChunk, row0);
                    if (sub_mask == 0) tma_load_3d(dst + c * C::CHUNK + kChunk * 128, map, f, c * 64, 0, row1);
                  }
                }
                tiles_sent = z + 1;
                if (kv == 0 && begins) {  // (behind K, which the segment before may wait for)
                  if (n > 0 && !(ok = wait_parked(bar(s_bar(1, n - 1)), s_parity(n - 1), ctl))) break;  // its last S
                  ptx::mbar_arrive_expect_tx(bar(C::B_QF), C::NTQ * C::TILE);
                  for (int t = 0; t < C::NTQ; ++t)
                    for (int c = 0; c < C::NCH; ++c)
                      tma_load_3d(base + C::OFF_Q + t * C::TILE + c * C::CHUNK, &maps.q, bar(C::B_QF), c * 64, g * G,
                                  tok0 + t * (kRows / G));
                }
              } else {
                const uint32_t s = z % C::NG, round = z / C::NG;
                if (round > 0 && !(ok = wait_parked(bar(C::B_GE + s), (round - 1) & 1, ctl))) break;
                if (kv == 0) unit_rec[n % kUnits] = make_int4(keys, rows, what, 0);
                constexpr int PER = FMT == BSA_CACHE_E4M3 ? 1 : 1 + D / 16;
                const uint8_t *codes = kv == 0 ? a.k_codes : a.v_codes, *scales = kv == 0 ? a.k_scales : a.v_scales;
                const uint32_t dst = base + C::OFF_G + s * C::STAGE, f = bar(C::B_GF + s);
                ptx::mbar_arrive_expect_tx(f, ((p0 >= 0 ? 1u : 0u) + (p1 >= 0 ? 1u : 0u)) * (C::STAGE / 2));
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
      }
      if (*abort_flag && lane == 0) {
        // let copies in flight land before the CTA's shared memory is released (a barrier that lacks an arrival never
        // completes: its wait runs out)
        if constexpr (!Q16) {
          if (seg > 0) drain_bar(bar(C::B_QF), (seg - 1) & 1);
          for (uint32_t z = tiles_sent > C::NS ? tiles_sent - C::NS : 0; z < tiles_sent; ++z)
            drain_bar(bar(full_bar(z)), z >> 3 & 1);
        } else {
          constexpr uint32_t RING = C::NG > 0 ? C::NG : 1;
          for (uint32_t z = stages_sent > RING ? stages_sent - RING : 0; z < stages_sent; ++z)
            drain_bar(bar(C::B_GF + z % RING), (z / RING) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 1 && lane == 0 && nu > 0) {
      // ================================================================ MMA issuer
      // Its instructions are what the tensor core waits for (a product of 16 keys or dimensions takes 64 cycles, and every
      // wait, commit or look costs 70 to 150 in which few products are queued), so it has one commit a row tile and
      // unit, and one wait.
      auto wait_for = [&](int i, uint32_t parity) { return wait_parked(bar(i), parity, ctl); };
      // descriptors differ in the address field of the low word alone
      const uint64_t dq0 = ptx::sdesc_sw128(base + C::OFF_Q, 16, 1024);
      const uint64_t dk0 = ptx::sdesc_sw128(base + C::OFF_T, 16, 1024);
      const uint64_t dv0 = ptx::sdesc_sw128(base + C::OFF_T, C::CHUNK, 1024);
      constexpr uint32_t TILE16 = C::TILE >> 4;
      auto issue_s = [&](int t, uint32_t ks, uint32_t n) {  // (ks: K's tile in the ring, in units of 16 bytes)
        const uint64_t dq = dq0 + (PAIR && t == 1 ? TILE16 : 0);
        const uint64_t dk = dk0 + ks;
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
        ptx::mma_commit(bar(s_bar(t, n)));
      };
      uint32_t pv_count[2] = {0, 0}, lane_segs[2] = {0, 0};  // P V products of each lane, segments in which it had a unit
      // `first`: the lane's first of a segment, which overwrites O: the last segment's must have been read
      auto issue_pv = [&](int t, uint32_t vs, bool first) -> bool {
        const uint64_t dv = dv0 + vs;
        const uint32_t dst = tmem + C::TM_O + t * 128, src = tmem + t * 128;
        const uint32_t count = t == 0 ? pv_count[0]++ : pv_count[1]++;
        if (first) {
          const uint32_t k = t == 0 ? lane_segs[0]++ : lane_segs[1]++;
          if (k > 0 && !wait_for(C::B_OE + t, (k - 1) & 1)) return false;
        }
        if (!wait_for(C::B_PR + t, count & 1)) return false;
        ptx::tc_fence_after();
        // 16 keys each: P of a half lies over the first of its columns
        mma_ts_at<0, 0>(dst, src, dv, C::IDESC_O, first ? 0u : 1u);
        mma_ts_at<8, 128>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<16, 256>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<24, 384>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<64, 512>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<72, 640>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<80, 768>(dst, src, dv, C::IDESC_O, 1u);
        mma_ts_at<88, 896>(dst, src, dv, C::IDESC_O, 1u);
        return true;
      };
      auto tile_there = [&](uint32_t z) { return wait_for(full_bar(z), z >> 3 & 1); };
      constexpr uint32_t RING16 = C::NS * TILE16;
      auto next_tile = [](uint32_t at, uint32_t by) { return at + by >= RING16 ? at + by - RING16 : at + by; };
      uint32_t n = 0, ks = 0, vs = TILE16, v_last = 0;  // tiles of the unit's K and V, and of the last step's V
      int seg = 0, left = nu;
      bool ok = !PAIR || tile_there(0);
      for (; ok && left > 0; ++seg) {
        if (!(ok = wait_for(C::B_SG + seg % kSegs, (seg / kSegs) & 1))) break;
        const int units = seg_rec[2 * (seg % kSegs)].x;
        left -= units;
        if (!(ok = wait_for(C::B_QF, seg & 1))) break;
        ptx::tc_fence_after();
        // S_t(n) overwrites what P_t V(n - 1) reads: MMAs of one thread run in the order of issue
        if constexpr (PAIR) {
          for (int i = 0; i < units; ++i, ++n) {
            issue_s(0, ks, n);
            if (i > 0 && !(ok = issue_pv(1, v_last, i == 1))) break;
            issue_s(1, ks, n);
            // (P_0's sign says as well that V of this unit and K of the next are there)
            if (!(ok = issue_pv(0, vs, i == 0))) break;
            v_last = vs;
            ks = next_tile(ks, 2 * TILE16);
            vs = next_tile(vs, 2 * TILE16);
          }
          if (!ok) break;
          ptx::mma_commit(bar(C::B_OD));
          if (!(ok = issue_pv(1, v_last, units == 1))) break;
          ptx::mma_commit(bar(C::B_OD + 1));
        } else {
#pragma unroll 1
          for (int i = 0; i <= units; ++i) {  // S of unit i, P V of unit i - 1
            if (i < units) {
              if (!(ok = tile_there(2 * n))) break;
              ptx::tc_fence_after();
              issue_s(i & 1, ks, n);
            }
            if (i > 0) {
              const uint32_t m = n - 1;
              if (!(ok = tile_there(2 * m + 1))) break;
              if (!(ok = issue_pv((i - 1) & 1, v_last, i < 3))) break;
              ptx::mma_commit(bar(C::B_EV + static_cast<int>(m & 3)));
              if (i >= units - 1) ptx::mma_commit(bar(C::B_OD + ((i - 1) & 1)));
            }
            v_last = vs;
            if (i < units) {
              ++n;
              ks = next_tile(ks, 2 * TILE16);
              vs = next_tile(vs, 2 * TILE16);
            }
          }
        }
      }
      if (!ok) {
        // every MMA issued so far must finish before TMEM is released
        ptx::mma_commit(bar(C::B_FIN));
        drain_bar(bar(C::B_FIN), 0);
      }
    } else if (PAIR && warp == 2 && lane == 0) {
      // ================================================================ V and the next K, as an arrival at P_0
      for (uint32_t z = 1; z < 2u * static_cast<uint32_t>(nu); z += 2) {
        if (!wait_parked(bar(full_bar(z)), z >> 3 & 1, ctl)) break;
        if (z + 1 < 2u * static_cast<uint32_t>(nu) && !wait_parked(bar(full_bar(z + 1)), (z + 1) >> 3 & 1, ctl)) break;
        ptx::mbar_arrive(bar(C::B_PR));
        if (!wait_parked(bar(C::B_PR), z >> 1 & 1, ctl)) break;  // (the next arrival belongs to the next phase)
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
    const int row = (PAIR ? t : 0) * kRows + r;  // of the tile (or pair of tiles)
    bool ok = true;
    uint32_t n = 0, lane_segs = 0;  // units of the run; segments in which this lane had one
    int seg = 0;
    for (int x = x0; ok && x < x1; ++seg) {
      if (!(ok = wait_warp(C::B_SG + seg % kSegs, (seg / kSegs) & 1))) break;
      const int units = seg_rec[2 * (seg % kSegs)].x;
      x += units;
      float rs = a.scale_log2;
      if constexpr (Q16) {
        if (PAIR || units > t) {
          if (!(ok = wait_warp(C::B_RS + (seg & 1), (seg >> 1) & 1))) break;
          rs *= row_scale[((seg & 1) * C::NTQ + (PAIR ? t : 0)) * 128 + r];
        }
      }
      const int4 rt = seg_rec[2 * (seg % kSegs)];  // (.y: the tile's first token)
      const int tok = rt.y + row / G, seq_start = row / G < rt.z ? __ldg(wk.token_start + tok) : INT32_MAX;
      float m = -INFINITY, l = 0.f;
      int oref = 0, done = 0;  // O's unit (8- and 4-bit caches); units of this lane in the segment
      for (int i = 0; i < units; ++i, ++n) {
        if (!PAIR && (i & 1) != t) continue;
        // (over codes K's scale comes after the copies, and they after the record)
        if (!(ok = wait_warp((Q16 ? C::B_IK : C::B_IN) + n % kUnits, (n / kUnits) & 1))) break;
        const int4 u = unit_rec[n % kUnits];
        // which of the thread's 64 keys the row sees
        uint32_t see0 = 0xffffffffu, see1 = 0xffffffffu;
        bool on = true;  // it sees some
        const bool whole_chunk = unit_keys(u, hf) == kChunk && unit_kind(u) != kDraft;
        const bool masked = !whole_chunk;
        if (whole_chunk) {
          if (unit_kind(u) == kOwn) on = row >= (u.y & 0xFFFF) && row < u.y >> 16;
        } else {
          const int keys = unit_keys(u, hf);
          int from = 0, to = keys;  // keys from .. to - 1
          if (unit_kind(u) == kOwn) {
            if (row < (u.y & 0xFFFF) || row >= u.y >> 16) to = 0;
          } else if (unit_kind(u) == kDraft) {
            const int first = u.z + hf * kChunk;
            to = 0;
            if (seq_start != INT32_MAX) {
              if (a.parents == nullptr) {
                from = max(0, seq_start - first);
                to = max(0, min(keys, tok - first + 1));
              } else {
                see0 = see1 = 0u;
                for (int p = tok - seq_start; p >= 0 && seq_start + p >= first; p = parent_of(a, seq_start, p)) {
                  const int k = seq_start + p - first;
                  if (k < 32) see0 |= 1u << k;
                  else if (k < 64) see1 |= 1u << (k - 32);
                }
                to = -1;
              }
            }
          }
          if (to >= 0) {  // (bits from .. to - 1 of 64)
            auto below = [](int k) { return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u; };
            see0 = below(to) & ~below(from);
            see1 = below(to - 32) & ~below(from - 32);
          }
          on = (see0 | see1) != 0u;
        }
        const bool any = __any_sync(0xffffffffu, on);  // of the warp's rows
        float scl = rs;
        int oref_new = 0;
        if constexpr (Q16) {
          if (!(ok = wait_warp(C::B_IV + n % kUnits, (n / kUnits) & 1))) break;
          // never 0, so that a masked -inf stays one (the logits below it are 0 to any precision)
          scl = fmaxf(scl * scale_k[n % kUnits], 1e-37f);
          oref_new = ref_v[n % kUnits];
        }
        if (!(ok = wait_warp(s_bar(t, n), s_parity(n)))) break;
        ptx::tc_fence_after();
        // The row's maximum first, then the logits again, 32 at a time (the first half stays in registers).  Beside the
        // loaders of codes 16 at a time and loops stay loops: what all the warps of a scheduler run has to fit its
        // instruction cache.
        uint32_t sr[Q16 ? 16 : 32];
        float top = -INFINITY;
        if constexpr (Q16) {
          if (any && !masked) {
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
              uint32_t unused[32];
              float mx;
              ptx::tmem_ld32_max(tS + c, unused, mx);
              ptx::tmem_wait_ld();
              top = fmaxf(top, mx);
            }
            if (!on) top = -INFINITY;
          } else if (any) {  // (written back masked, so that the loop below knows no masks)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              ptx::tmem_ld16(tS + c * 16, sr);
              ptx::tmem_wait_ld();
              const uint32_t see = (c < 2 ? see0 : see1) >> (16 * (c & 1));
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if (!((see >> e) & 1u)) sr[e] = 0xFF800000u;
                top = fmaxf(top, __uint_as_float(sr[e]));
              }
              tmem_st_cols(tS + c * 16, sr);
            }
            ptx::tmem_wait_st();
          }
        } else {
          if (any) {
#pragma unroll
            for (int c = 1; c >= 0; --c) {
              float mx;
              ptx::tmem_ld32_max(tS + c * 32, sr, mx);
              ptx::tmem_wait_ld();
              if (masked) {
                const uint32_t see = c == 0 ? see0 : see1;
                mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  if (!((see >> e) & 1u)) sr[e] = 0xFF800000u;
                  mx = fmaxf(mx, __uint_as_float(sr[e]));
                }
              }
              top = fmaxf(top, mx);
            }
            if (!on) top = -INFINITY;
          }
        }
        // the maximum of both halves: each half's rounded up to bf16 (any upper bound is a valid reference, and
        // both halves then hold the same value).  The slot is written again only after the partner has released P,
        // which the lane's next S waits for.
        uint32_t up = __float_as_uint(top);
        if ((up & 0xFFFFu) != 0u && !(up >> 31)) up += 0x10000u;
        *mine_max = static_cast<uint16_t>(up >> 16);
        ptx::named_barrier(pair_bar, 64);
        const float mx = fmaxf(__uint_as_float(up & 0xFFFF0000u), __uint_as_float(static_cast<uint32_t>(*other_max) << 16));
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
        const float bias = static_cast<float>(C::SHIFT) - (m == -INFINITY ? 0.f : m);
        uint64_t acc[2] = {0ull, 0ull};
        const uint64_t scl2 = ptx::f32x2(scl, scl), bias2 = ptx::f32x2(bias, bias);
        constexpr int W = Q16 ? 16 : 32, UNROLL = Q16 ? 1 : 2;
#pragma unroll UNROLL
        for (int c = 0; c < 64 / W; ++c) {
          uint32_t pk[W / 2];
#pragma unroll
          for (int e = 0; e < W / 2; ++e) pk[e] = 0u;
          if (any) {
            if (Q16 || c == 1) {
              tmem_ld_cols(tS + c * W, sr);
              ptx::tmem_wait_ld();
              if (!Q16 && masked) {
#pragma unroll
                for (int e = 0; e < W; ++e)
                  if (!((see1 >> e) & 1u)) sr[e] = 0xFF800000u;
              }
            }
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
              const uint64_t y =
                  ptx::fma_f32x2(ptx::f32x2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), scl2, bias2);
              float y0, y1;
              ptx::f32x2_split(y, y0, y1);
              const float p0 = ptx::ex2_approx(y0), p1 = ptx::ex2_approx(y1);
              acc[e & 1] = ptx::add_f32x2(acc[e & 1], ptx::f32x2(p0, p1));
              pk[e] = Q16 ? pack_f16x2(p0, p1) : ptx::pack_bf16x2(p0, p1);
            }
            if (!on) {  // (whatever the logits of another sequence's keys are)
#pragma unroll
              for (int e = 0; e < W / 2; ++e) pk[e] = 0u;
            }
          }
          tmem_st_cols(tS + c * (W / 2), pk);
          if (c == 0 && __any_sync(0xffffffffu, resc)) {
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
        }
        if constexpr (!Q16) {
          // V of a unit with masked places: Inf and NaN become 0.  (By the first lane to use it.)
          if (unit_kind(u) != kShared && (!PAIR || t == 0)) {
            if (!(ok = wait_warp(full_bar(2 * n + 1), (n >> 2) & 1))) break;
            clean_v<D>(sb + C::OFF_T + (2 * n + 1) % C::NS * C::TILE, ((warp - kSoftWarp) & 7) * 32 + lane, u,
                       wk.odd + (static_cast<size_t>(u.z) * a.c.hkv + seg_rec[2 * (seg % kSegs)].w) * kOdd, wk.totals + 2);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        arrive_warp(C::B_PR + t);
        float s4[4];
        ptx::f32x2_split(acc[0], s4[0], s4[1]);
        ptx::f32x2_split(acc[1], s4[2], s4[3]);
        constexpr float unshift = 1.f / (1 << C::SHIFT);
        l = fmaf(on ? (s4[0] + s4[1]) + (s4[2] + s4[3]) : 0.f, unshift, l * factor);
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
      const int4 ra = seg_rec[2 * (seg % kSegs)], rb = seg_rec[2 * (seg % kSegs) + 1];  // (their place is taken after B_SE)
      const bool whole = (rb.x & 1) != 0, live = row / G < ra.z;
      const size_t out = static_cast<size_t>(ra.y + row / G) * a.hq + ra.w * G + row % G;
      const size_t slot = 2 * (2 * static_cast<size_t>(cta) + (rb.x >> 1)) + t;
      float unit_f = 1.f;
      if constexpr (Q16) unit_f = exp2f(static_cast<float>(oref - 127 - C::SHV - C::SHIFT));
      if (done > 0) {
        float4 *po = reinterpret_cast<float4 *>(wk.part_o) + (slot * (D / 4) + hf * (D / 8)) * kRows + r;
        float4 *ro = reinterpret_cast<float4 *>(wk.row_o + ((PAIR ? 0 : t) * wk.rows + out) * D) + hf * (D / 8);
#pragma unroll 1
        for (int q = 0; q < D / 64; ++q) {
          uint32_t ov[32];
          ptx::tmem_ld32(tO + q * 32, ov);
          ptx::tmem_wait_ld();
          if (q == D / 64 - 1) {  // O may be overwritten
            ptx::tc_fence_before();
            arrive_warp(C::B_OE + t);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 v = make_float4(__uint_as_float(ov[4 * e]) * unit_f, __uint_as_float(ov[4 * e + 1]) * unit_f,
                                         __uint_as_float(ov[4 * e + 2]) * unit_f, __uint_as_float(ov[4 * e + 3]) * unit_f);
            if (!whole) po[(8 * q + e) * kRows] = v;
            else if (live) ro[8 * q + e] = v;
          }
        }
      }
      if (!whole) wk.part_ml[(slot * 2 + hf) * kRows + r] = make_float2(m, l);
      else if (live) wk.row_ml[((PAIR ? 0 : t) * 2 + hf) * wk.rows + out] = make_float2(m, l);
      arrive_warp(C::B_SE + seg % kSegs);
    }
  } else if constexpr (Q16) {
    // ================================================================ loaders
    ptx::setmaxnreg_dec<C::REG_LOAD>();
    const int lt = tid - kLoadWarp * 32;
    // four warps for K, four for V; a thread takes pieces of 16 bytes of rows STEP apart
    constexpr int PP = C::RB / 16, ST = kLoadWarps * 16, STEP = ST / PP, LT = 2 * ST;
    const int kv = lt / ST, st = lt % ST;
    // Eight lanes read and write eight different banks: with eight pieces a row they take four of one row and the other
    // four of the next (whose units stand in the other order).
    const int p = PP == 8 ? (st & 3) | ((st >> 2 ^ st >> 3) & 1) << 2 : st % PP;
    const int r0 = PP == 8 ? st >> 4 << 1 | (st >> 2 & 1) : st / PP;
    uint32_t *factors = reinterpret_cast<uint32_t *>(sb + C::OFF_FACTORS) + (warp - kLoadWarp) * 128;  // of the tile's rows
    bool ok = true;
    uint32_t n = 0;
    int seg = 0;
    for (int x = x0; ok && x < x1; ++seg) {
      if (!(ok = wait_warp(C::B_SG + seg % kSegs, (seg / kSegs) & 1))) break;
      const int4 ra = seg_rec[2 * (seg % kSegs)];
      const int units = ra.x, g = ra.w;
      x += units;
      // ---- Q: rows as f16, the largest element of each brought to [2^14, 2^15)
      if (n > 0 && !(ok = wait_warp(s_bar(1, n - 1), s_parity(n - 1)))) break;  // (the last S of the segment before)
      constexpr int LPR = D / 8, RS = LT / LPR, U = 4;  // threads of a row, rows of a step, steps in flight
#pragma unroll 1
      for (int q0 = 0; q0 < C::NTQ * kRows; q0 += RS * U) {
        uint4 v[U];
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int row = q0 + e * RS + lt / LPR, tok = row / G;
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (tok < ra.z)
            v[e] = __ldg(reinterpret_cast<const uint4 *>(
                a.q + (static_cast<size_t>(ra.y + tok) * a.hq + g * G + row % G) * D + lt % LPR * 8));
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
        // ---- the unit's scales, K's and V's (its record was written before the copies were announced)
        const uint32_t z = 2 * n + kv, s = z % C::NS;
        if (!(ok = wait_warp(C::B_GF + z % C::NG, (z / C::NG) & 1))) break;
        const int4 u = unit_rec[n % kUnits];
        const int n0 = unit_keys(u, 0), n1 = unit_keys(u, 1), kind = unit_kind(u);
        const size_t dstride = static_cast<size_t>(a.c.hkv) * D;
        const uint16_t *drafted = (kv == 0 ? a.k_new : a.v_new) + (static_cast<size_t>(kind == kDraft ? u.z : 0) * a.c.hkv + g) * D;
        int top;
        uint32_t exps = 0u;  // of the lane's four rows
        if (kind == kDraft) {  // the largest finite element lands in [2^14, 2^15); every warp looks at all rows
          float am = 0.f;
          uint32_t lost = 0u;
#pragma unroll 4
          for (int c = lane; c < (n0 + n1) * LPR; c += 32)
            am = fmaxf(am, amax8(finite_bf16x8(
                               __ldg(reinterpret_cast<const uint4 *>(drafted + (c / LPR) * dstride + c % LPR * 8)), lost)));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
          top = max(8, (__float_as_int(am) >> 23) + C::SHV - 14);
        } else {
          const uint32_t w = *reinterpret_cast<const uint32_t *>(sb + C::OFF_G + (z % C::NG) * C::STAGE + C::EXPS + lane * 4);
          const int live = (lane < 16 ? n0 : n1) - 4 * (lane & 15);  // of the lane's four rows
          exps = live >= 4 ? w : live <= 0 ? 0u : w & ((1u << (8 * live)) - 1u);
          const uint32_t m = __vmaxu4(exps, exps >> 16);
          top = static_cast<int>(__reduce_max_sync(0xffffffffu, max(m & 0xFFu, (m >> 8) & 0xFFu)));
        }
        if (kv == 1) top = oref = max(oref, top);
        if (st == 0) {
          if (kv == 0) scale_k[n % kUnits] = exp2f(static_cast<float>(top - C::SHV - 127));
          else ref_v[n % kUnits] = top;
          ptx::mbar_arrive(bar((kv == 0 ? C::B_IK : C::B_IV) + n % kUnits));
        }
        // ---- the tile
        {
          uint32_t parity = 0;
          if (z >= C::NS) {
            const int fb = free_bar(z, parity);
            if (!(ok = wait_warp(fb, parity))) break;
          }
          unsigned char *stage = sb + C::OFF_G + (z % C::NG) * C::STAGE;
          const uint32_t dst = C::OFF_T + s * C::TILE;
          if (kind == kDraft) {
            const float f = pow2_biased(254 + C::SHV - top);
            uint32_t lost = 0u;
#pragma unroll 2
            for (int c = st; c < 128 * LPR; c += ST) {
              const int row = c / LPR, q = c % LPR;
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (row < n0 + n1) v = __ldg(reinterpret_cast<const uint4 *>(drafted + row * dstride + q * 8));
              if (kv == 1) v = finite_bf16x8(v, lost);
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_f16x2(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xFFFF0000u) * f);
              *reinterpret_cast<uint4 *>(sb + swizzled(dst, q >> 3, row, q & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (__any_sync(0xffffffffu, lost != 0u) && lane == 0) wk.totals[2] = 1;
          } else {
            __syncwarp();  // the last tile's factors have been read
            {
              auto factor = [&](int x) { return pow2_f16x2(static_cast<int>(exps >> (8 * x) & 0xFFu) - top + C::SHV); };
              reinterpret_cast<uint4 *>(factors)[lane] = make_uint4(factor(0), factor(1), factor(2), factor(3));
            }
            __syncwarp();
            // Of V, rows behind the last key become 0 and a NaN that some rows do not see goes by way of the combine (of K
            // neither matters: those logits are masked).  Apart, because what the loop below takes in instructions counts.
            if (kv == 1 && (kind == kOwn || n0 + n1 < kUnit)) {
              uint32_t *odd = wk.odd + (static_cast<size_t>(u.z) * a.c.hkv + g) * kOdd;
#pragma unroll 1
              for (int e = 0; e < 128 / STEP; ++e) {
                const int row = r0 + e * STEP;
                const bool live = (row & 63) < (row >= 64 ? n1 : n0);
                if constexpr (FMT == BSA_CACHE_E4M3) {
                  uint4 *piece = reinterpret_cast<uint4 *>(stage + row * C::RB + p * 16);
                  const uint4 c = *piece;
                  if (!live)
                    *piece = make_uint4(0u, 0u, 0u, 0u);
                  else if (kind == kOwn && (nan_codes(c.x) | nan_codes(c.y) | nan_codes(c.z) | nan_codes(c.w)) != 0u)
                    *piece = make_uint4(without_nan(c.x, p * 16, 1, odd), without_nan(c.y, p * 16 + 4, 1, odd),
                                        without_nan(c.z, p * 16 + 8, 1, odd), without_nan(c.w, p * 16 + 12, 1, odd));
                } else {
                  uint16_t *scale = reinterpret_cast<uint16_t *>(stage + C::GROUPS + row * (D / 16) + 2 * p);
                  if (!live) *scale = 0;
                  else if (kind == kOwn) *scale = static_cast<uint16_t>(without_nan(*scale, p * 32, 16, odd));
                }
              }
            }
#pragma unroll 4
            for (int e = 0; e < 128 / STEP; ++e) {
              const int row = r0 + e * STEP;
              const uint4 cw = *reinterpret_cast<const uint4 *>(stage + row * C::RB + p * 16);
              const uint32_t f = factors[row];
              const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
              const uint32_t at = dst + static_cast<uint32_t>(row) * 128;
              auto put = [&](int c, int q, uint4 v) {  // eight values into unit q of swizzle chunk c
                *reinterpret_cast<uint4 *>(sb + at + static_cast<uint32_t>(c) * C::CHUNK +
                                           static_cast<uint32_t>((q ^ (row & 7)) * 16)) = v;
              };
              if constexpr (FMT == BSA_CACHE_E4M3) {
                uint32_t h[8];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  h[2 * c] = mul_f16x2(e4m3x2_f16(w[c]), f);
                  h[2 * c + 1] = mul_f16x2(e4m3x2_f16(w[c] >> 16), f);
                }
                put(p >> 2, 2 * (p & 3), make_uint4(h[0], h[1], h[2], h[3]));
                put(p >> 2, 2 * (p & 3) + 1, make_uint4(h[4], h[5], h[6], h[7]));
              } else {
                const uint32_t scale2 = *reinterpret_cast<const uint16_t *>(stage + C::GROUPS + row * (D / 16) + 2 * p);
                const uint32_t g2 = mul_f16x2(e4m3x2_f16(scale2), f);
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
          }
          ptx::fence_proxy_async_smem();
          arrive_warp(full_bar(z));
          arrive_warp(C::B_GE + z % C::NG);
        }
      }
    }
  }

  // A softmax warp that gave up lets the one that shares its rows go.  (Here, and from the flag: a test of the lanes' own
  // variable behind their loop costs 2 to 4 % of a step in bf16, by the code around it alone.)
  if (__builtin_expect(*abort_flag, 0)) {
    const int w = static_cast<int>(threadIdx.x) >> 5, pair_bar = 1 + ((w - kSoftWarp) >> 3) * 4 + (w & 3);
    if (w >= kSoftWarp && w < kLoadWarp) wait::leave_pair(pair_bar);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag && a.status != nullptr)
    atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_DEVICE_TIMEOUT));
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- the combine

// A block is kItems (row, four dimensions) of one token and KV head.  The weights of all parts of the token's rows come
// first, a warp a row; then its teams take the parts i, i + teams, .., and the teams' sums are added in a fixed order.
constexpr int kCombineThreads = 256, kMaxParts = 2 * (kSms + 1);

template <int D, bool PAIR, int kItems>
__global__ void __launch_bounds__(kCombineThreads) shared_combine_kernel(const TreeArgs a, const SharedWork wk) {
  constexpr int kSplit = kCombineThreads / kItems;
  constexpr int LANES = PAIR ? 1 : 2;  // results of a row and part
  constexpr int TILE_ROWS = PAIR ? 2 * kRows : kRows;
  extern __shared__ float2 part[];  // [parts][G] maximum (later: weight) and sum
  __shared__ float4 red_o[kSplit][kItems];
  __shared__ float2 row_ml[16];  // maximum and sum of the rows
  const int G = a.group, items = G * (D / 4), slices = (items + kItems - 1) / kItems;
  const int i = blockIdx.x / slices, g = blockIdx.y, b = blockIdx.z;
  // (the plan was there before the kernel ahead could let this one start)
  const SeqRecord dr = wk.seqs[b];
  const int tiles = wk.totals[1], places = wk.totals[3] * a.c.hkv;
  const int row0 = (dr.at + i) * G, e = dr.tile0 + row0 / TILE_ROWS;
  if (i >= dr.len || e >= tiles) {
    // One block without rows waits all the same: where none has any (a step without drafts), this kernel would else end
    // before the one ahead, and what follows in the stream could use its workspace.
    if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0) after_previous_kernel();
    return;
  }
  const TileRecord tr = wk.tiles[e], prev = wk.tiles[max(e - 1, 0)];
  const int run = (places + kSms - 1) / kSms, span = span_of(tr.shared, tr.units);
  const int first = tr.place * a.c.hkv + g * span, cta0 = first / run;
  const int count = (first + place_of(tr.units - 1, tr.shared)) / run - cta0 + 1;
  const int tile = row0 % TILE_ROWS / kRows, rr = row0 % kRows, n = count * LANES;
  const int item = threadIdx.x % kItems, team = threadIdx.x / kItems;
  const int it = blockIdx.x % slices * kItems + item, h = it % G, q = it / G;
  const size_t out0 = static_cast<size_t>(dr.start + i) * a.hq + g * G, out = out0 + h;
  // a CTA's run begins with this tile if no unit lies between: in the places behind the last unit of the one before too
  const TileRecord &ahead = g > 0 ? tr : prev;
  const int before = g > 0 || e > 0 ? first - (span_of(ahead.shared, ahead.units) - place_of(ahead.units - 1, ahead.shared) - 1) : 0;
  auto slot_of = [&](int x) {
    const int cta = cta0 + x / LANES;
    return 2 * (2 * static_cast<size_t>(cta) + (before <= cta * run ? 0 : 1)) + (PAIR ? tile : x & 1);
  };
  after_previous_kernel();

  const uint32_t *mark = wk.odd + static_cast<size_t>(b * a.c.hkv + g) * kOdd;
  const uint32_t own_odd = mark[0];
  const int drafts_odd = wk.totals[2];
  constexpr int U = 5;  // parts in flight
  float4 v[U];
  auto fetch = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = base + u * kSplit;
      if (x >= n || it >= items) continue;
      v[u] = count == 1 ? reinterpret_cast<const float4 *>(wk.row_o)[((PAIR ? 0 : x & 1) * wk.rows + out) * (D / 4) + q]
                        : reinterpret_cast<const float4 *>(wk.part_o)[(slot_of(x) * (D / 4) + q) * kRows + rr + h];
    }
  };
  fetch(team);
  for (int x = threadIdx.x; x < n * G; x += kCombineThreads) {
    const int p = x / G, r = x - p * G, lane = PAIR ? 0 : p & 1;
    float2 ml = make_float2(-INFINITY, 0.f), ml2 = ml;
    const int from = max(0, (cta0 + p / LANES) * run - first), to = (cta0 + p / LANES + 1) * run - first;
    if (unit_at(from, tr.shared, tr.units) == unit_at(to, tr.shared, tr.units)) {
      // (a short run may fall on a place without a unit)
    } else if (count == 1) {
      ml = wk.row_ml[2 * lane * wk.rows + out0 + r];
      ml2 = wk.row_ml[(2 * lane + 1) * wk.rows + out0 + r];
    } else {
      const size_t slot = slot_of(p);
      ml = wk.part_ml[slot * 2 * kRows + rr + r];
      ml2 = wk.part_ml[(slot * 2 + 1) * kRows + rr + r];
    }
    part[x] = make_float2(ptx::max_nan(ml.x, ml2.x), ml.y + ml2.y);  // (the halves differ where one holds NaN alone)
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int warp = threadIdx.x >> 5; warp < G; warp += kCombineThreads / 32) {  // a warp a row
    float m = -INFINITY, l = 0.f;
    for (int p = lane; p < n; p += 32) m = ptx::max_nan(m, part[p * G + warp].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = ptx::max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int p = lane; p < n; p += 32) {
      const float2 ml = part[p * G + warp];
      const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
      l = ml.x == -INFINITY ? l : fmaf(ml.y, w, l);
      part[p * G + warp].x = w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) row_ml[warp] = make_float2(m, l);
  }
  __syncthreads();
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = team; base < n; base += U * kSplit) {
    if (base != team) fetch(base);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = base + u * kSplit;
      const float w = x < n && it < items ? part[x * G + h].x : 0.f;
      if (w == 0.f) continue;  // (a part without a key may hold anything)
      s.x = fmaf(v[u].x, w, s.x);
      s.y = fmaf(v[u].y, w, s.y);
      s.z = fmaf(v[u].z, w, s.z);
      s.w = fmaf(v[u].w, w, s.w);
    }
  }
  if (kSplit > 1) {
    red_o[team][item] = s;
    __syncthreads();
    if (team != 0) return;
#pragma unroll
    for (int w = 1; w < kSplit; ++w) {
      const float4 x = red_o[w][item];
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
  }
  if (it >= items) return;
  const float mm = row_ml[h].x, ls = row_ml[h].y;
  float o[4] = {s.x, s.y, s.z, s.w};
  if (own_odd != 0u) {  // Inf and NaN of own values, which every row of the sequence sees
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int dim = 4 * q + d;
      auto marked = [&](int which) { return (mark[1 + which * 4 + dim / 32] >> (dim & 31) & 1u) != 0u; };
      if (marked(0)) o[d] += INFINITY;
      if (marked(1)) o[d] -= INFINITY;
      if (marked(2)) o[d] = __int_as_float(0x7FC00000);
    }
  }
  if (drafts_odd != 0) {  // and of the drafted values on its path
    const uint16_t *vn = a.v_new + (static_cast<size_t>(dr.start) * a.c.hkv + g) * D + 4 * q;
    for (int p = i; p >= 0; p = parent_of(a, dr.start, p)) {
      const uint2 w = __ldg(reinterpret_cast<const uint2 *>(vn + static_cast<size_t>(p) * a.c.hkv * D));
      o[0] += not_finite(w.x & 0xFFFFu);
      o[1] += not_finite(w.x >> 16);
      o[2] += not_finite(w.y & 0xFFFFu);
      o[3] += not_finite(w.y >> 16);
    }
  }
  const float inv = ls == 0.f ? 0.f : 1.f / ls;
  *reinterpret_cast<uint2 *>(a.o + out * D + 4 * q) =
      make_uint2(ptx::pack_bf16x2(o[0] * inv, o[1] * inv), ptx::pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse != nullptr && q == 0) a.lse[out] = ls == 0.f ? -INFINITY : (mm + log2f(ls)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------- host side

// Lays the workspace out from `base` (null: sizes only); *bytes gets what it takes.
SharedWork work_layout(const CacheDims &c, int groups, int batch, int total, int hq, char *base, size_t *bytes) {
  size_t at = 0;
  auto take = [&](size_t n) {
    char *p = base + at;
    at += (n + 255) / 256 * 256;
    return p;
  };
  const size_t d = c.d, parts = 4ull * kSms * kRows;  // two parts per CTA, two row tiles or lanes each
  SharedWork w;
  w.rows = static_cast<size_t>(total) * hq;
  w.max_tiles = static_cast<int>(static_cast<long long>(total) * (hq / c.hkv) / kRows) + groups;
  w.part_o = reinterpret_cast<float *>(take(parts * d * 4));
  w.part_ml = reinterpret_cast<float2 *>(take(2 * parts * 8));
  w.row_o = reinterpret_cast<float *>(take(2 * w.rows * d * 4));
  w.row_ml = reinterpret_cast<float2 *>(take(4 * w.rows * 8));
  w.seqs = reinterpret_cast<SeqRecord *>(take(static_cast<size_t>(batch) * sizeof(SeqRecord)));
  w.tiles = reinterpret_cast<TileRecord *>(take(static_cast<size_t>(w.max_tiles) * sizeof(TileRecord)));
  w.own_before = reinterpret_cast<int *>(take((static_cast<size_t>(batch) + 1) * 4));
  w.token_start = reinterpret_cast<int *>(take(static_cast<size_t>(total) * 4));
  w.totals = reinterpret_cast<int *>(take(16));
  w.odd = reinterpret_cast<uint32_t *>(take(static_cast<size_t>(batch) * c.hkv * kOdd * 4));
  *bytes = at;
  return w;
}

// Rows of q, or of drafted k or v [total, heads, d]: box of 64 dimensions, `box_heads` heads and 128 / box_heads tokens;
// 128-byte swizzle.
bool token_map(EncodeTiledFn fn, CUtensorMap *map, const uint16_t *ptr, int d, int heads, int total, int box_heads) {
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(total)};
  const cuuint64_t strides[2] = {row, row * static_cast<cuuint64_t>(heads)};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(kRows / box_heads)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int FMT, bool PAIR>
bsa_status launch_t(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  using C = Shared<D, FMT, PAIR>;
  SharedMaps maps{};
  if (!C::Q16) {
    cudaError_t e = cudaSuccess;
    EncodeTiledFn fn = tensor_map_encoder(&e);
    if (fn == nullptr || e != cudaSuccess || !token_map(fn, &maps.q, a.q, D, a.hq, a.total, a.group) ||
        !token_map(fn, &maps.kn, a.k_new, D, a.c.hkv, a.total, 1) || !token_map(fn, &maps.vn, a.v_new, D, a.c.hkv, a.total, 1) ||
        !chunk_map(fn, &maps.k, a.k_codes, a.c) || !chunk_map(fn, &maps.v, a.v_codes, a.c))
      return BSA_ERR_CUDA;
  }
  size_t bytes = 0;
  const SharedWork w = work_layout(a.c, a.groups, a.batch, a.total, a.hq, static_cast<char *>(workspace), &bytes);
  auto kern = shared_kernel<D, FMT, PAIR>;
  // setmaxnreg.inc waits until the registers it asks for are free: the split is only safe if the
  // kernel really launches with that many registers per thread
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_up(kern, C::SMEM, C::LAUNCH_REGS, done);
  if (e != cudaSuccess) return e == cudaErrorNotSupported ? BSA_ERR_UNSUPPORTED : BSA_ERR_CUDA;
  static std::atomic<uint64_t> plan_done{0};
  e = set_up(shared_plan_kernel, plan_smem(kMaxDecodeRows, kMaxDecodeRows), 0, plan_done);
  if (e != cudaSuccess) return BSA_ERR_CUDA;
  const int plan_threads = a.batch <= 128 ? 128 : a.batch <= 512 ? 512 : 1024;
  shared_plan_kernel<<<1, plan_threads, plan_smem(a.batch, a.groups), stream>>>(a, w, C::NTQ * kRows);
  if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  e = launch_after(kern, dim3(kSms), C::THREADS, C::SMEM, stream, maps, a, w);
  if (e != cudaSuccess) return BSA_ERR_CUDA;
  // Teams to a row's parts: as many as let all blocks run at once (1024 threads an SM).  A step of 32 answers over 128K (4 KV
  // heads, 38 parts a row) with 2, 4, 8, 16 teams: 81, 77, 79, 86 us; of 8 answers (76 parts) with 8, 16: 87, 85.
  const long long threads = static_cast<long long>(a.total) * a.c.hkv * a.group * (D / 4);
  int items = kCombineThreads;
  while (items > 16 && threads * (2 * kCombineThreads / items) <= 1024ll * kSms) items /= 2;
  auto combine = items == 16    ? shared_combine_kernel<D, PAIR, 16>
                 : items == 32  ? shared_combine_kernel<D, PAIR, 32>
                 : items == 64  ? shared_combine_kernel<D, PAIR, 64>
                 : items == 128 ? shared_combine_kernel<D, PAIR, 128>
                                : shared_combine_kernel<D, PAIR, 256>;
  const int slices = (a.group * (D / 4) + items - 1) / items;
  e = launch_after(combine, dim3(a.max_draft * slices, a.c.hkv, a.batch), kCombineThreads,
                   static_cast<size_t>(kMaxParts) * a.group * sizeof(float2), stream, a, w);
  return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <int D, int FMT>
bsa_status launch_fmt(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  // two row tiles per unit halve the reads and conversions of the shared pages where a group fills more than one
  const bool pair = static_cast<long long>(a.total) * a.group > static_cast<long long>(kRows) * a.groups;
  return pair ? launch_t<D, FMT, true>(a, workspace, stream) : launch_t<D, FMT, false>(a, workspace, stream);
}

}  // namespace

size_t shared_workspace_bytes(const CacheDims &c, int groups, int batch, int total, int hq) {
  size_t bytes = 0;
  work_layout(c, groups, batch, total, hq, nullptr, &bytes);
  return bytes;
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
