// Verification of drafted tokens against the target's probabilities.
//
// At a node of the draft tree with target probabilities p, the children are tried in order: token x, drawn from q, is
// taken when u M q(x) < R(x), where R = p and M = 1 at first, and every refusal makes R = max(R - M q, 0), M = sum R.
// Where no child is taken the next token comes from R / M (from p where R is nothing): the lowest j with
// R_0 + .. + R_j > u M.  The token's distribution is then p whatever q was.
//
// Which child is taken hangs on single values of p and q, read for all drafted tokens at once; rows are read whole only
// where a child was refused and a sibling follows, and once for the token that is drawn.  A cluster of CTAs shares a
// row.  M and the running sums are integers in units of 2^-60 (a probability's 24 bits shifted, products truncated
// there), so that no order of summation moves a border; a border in 64-bit floating point is off by as much.
// What is left of a row stays in shared memory from refusal to refusal, so that each reads one more row of q; 8 bytes an
// element, as far as a second CTA still fits beside this one.
// Bound by the latency of a walk of dependent decisions, not by its bytes: 32 trees of 32 tokens over 131072 ids (34 MB,
// 5 us of them) take 45 us, as long as the sequence with most refusals (39 to 55 by the draws; 104 with rows read anew each
// time), in bf16 the same; 19 chains of 8 over 50021 ids 9.7; one chain of 4 over 32768 ids 7.4.
#include <stdint.h>

#include <atomic>

#include "bsa_pages.h"
#include "bsa_internal.h"
#include "bsa_tree.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxDraft = 256;
constexpr int kLane = 8;              // neighbouring elements of a lane
constexpr int kTile = 32 * kLane;     // elements that a warp sums at a time
constexpr int kMaxCluster = 8;
constexpr int kMaxTiles = (1 << 22) / (kMaxCluster * kTile);  // of a slice
// Elements of a slice whose rest after the last refusal stays in shared memory (the others start from p again): as many
// as let a second CTA run beside this one.
constexpr int kKept = 12288;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Stores `v` at the place of `mine` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void store_at(uint64_t *mine, uint32_t rank, uint64_t v) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(there), "l"(v) : "memory");
}

// floor(m x) in units of 2^-60 for any m in those units and a probability x; what is no probability counts as 0
// (below, or NaN) or 1 (above).
__device__ __forceinline__ uint64_t scaled(uint64_t m, float x) {
  if (!(x > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(fminf(x, 1.f));
  const uint32_t f = (bits >> 23) == 0 ? bits : (bits & 0x7FFFFFu) | 0x800000u;
  const int sh = 150 - max(1, static_cast<int>(bits >> 23));  // 23 at least
  const uint64_t lo = static_cast<uint64_t>(static_cast<uint32_t>(m)) * f;
  const uint64_t hi = static_cast<uint64_t>(static_cast<uint32_t>(m >> 32)) * f + (lo >> 32);  // m f / 2^32
  if (sh < 32) return hi << (32 - sh) | static_cast<uint32_t>(lo) >> sh;
  return sh < 96 ? hi >> (sh - 32) : 0;
}
constexpr uint64_t kOne = 1ull << 60;
// scaled(kOne, x)
__device__ __forceinline__ uint64_t whole(float x) {
  if (!(x > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(fminf(x, 1.f));
  const uint64_t f = (bits >> 23) == 0 ? bits : (bits & 0x7FFFFFu) | 0x800000u;
  const int sh = 90 - max(1, static_cast<int>(bits >> 23));  // -37 at least
  return sh <= 0 ? f << -sh : sh < 32 ? f >> sh : 0;
}

template <bool BF16>
__device__ __forceinline__ float at(const void *row, int64_t i) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t *>(row) + i)) << 16);
  else return __ldg(static_cast<const float *>(row) + i);
}
// The same as a probability: what is none counts as `scaled` says.
template <bool BF16>
__device__ __forceinline__ float prob_at(const void *row, int64_t i) {
  const float x = at<BF16>(row, i);
  return x > 0.f ? fminf(x, 1.f) : 0.f;
}
template <bool BF16>
__device__ __forceinline__ const void *row_of(const void *base, int64_t row, int64_t stride) {
  return static_cast<const char *>(base) + row * stride * (BF16 ? 2 : 4);
}

// Elements j .. j + 7, 0 from `end` on; `wide`: the row begins on a 16-byte boundary (and j is a multiple of 8).
template <bool BF16>
__device__ __forceinline__ void load8(const void *row, int j, int end, bool wide, float (&x)[kLane]) {
  if (wide && j + kLane <= end) {
    if constexpr (BF16) {
      const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + j));
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    } else {
      const float4 w = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(row) + j));
      const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(row) + j) + 1);
      x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
      x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kLane; ++i) x[i] = j + i < end ? at<BF16>(row, j + i) : 0.f;
}
__device__ __forceinline__ bool is_wide(const void *row) { return (reinterpret_cast<uintptr_t>(row) & 15) == 0; }

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a, int per) {
  extern __shared__ uint64_t dyn[];               // [tiles of a slice] their sums, [kept elements] what is left of them
  __shared__ int parent[kMaxDraft], token[kMaxDraft], rank[kMaxDraft];
  __shared__ float u_of[kMaxDraft], q_at[kMaxDraft];
  __shared__ double left[kMaxDraft];              // what is left of the node's row at its children's tokens
  __shared__ int turned[kMaxDraft];               // refused children of the node
  __shared__ uint64_t mass[kMaxDraft];            // M after as many refusals
  __shared__ uint64_t slice_sum[2][kMaxCluster];
  __shared__ int walk_node, walk_k, walk_child, walk_depth;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int me = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_size());
  const int b = blockIdx.x / ctas;
  const SeqSpan sp = seq_span(a.cu, b, a.max_draft, a.total, a.status);
  if (sp.len == 0) {  // (the whole cluster)
    if (me == 0 && tid == 0) {
      a.count[b] = 0;
      a.next[b] = -1;
    }
    return;
  }
  cluster_arrive();  // (waited for before the first store into another CTA's shared memory: by then it must run)
  for (int i = tid; i < sp.len; i += kThreads) {
    const int t = sp.start + i;
    int up = i == 0 ? -1 : i - 1, x = __ldg(a.tokens + t);
    if (a.parents != nullptr && i > 0) {
      up = __ldg(a.parents + t);
      if (up < -1 || up >= i) {
        if (a.status != nullptr) atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
        up = -1;
      }
    }
    if (i > 0 && (x < 0 || x >= a.vocab)) {
      if (a.status != nullptr) atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
      x = 0;
      up = -1;  // not reached
    }
    parent[i] = up;
    token[i] = x;
    rank[i] = i == 0 ? 0 : -1;
    u_of[i] = __ldg(a.u_accept + t);
    left[i] = up < 0 ? 0.f : prob_at<BF16>(row_of<BF16>(a.p, sp.start + up, a.p_stride), x);
    q_at[i] = up < 0 || a.q == nullptr ? 1.f : prob_at<BF16>(row_of<BF16>(a.q, t, a.q_stride), x);
  }

  const int v0 = min(a.vocab, me * per), v1 = min(a.vocab, v0 + per), tiles = (v1 - v0 + kTile - 1) / kTile;
  uint64_t *tile_sum = dyn, *rest = dyn + per / kTile;  // rest: [tile][element of a lane][lane]
  int passes = 0;
  if (tid == 0) {
    mass[0] = kOne;
    walk_node = walk_k = walk_child = 0;
    walk_depth = 1;
  }
  __syncthreads();

  // what is left of the node's row at a tile's elements of this lane after k refusals, of which `rest` holds `have`
  auto left_of = [&](const void *row, int tile, int k, int have, uint64_t (&r)[kLane]) {
    const int j = v0 + tile * kTile + lane * kLane;
    int i = 0;
    if (have >= 0 && (tile + 1) * kTile <= kKept) {
      i = have;
#pragma unroll
      for (int e = 0; e < kLane; ++e) r[e] = rest[tile * kTile + e * 32 + lane];
    } else {
      float x[kLane];
      load8<BF16>(row, j, v1, is_wide(row), x);
#pragma unroll
      for (int e = 0; e < kLane; ++e) r[e] = whole(x[e]);
    }
    for (; i < k; ++i) {
      const uint64_t m = mass[i];
      float q[kLane];
      if (a.q == nullptr) {
        const int at = token[turned[i]] - j;
#pragma unroll
        for (int e = 0; e < kLane; ++e) q[e] = e == at ? 1.f : 0.f;
      } else {
        const void *q_row = row_of<BF16>(a.q, sp.start + turned[i], a.q_stride);
        load8<BF16>(q_row, j, v1, is_wide(q_row), q);
      }
#pragma unroll
      for (int e = 0; e < kLane; ++e) {
        const uint64_t less = scaled(m, q[e]);
        r[e] = r[e] > less ? r[e] - less : 0;
      }
    }
  };
  // its sum over the vocabulary; the slice's tiles' sums stay in tile_sum, the slices' in slice_sum[passes & 1]
  auto sum_left = [&](const void *row, int k, int have) -> uint64_t {
#pragma unroll 2
    for (int tile = warp; tile < tiles; tile += kWarps) {
      uint64_t r[kLane], s = 0;
      left_of(row, tile, k, have, r);
#pragma unroll
      for (int e = 0; e < kLane; ++e) s += r[e];
      if ((tile + 1) * kTile <= kKept) {
#pragma unroll
        for (int e = 0; e < kLane; ++e) rest[tile * kTile + e * 32 + lane] = r[e];
      }
      s = warp_sum(s);
      if (lane == 0) tile_sum[tile] = s;
    }
    __syncthreads();
    if (passes++ == 0) cluster_wait();
    uint64_t *sums = slice_sum[passes & 1];
    if (warp == 0) {
      uint64_t s = 0;
      for (int tile = lane; tile < tiles; tile += 32) s += tile_sum[tile];
      s = warp_sum(s);
      if (lane < ctas) store_at(sums + me, lane, s);
    }
    cluster_arrive();
    cluster_wait();
    uint64_t all = 0;
    for (int c = 0; c < ctas; ++c) all += sums[c];
    return all;
  };

  // ---- the walk; every CTA of the cluster takes the same decisions.  Warp 0 goes on until a child was refused that has
  // a sibling: then M is summed by all.
  int node = 0, k = 0, have = -1;  // `rest` holds the node's row after so many refusals (-1: another row)
  for (;;) {
    if (warp == 0) {
      int at_node = walk_node, refused = walk_k, child = walk_child, depth = walk_depth;
      bool decide = child > 0;  // (a sibling whose M has been summed)
      for (;;) {
        if (!decide) {
          const int last = child;
          child = -1;
          for (int base = (last + 1) & ~31; base < sp.len && child < 0; base += 32) {
            const int i = base + lane;
            const unsigned vote = __ballot_sync(0xffffffffu, i > last && i < sp.len && parent[i] == at_node);
            if (vote != 0) child = base + __ffs(vote) - 1;
          }
          if (child < 0 || refused > 0) break;
        }
        decide = false;
        const double m = static_cast<double>(mass[refused]) * 0x1p-60;
        if (static_cast<double>(u_of[child]) * m * static_cast<double>(q_at[child]) < left[child]) {
          if (lane == 0) rank[child] = depth;
          at_node = child;
          ++depth;
          refused = 0;
        } else {
          if (lane == 0) turned[refused] = child;
          ++refused;
        }
      }
      __syncwarp();
      if (lane == 0) {
        walk_node = at_node;
        walk_k = refused;
        walk_child = child;
        walk_depth = depth;
      }
    }
    __syncthreads();
    if (walk_node != node) have = -1;
    node = walk_node;
    k = walk_k;
    const int child = walk_child;
    if (child < 0) break;
    // the refused child's share leaves its siblings' tokens
    const int t = turned[k - 1];
    for (int i = tid; i < sp.len; i += kThreads) {
      if (i <= t || parent[i] != node) continue;
      const float q = a.q == nullptr ? (token[t] == token[i] ? 1.f : 0.f)
                                     : prob_at<BF16>(row_of<BF16>(a.q, sp.start + t, a.q_stride), token[i]);
      left[i] = fmax(left[i] - static_cast<double>(mass[k - 1]) * 0x1p-60 * static_cast<double>(q), 0.);
    }
    const uint64_t m = sum_left(row_of<BF16>(a.p, sp.start + node, a.p_stride), k, have);
    have = k;
    if (tid == 0) mass[k] = m;
    __syncthreads();
  }

  // ---- the token behind the path
  const void *row = row_of<BF16>(a.p, sp.start + node, a.p_stride);
  uint64_t all = sum_left(row, k, have);
  if (all == 0 && k > 0) {
    k = 0;
    all = sum_left(row, 0, -1);
  }
  const float u = __ldg(a.u_sample + b);
  uint64_t t = all == 0 ? 0 : all - 1;  // the last token with anything left, unless u is below 1
  if (u < 1.f) {
    // floor(u all)
    const float f = fmaxf(u, 0.f);
    t = min(t, scaled(all, f));
  }
  const uint64_t *sums = slice_sum[passes & 1];
  uint64_t before = 0;
  int owner = -1;
  for (int c = 0; c < ctas; ++c) {
    if (before + sums[c] > t) {
      owner = c;
      break;
    }
    before += sums[c];
  }
  if (owner == me && warp == 0) {
    // the tile, 32 at a time, then the element
    int found = -1;
    for (int base = 0; base < tiles && found < 0; base += 32) {
      const uint64_t s = base + lane < tiles ? tile_sum[base + lane] : 0;
      uint64_t run = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      const unsigned over = __ballot_sync(0xffffffffu, before + run > t);
      if (over != 0) {
        const int first = __ffs(over) - 1;
        before += __shfl_sync(0xffffffffu, run - s, first);
        found = base + first;
      } else {
        before += __shfl_sync(0xffffffffu, run, 31);
      }
    }
    int next = -1;
    if (found >= 0) {
      uint64_t r[kLane], s = 0;
      left_of(row, found, k, k, r);
#pragma unroll
      for (int e = 0; e < kLane; ++e) s += r[e];
      uint64_t run = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      const unsigned over = __ballot_sync(0xffffffffu, before + run > t);
      if (over != 0) {
        const int first = __ffs(over) - 1;
        run += before - s;
        int e = 0;
#pragma unroll
        for (int x = 0; x < kLane - 1; ++x) {
          run += r[x];
          e += run > t ? 0 : 1;
        }
        next = v0 + found * kTile + first * kLane + __shfl_sync(0xffffffffu, e, first);
      }
    }
    if (lane == 0) a.next[b] = max(next, 0);  // (-1: the sum has wrapped)
  }
  if (me == 0) {
    if (tid == 0) {
      a.count[b] = walk_depth;
      if (owner < 0) a.next[b] = 0;  // (no probability above 0 in the row)
    }
    for (int i = tid; i < sp.len; i += kThreads) a.rank[sp.start + i] = rank[i];
  }
}

template <bool BF16>
cudaError_t launch_t(const VerifyArgs &a, cudaStream_t stream) {
  // CTAs of a row
  int ctas = 1;
  while (ctas < kMaxCluster && a.vocab > ctas * 4096) ctas *= 2;
  const int tiles = (a.vocab + ctas * kTile - 1) / (ctas * kTile), per = tiles * kTile;  // of a slice
  auto smem_of = [](int n) { return static_cast<size_t>(n + (n * kTile < kKept ? n * kTile : kKept)) * sizeof(uint64_t); };
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_up(verify_kernel<BF16>, smem_of(kMaxTiles), 0, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_of(tiles);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<BF16>, a, per);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_t<true>(a, stream) : launch_t<false>(a, stream);
}

}  // namespace bsa
