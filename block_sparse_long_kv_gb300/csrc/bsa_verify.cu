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
// Bound by the two rows (p, and q where a token was refused) of every sequence, and by the latency of a walk of
// dependent decisions.
#include <stdint.h>

#include "bsa_pages.h"
#include "bsa_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxDraft = 256;
constexpr int kTile = 256;            // elements a warp sums at a time
constexpr int kMaxTiles = 2048;       // of a CTA's slice
constexpr int kMaxCluster = 8;
constexpr int kMaxTurned = 255;       // refused children of one node

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

// floor(m x) in units of 2^-60 for m in those units and a probability x; what is no probability counts as 0 (below, or
// NaN) or 1 (above).
__device__ __forceinline__ uint64_t scaled(uint64_t m, float x) {
  if (!(x > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(fminf(x, 1.f));
  const int e = static_cast<int>(bits >> 23);
  const uint64_t f = e == 0 ? bits : (bits & 0x7FFFFFu) | 0x800000u;
  const int sh = 150 - (e == 0 ? 1 : e);  // 23 at least
  const uint64_t lo = m * f, hi = __umul64hi(m, f);
  return sh < 64 ? lo >> sh | hi << (64 - sh) : sh < 128 ? hi >> (sh - 64) : 0;
}
constexpr uint64_t kOne = 1ull << 60;

template <bool BF16>
__device__ __forceinline__ float at(const void *row, int64_t i) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t *>(row) + i)) << 16);
  else return __ldg(static_cast<const float *>(row) + i);
}
template <bool BF16>
__device__ __forceinline__ const void *row_of(const void *base, int64_t row, int64_t stride) {
  return static_cast<const char *>(base) + row * stride * (BF16 ? 2 : 4);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  __shared__ int parent[kMaxDraft], token[kMaxDraft], rank[kMaxDraft];
  __shared__ float u_of[kMaxDraft], p_at[kMaxDraft], q_at[kMaxDraft];
  __shared__ int turned[kMaxTurned + 1];          // refused children of the node
  __shared__ uint64_t mass[kMaxTurned + 1];       // M after as many refusals
  __shared__ uint64_t tile_sum[kMaxTiles];
  __shared__ uint64_t slice_sum[2][kMaxCluster];
  __shared__ int step;                            // the walk's next move
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
    p_at[i] = up < 0 ? 0.f : at<BF16>(row_of<BF16>(a.p, sp.start + up, a.p_stride), x);
    q_at[i] = up < 0 || a.q == nullptr ? 1.f : at<BF16>(row_of<BF16>(a.q, t, a.q_stride), x);
  }

  const int per = (a.vocab + ctas - 1) / ctas;   // elements of a slice
  const int v0 = min(a.vocab, me * per), v1 = min(a.vocab, v0 + per), tiles = (v1 - v0 + kTile - 1) / kTile;
  int passes = 0;
  __syncthreads();

  // what is left of the node's row at j after the first k refusals
  auto left_of = [&](const void *row, int64_t j, int k) -> uint64_t {
    uint64_t r = scaled(kOne, at<BF16>(row, j));
    for (int i = 0; i < k; ++i) {
      const float q = a.q == nullptr ? (j == token[turned[i]] ? 1.f : 0.f)
                                     : at<BF16>(row_of<BF16>(a.q, sp.start + turned[i], a.q_stride), j);
      const uint64_t less = scaled(mass[i], q);
      r = r > less ? r - less : 0;
    }
    return r;
  };
  // its sum over the vocabulary; the slice's tiles' sums stay in tile_sum, the slices' in slice_sum[passes & 1]
  auto sum_left = [&](const void *row, int k) -> uint64_t {
    for (int tile = warp; tile < tiles; tile += kWarps) {
      uint64_t s = 0;
#pragma unroll
      for (int e = 0; e < kTile / 32; ++e) {
        const int j = v0 + tile * kTile + e * 32 + lane;
        if (j < v1) s += left_of(row, j, k);
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

  // ---- the walk; every CTA of the cluster takes the same decisions
  int node = 0, depth = 1, last = 0, k = 0;  // refusals at the node; the child tried last
  mass[0] = kOne;
  bool known = true;                          // mass[k] has been summed
  for (;;) {
    const void *row = row_of<BF16>(a.p, sp.start + node, a.p_stride);
    if (warp == 0) {
      int child = -1;
      for (int base = (last + 1) & ~31; base < sp.len && child < 0; base += 32) {
        const int i = base + lane;
        const unsigned vote = __ballot_sync(0xffffffffu, i > last && i < sp.len && parent[i] == node);
        if (vote != 0) child = base + __ffs(vote) - 1;
      }
      if (lane == 0) step = child;
    }
    __syncthreads();
    const int child = step;
    if (child < 0) break;
    if (!known) {
      const uint64_t m = sum_left(row, k);
      if (tid == 0) mass[k] = m;
      known = true;
      __syncthreads();
    }
    if (tid == 0) {
      double left = p_at[child];
      for (int i = 0; i < k; ++i) {
        const int x = token[child];
        const double q = a.q == nullptr ? (token[turned[i]] == x ? 1. : 0.)
                                        : at<BF16>(row_of<BF16>(a.q, sp.start + turned[i], a.q_stride), x);
        left = fmax(left - static_cast<double>(mass[i]) * 0x1p-60 * q, 0.);
      }
      const double m = static_cast<double>(mass[k]) * 0x1p-60;
      const bool take = static_cast<double>(u_of[child]) * m * static_cast<double>(q_at[child]) < left;
      if (take) rank[child] = depth;
      else turned[k] = child;
      step = take ? 1 : 0;
    }
    __syncthreads();
    const bool take = step == 1;
    __syncthreads();  // everyone has read it
    last = child;
    if (take) {
      node = child;
      ++depth;
      k = 0;
      known = true;
    } else {
      ++k;
      known = false;
    }
  }

  // ---- the token behind the path
  const void *row = row_of<BF16>(a.p, sp.start + node, a.p_stride);
  uint64_t all = sum_left(row, k);
  if (all == 0 && k > 0) {
    k = 0;
    all = sum_left(row, 0);
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
    for (int e = 0; found >= 0 && e < kTile / 32 && next < 0; ++e) {
      const int j = v0 + found * kTile + e * 32 + lane;
      uint64_t run = j < v1 ? left_of(row, j, k) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      const unsigned over = __ballot_sync(0xffffffffu, before + run > t);
      if (over != 0) next = v0 + found * kTile + e * 32 + __ffs(over) - 1;
      else before += __shfl_sync(0xffffffffu, run, 31);
    }
    if (lane == 0) a.next[b] = next;
  }
  if (me == 0) {
    if (tid == 0) {
      a.count[b] = depth;
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
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<BF16>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_t<true>(a, stream) : launch_t<false>(a, stream);
}

}  // namespace bsa
