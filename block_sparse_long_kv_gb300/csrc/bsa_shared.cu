// Attention of sequences that share the first pages of their tables, the shared pages read once for all.
//
// softmax over the union of two sets of keys splits: with m, l and O the maximum, the sum of 2^(x - m) and the
// weighted values over each set, the union's are those of the sets brought to the larger maximum and added.  So the
// rows of all sequences of a group meet the shared pages together, as the row tiles of one long "sequence", each
// sequence's rows meet its own pages and drafts, and the combine adds the two.
//
// One launch of the drafted-token kernel does both: shared tiles and own tiles lie in one plan, laid end to end and
// cut into equal runs, so that short own parts fill the SMs beside the long shared one.
#include "bsa_tree_mma.cuh"

namespace bsa {
namespace {

// The combine.  A block is up to kItems (row, four dimensions) of one token and KV head; its kSplit teams take parts
// i, i + kSplit, ..: the parts of the token's rows over the shared pages, then those over its own keys.  Sums are
// added in a fixed order.
constexpr int kItems = 64, kSplit = 8;

// Where the parts of a token's rows in one row tile are.
struct Parts {
  int count;      // 0: no keys
  bool whole;     // one part, left row by row
  int first_cta, tile_first, run, lane, row;
};
__device__ __forceinline__ Parts parts_of(const int *plan, int x, int row, int rows, int ntq, int run) {
  Parts p{0, false, 0, 0, run, 0, 0};
  const int u0 = plan[x], units = plan[x + 1] - u0;
  if (units == 0) return p;
  const int tile_rows = kRows * ntq, tiles = (rows + tile_rows - 1) / tile_rows, per = units / tiles;
  p.tile_first = u0 + row / tile_rows * per;
  const int last = p.tile_first + per - 1;
  p.first_cta = p.tile_first / run;
  p.count = last / run - p.first_cta + 1;
  p.whole = p.count == 1;
  p.lane = row / kRows % ntq;
  p.row = row % kRows;
  return p;
}

template <int D, bool PAIR>
__global__ void __launch_bounds__(kItems * kSplit)
    shared_combine_kernel(const TreeArgs a, const float *part_o, const float *part_ml, const SharedOut so) {
  constexpr int NTQ = PAIR ? 2 : 1;
  after_previous_kernel();
  __shared__ float red_m[kSplit][kItems], red_l[kSplit][kItems];
  __shared__ float4 red_o[kSplit][kItems];
  const int G = a.group, items = G * (D / 4), slices = (items + kItems - 1) / kItems;
  const int i = blockIdx.x / slices, g = blockIdx.y, b = blockIdx.z;
  const Drafts dr = drafts_of(a, b);
  if (i >= dr.len) return;
  const int jobs = (a.groups + a.batch) * a.c.hkv, units = so.plan[jobs];
  const int run = (units + kSms - 1) / kSms;
  const int y = group_of(a, b);
  Parts p[2] = {};
  if (y >= 0) {
    const Drafts all = shared_job(a, y * a.c.hkv + g).rows;
    const int at = dr.start + i - all.start;
    if (at >= 0 && at < all.len) p[0] = parts_of(so.plan, y * a.c.hkv + g, at * G, all.len * G, NTQ, run);
  }
  p[1] = parts_of(so.plan, (a.groups + b) * a.c.hkv + g, i * G, dr.len * G, NTQ, run);

  const int item = threadIdx.x % kItems, team = threadIdx.x / kItems;
  const int it = blockIdx.x % slices * kItems + item, h = it % G, q = it / G;
  const size_t out = static_cast<size_t>(dr.start + i) * a.hq + g * G + h;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (it < items) {
    const int n = p[0].count + p[1].count;
    constexpr int U = 2;  // parts in flight
    for (int base = team; base < n; base += U * kSplit) {
      float2 ml[U];
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = base + u * kSplit;
        ml[u] = make_float2(-INFINITY, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < n) {
          const bool own = x >= p[0].count;
          const Parts &s = own ? p[1] : p[0];
          if (s.whole) {
            const size_t row = (own ? static_cast<size_t>(a.total) * a.hq : 0) + out;
            ml[u] = so.row_ml[row];
            v[u] = reinterpret_cast<const float4 *>(so.row_o)[row * (D / 4) + q];
          } else {
            const int cta = s.first_cta + x - (own ? p[0].count : 0);
            const size_t slot = (2 * static_cast<size_t>(cta) + (s.tile_first <= cta * s.run ? 0 : 1)) * NTQ + s.lane;
            ml[u] = reinterpret_cast<const float2 *>(part_ml)[slot * kRows + s.row + h];
            v[u] = reinterpret_cast<const float4 *>(part_o)[(slot * (D / 4) + q) * kRows + s.row + h];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (ml[u].x == -INFINITY) continue;
        const float mn = ptx::max_nan(m, ml[u].x);
        const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(ml[u].x - mn);
        m = mn;
        l = fmaf(ml[u].y, w, l * f);
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
  size_t part_o, part_ml, lane_o, row_o, row_ml, plan, total;
};
Workspace workspace_layout(int d, int jobs, size_t rows) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Workspace w;
  w.part_o = 0;  // two parts per CTA, up to two row tiles each
  w.part_ml = up(4ull * kSms * kRows * d * 4);
  w.lane_o = w.part_ml + up(4ull * kSms * kRows * 2 * 4);
  w.row_o = w.lane_o + up(static_cast<size_t>(kSms) * kRows * (d + 4) * 4);
  w.row_ml = w.row_o + up(2 * rows * d * 4);
  w.plan = w.row_ml + up(2 * rows * 8);
  w.total = w.plan + up((static_cast<size_t>(jobs) + 1) * 4);
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
  const int jobs = (a.groups + a.batch) * a.c.hkv;
  const Workspace ws = workspace_layout(D, jobs, static_cast<size_t>(a.total) * a.hq);
  char *base = static_cast<char *>(workspace);
  float *part_o = reinterpret_cast<float *>(base + ws.part_o), *part_ml = reinterpret_cast<float *>(base + ws.part_ml);
  const SharedOut so{reinterpret_cast<float *>(base + ws.row_o), reinterpret_cast<float2 *>(base + ws.row_ml),
                     reinterpret_cast<int *>(base + ws.plan)};
  auto kern = tree_mma_kernel<D, FMT, PAIR, true>;
  // setmaxnreg.inc waits until the registers it asks for are free: the split is only safe if the
  // kernel really launches with that many registers per thread
  static std::atomic<uint64_t> done{0};
  const cudaError_t ready = set_up(kern, kMaxSmem, kLaunchRegs, done);
  if (ready != cudaSuccess) return ready == cudaErrorNotSupported ? BSA_ERR_UNSUPPORTED : BSA_ERR_CUDA;
  kern<<<kSms, kThreads, C::smem(jobs), stream>>>(mk, mv, a, part_o, part_ml,
                                                  reinterpret_cast<float *>(base + ws.lane_o), nullptr, so);
  if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  const int slices = (a.group * (D / 4) + kItems - 1) / kItems;
  const cudaError_t e = launch_after(shared_combine_kernel<D, PAIR>, dim3(a.max_draft * slices, a.c.hkv, a.batch),
                                     kItems * kSplit, stream, a, static_cast<const float *>(part_o),
                                     static_cast<const float *>(part_ml), so);
  return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <int D, int FMT>
bsa_status launch_fmt(const TreeArgs &a, void *workspace, cudaStream_t stream) {
  // two row tiles per unit halve the reads and conversions of the shared pages where a group fills more than one
  const int jobs = (a.groups + a.batch) * a.c.hkv;
  const bool pair = static_cast<long long>(a.total) * a.group > static_cast<long long>(kRows) * a.groups &&
                    Cfg<D, FMT, true>::smem(jobs) <= kMaxSmem;
  return pair ? launch_t<D, FMT, true>(a, workspace, stream) : launch_t<D, FMT, false>(a, workspace, stream);
}

}  // namespace

size_t shared_workspace_bytes(const CacheDims &c, int groups, int batch, int total, int hq) {
  return workspace_layout(c.d, (groups + batch) * c.hkv, static_cast<size_t>(total) * hq).total;
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
