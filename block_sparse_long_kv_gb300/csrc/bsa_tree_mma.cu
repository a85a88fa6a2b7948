// Drafted-token attention with many query rows: the launch of the tcgen05 kernel, and the combine of the row tiles
// that several of its CTAs share.

#include "bsa_tree_mma.cuh"

namespace bsa {
namespace {

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
  auto kern = tree_mma_kernel<D, FMT, PAIR, false>;
  // setmaxnreg.inc waits until the registers it asks for are free: the split is only safe if the
  // kernel really launches with that many registers per thread
  static std::atomic<uint64_t> done{0};
  const cudaError_t ready = set_up(kern, kMaxSmem, kLaunchRegs, done);
  if (ready != cudaSuccess) return ready == cudaErrorNotSupported ? BSA_ERR_UNSUPPORTED : BSA_ERR_CUDA;
  const size_t smem = C::smem(a.batch * a.c.hkv);
  kern<<<kSms, kThreads, smem, stream>>>(mk, mv, a, part_o, part_ml, lane_o, runs, SharedOut{});
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
