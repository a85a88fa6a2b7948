// The part of a call over shared pages that sequences do not share, where it has more than sixteen rows: launches of
// the tcgen05 kernel of drafted tokens over the keys behind the shared pages.
#include "bsa_tree_mma.cuh"

namespace bsa {
namespace {

template <int D, int FMT, bool PAIR>
cudaError_t launch_t(const TreeArgs &a, const SharedOut &so, float *part_o, float *part_ml, float *lane_o,
                     cudaStream_t stream) {
  using C = Cfg<D, FMT, PAIR>;
  CUtensorMap mk{}, mv{};
  if (!C::Q16) {
    cudaError_t e = cudaSuccess;
    EncodeTiledFn fn = tensor_map_encoder(&e);
    if (e != cudaSuccess) return e;
    if (fn == nullptr || !chunk_map(fn, &mk, a.k_codes, a.c) || !chunk_map(fn, &mv, a.v_codes, a.c))
      return cudaErrorInvalidValue;
  }
  auto kern = tree_mma_kernel<D, FMT, PAIR, true>;
  // setmaxnreg.inc waits until the registers it asks for are free: the split is only safe if the
  // kernel really launches with that many registers per thread
  static std::atomic<uint64_t> done{0};
  const cudaError_t ready = set_up(kern, kMaxSmem, kLaunchRegs, done);
  if (ready != cudaSuccess) return ready;
  kern<<<kSms, kThreads, C::smem(a.batch * a.c.hkv), stream>>>(mk, mv, a, part_o, part_ml, lane_o, nullptr, so);
  return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t launch_fmt(const TreeArgs &a, const SharedOut &so, float *part_o, float *part_ml, float *lane_o,
                       cudaStream_t stream) {
  return own_many_parts(a).rows > kRows ? launch_t<D, FMT, true>(a, so, part_o, part_ml, lane_o, stream)
                                        : launch_t<D, FMT, false>(a, so, part_o, part_ml, lane_o, stream);
}

}  // namespace

// (of tree_fwd's rule on two row tiles the part that does not hang on the format: the plan fits beside them here)
OwnParts own_many_parts(const TreeArgs &a) {
  return OwnParts{a.max_draft * a.group > kRows && a.batch * a.c.hkv <= 1024 ? 2 * kRows : kRows, kSms, false};
}

cudaError_t launch_own_many(const TreeArgs &a, const SharedOut &so, float *part_o, float *part_ml, float *lane_o,
                            cudaStream_t stream) {
  const bool wide = a.c.d == 128;
  switch (a.c.format) {
    case BSA_CACHE_E4M3:
      return wide ? launch_fmt<128, BSA_CACHE_E4M3>(a, so, part_o, part_ml, lane_o, stream)
                  : launch_fmt<64, BSA_CACHE_E4M3>(a, so, part_o, part_ml, lane_o, stream);
    case BSA_CACHE_E2M1:
      return wide ? launch_fmt<128, BSA_CACHE_E2M1>(a, so, part_o, part_ml, lane_o, stream)
                  : launch_fmt<64, BSA_CACHE_E2M1>(a, so, part_o, part_ml, lane_o, stream);
    default:
      return wide ? launch_fmt<128, BSA_CACHE_BF16>(a, so, part_o, part_ml, lane_o, stream)
                  : launch_fmt<64, BSA_CACHE_BF16>(a, so, part_o, part_ml, lane_o, stream);
  }
}

}  // namespace bsa
