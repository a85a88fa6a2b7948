// Shared by the two drafted-token kernels: the arguments they check, the f16 forms of the cache's codes, and the
// records that their runs leave for the combine.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "bsa_cache.h"
#include "bsa_internal.h"

namespace bsa {

// 2^(e - 127); 0 for e <= 0.
__device__ __forceinline__ float pow2_biased(int e) { return __int_as_float(max(e, 0) << 23); }

// Two codes as f16, the low one in the low half (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x2_f16(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b8 c, z;\n\tmov.b16 {c, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
      : "=r"(r)
      : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A sequence's drafted tokens, its cached tokens and the parent of its drafted token i, checked: what is not as
// documented sets *status and reads as none, none and a root.
struct Drafts {
  int start, len;
};
__device__ __forceinline__ Drafts drafts_of(const TreeArgs &a, int b) {
  const SeqSpan sp = seq_span(a.cu, b, a.max_draft, a.total, a.status);
  return Drafts{sp.start, sp.len};
}
__device__ __forceinline__ int cached_of(const TreeArgs &a, int b) {
  const int n = __ldg(a.cached + b);
  if (n >= 0 && n <= a.max_cached) return n;
  if (a.status != nullptr) atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
  return 0;
}
__device__ __forceinline__ int parent_of(const TreeArgs &a, int start, int i) {
  if (a.parents == nullptr) return i - 1;
  const int p = __ldg(a.parents + start + i);
  if (p >= -1 && p < i) return p;
  if (a.status != nullptr) atomicCAS(a.status, 0, static_cast<int32_t>(BSA_ERR_INVALID_ARG));
  return -1;
}

// Lets the next kernel of the stream start beside this one, if it was launched by launch_after.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A kernel launched by launch_after may start before the one ahead of it in the stream has ended; it waits
// here, before its first read, until that one has ended and its writes are visible.
__device__ __forceinline__ void after_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches a kernel so that its launch overlaps the end of the kernel ahead of it.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Sets a kernel up once per device: its shared-memory limit, to the most that any call asks for (the limit belongs
// to the process: one that followed each call's size could be lowered under another thread's launch), and a check
// of its registers per thread (0: none).  `done` is the kernel's own, a bit per device.
template <typename Kernel>
cudaError_t set_up(Kernel kern, size_t most_smem, int registers, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if ((done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  if (registers != 0) {
    cudaFuncAttributes fa{};
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs != registers) return cudaErrorNotSupported;
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most_smem));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// What CTA c of an attention launch records of its run of units: the group (sequence * hkv + KV head) of its
// first row tile (-1 without units), that tile, the tile's first unit and the one past its last, the units of
// a run, and the sequence's first drafted token and their number.
struct alignas(16) TreeRun {
  int group, tile, first, last, run, draft0, drafts, pad;
};

// The run c >= 1 whose first row tile is the x-th of those that begin in run c - 1 and go on in run c; its
// number, or -1 when there are fewer.  Every thread of the block takes part, and finds the record in *out.
__device__ __forceinline__ int shared_tile(const TreeRun *runs, int ctas, int x, TreeRun *out) {
  __shared__ int warp_count[32];
  __shared__ TreeRun found;
  __shared__ int found_at;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
  if (threadIdx.x == 0) found_at = -1;
  int seen = 0;
  for (int base = 1; base < ctas; base += blockDim.x) {
    const int c = base + static_cast<int>(threadIdx.x);
    TreeRun r;
    bool mine = false;
    if (c < ctas) {
      const int4 *p = reinterpret_cast<const int4 *>(runs + c);
      const int4 a = p[0], b = p[1];
      r = TreeRun{a.x, a.y, a.z, a.w, b.x, b.y, b.z, 0};
      mine = r.group >= 0 && r.first < c * r.run && r.first >= (c - 1) * r.run;
    }
    const unsigned vote = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) warp_count[warp] = __popc(vote);
    __syncthreads();
    int before = seen, total = seen;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += warp_count[w];
      total += warp_count[w];
    }
    if (mine && before + __popc(vote & ((1u << lane) - 1u)) == x) {
      found = r;
      found_at = c;
    }
    __syncthreads();
    seen = total;
    if (seen > x) break;
  }
  *out = found;
  return found_at;
}

// Infinities and NaN of two bf16 values become 0.  A drafted value row that holds some is hidden from the rows of
// other branches by p = 0 alone, and 0 times it would not be 0: P V runs without them, and the rows that do attend
// to the token get them added to O, which is what p > 0 times them adds up to.  (A key's stay in its logit.)
// `lost` gets a bit where there were any.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w, uint32_t &lost) {
  const uint32_t bad = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;  // an exponent of ones carries into its sign bit
  lost |= bad;
  return w & ~((bad >> 15) * 0xFFFFu);
}
// A bf16 value if it is Inf or NaN, else 0.
__device__ __forceinline__ float not_finite(uint32_t bf16) {
  return (bf16 & 0x7F80u) == 0x7F80u ? __uint_as_float(bf16 << 16) : 0.f;
}

}  // namespace bsa
