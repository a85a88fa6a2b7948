// Shared by the two drafted-token kernels: the records that their runs leave for the combine.
#pragma once

#include <stdint.h>

namespace bsa {

// What CTA c of an attention launch records of its run of units, kTreeSeg ints:
//   [0] the group (sequence * hkv + KV head) of its first row tile, -1 without units
//   [1] that tile, [2] [3] the tile's first unit and the one past its last, [4] units per run
constexpr int kTreeSeg = 8;

// The CTA c >= 1 whose first row tile is the x-th of those that begin in run c - 1 and go on in run c; -1
// when there are fewer.  Every thread of the block takes part.
__device__ __forceinline__ int shared_tile(const int *seg, int ctas, int x) {
  __shared__ int warp_count[32];
  __shared__ int found;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
  if (threadIdx.x == 0) found = -1;
  int seen = 0;
  for (int base = 1; base < ctas; base += blockDim.x) {
    const int c = base + static_cast<int>(threadIdx.x);
    bool mine = false;
    if (c < ctas && seg[c * kTreeSeg] >= 0) {
      const int rs = seg[c * kTreeSeg + 2], W = seg[c * kTreeSeg + 4];
      mine = rs < c * W && rs >= (c - 1) * W;
    }
    const unsigned vote = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) warp_count[warp] = __popc(vote);
    __syncthreads();
    int before = seen, total = seen;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += warp_count[w];
      total += warp_count[w];
    }
    if (mine && before + __popc(vote & ((1u << lane) - 1u)) == x) found = c;
    __syncthreads();
    seen = total;
    if (seen > x) break;
  }
  return found;
}

}  // namespace bsa
