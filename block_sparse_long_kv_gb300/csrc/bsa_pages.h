// Declarations of the page tables' calls (fork, growth, trim, compaction) and of the verification of drafted tokens.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_cache.h"

namespace bsa {

struct ForkArgs {
  const int32_t *source, *cached, *table;
  int32_t *refs, *cached_out, *table_out;
  int32_t *status;
  int pages, page_shift, batch, batch_out, stride;
};
cudaError_t launch_fork(const ForkArgs &a, cudaStream_t stream);

struct TrimArgs {
  const int32_t *keep;
  int32_t *cached, *table, *refs;
  int32_t *status;
  int pages, page_shift, batch, stride;
};
cudaError_t launch_trim(const TrimArgs &a, cudaStream_t stream);

// What growth leaves for its second kernel, per sequence: tokens it held (-1: it got none), the shared last page, the
// page that takes its place (-1: none) and the rows to copy.
struct GrowJob {
  int start, from, to, rows;
};
struct GrowArgs {
  CacheDims c;
  const int32_t *cu, *rank, *grow;
  int32_t *cached, *table, *refs, *slots;
  uint8_t *planes[4];  // k codes, v codes, k scales, v scales
  GrowJob *jobs;
  int32_t *status;
  int batch, total, stride;
};
size_t grow_workspace_bytes(int batch);
cudaError_t launch_grow(const GrowArgs &a, cudaStream_t stream);

struct CompactArgs {
  CacheDims c;
  const int32_t *cached;
  int32_t *table, *refs, *live;
  uint8_t *planes[4];
  int32_t *work;  // moves, from [4] on [pages] holes, [pages] moved pages, and [pages] new places (-1: a free page)
  int32_t *status;
  int batch, stride;
};
size_t compact_workspace_bytes(int pages);
cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream);

struct VerifyArgs {
  const int32_t *cu, *parents, *tokens;
  const void *p, *q;
  int64_t p_stride, q_stride;
  const float *u_accept, *u_sample;
  int32_t *count, *rank, *next;
  int32_t *status;
  int batch, total, max_draft, vocab;
};
cudaError_t launch_verify(const VerifyArgs &a, bool bf16, cudaStream_t stream);

}  // namespace bsa
