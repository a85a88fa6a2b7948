// Declarations shared by the norm / rotation, paged cache and drafted-token kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa.h"

namespace bsa {

// Rows of q and k: strides in elements between tokens, the heads of a token contiguous.
struct RopeArgs {
  const uint16_t *q, *k, *q_weight, *k_weight;
  uint16_t *q_out, *k_out;
  const int32_t *positions;
  const float *inv_freq;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int tokens, hq, hkv, rotary;
  float eps;
};
cudaError_t launch_rope(const RopeArgs &a, int head_dim, bool pairs, bool norm, cudaStream_t stream);

// Sizes of the paged cache.  A (page, head) tile of codes is page * row contiguous bytes, its
// scale bytes page * per_row: the row exponents first, then the group scales.
struct CacheDims {
  int pages, page, page_shift, hkv, d, format;
  int row, per_row;
};

struct CacheWriteArgs {
  CacheDims c;
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
  const int32_t *slots;
  int tokens;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int32_t *status;
};
// CTAs of a cache write or read of `tokens` tokens (at least one).
int64_t cache_ctas(const CacheDims &c, int tokens);
cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t stream);

struct CacheReadArgs {
  CacheDims c;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const int32_t *cu, *table;
  int batch, total, max_seqlen, table_stride;
  uint16_t *k, *v;
  int32_t *status;
};
cudaError_t launch_cache_read(const CacheReadArgs &a, cudaStream_t stream);

struct TreeArgs {
  CacheDims c;
  const int32_t *cu, *cached, *table, *parents, *kv_idx, *kv_cnt;
  const uint16_t *q, *k_new, *v_new;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  uint16_t *o;
  float *lse;
  int batch, total, max_draft, max_cached, hq, group, table_stride;
  float scale_log2;
  int32_t *status;
  // sequences that share pages (bsa_shared.cu only): [groups + 1] first sequences, [groups] shared pages
  const int32_t *cu_group, *shared_pages;
  int groups;
};
// Few query rows per KV head (bsa_tree.cu), and many (bsa_tree_mma.cu).
size_t tree_mma_workspace_bytes(const CacheDims &c);
bsa_status launch_tree_mma(const TreeArgs &a, void *workspace, cudaStream_t stream);
// Sequences that share pages (bsa_shared.cu).
size_t shared_workspace_bytes(const CacheDims &c, int groups, int batch, int total, int hq);
bsa_status launch_shared(const TreeArgs &a, void *workspace, cudaStream_t stream);
size_t tree_workspace_bytes(const CacheDims &c, int batch, int hq, int max_draft);
bsa_status launch_tree(const TreeArgs &a, void *workspace, cudaStream_t stream);

}  // namespace bsa
