// C entry points of the norm / rotation, the paged cache and the drafted-token
// attention: argument checks on the host before anything is launched, then dispatch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa.h"
#include "bsa_cache.h"
#include "bsa_internal.h"

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool good(const void *p) { return p != nullptr && aligned(p, 16); }
bool good4(const void *p) { return p != nullptr && aligned(p, 4); }
bool status_ok(const int32_t *p) { return aligned(p, 4); }

// Rows of `width` bf16 values at `stride` elements: a stride the 16-byte accesses can take.
bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0 && stride <= (1ll << 30); }

// Whether `tokens` rows of one array share a byte with rows of another.  Rows of one buffer at one
// stride are compared by their columns; of other overlapping buffers nothing is known.
bool rows_overlap(const void *a, int64_t sa, int64_t wa, const void *b, int64_t sb, int64_t wb, int64_t tokens) {
  const int64_t pa = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a));
  const int64_t pb = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b));
  const int64_t ea = pa + 2 * ((tokens - 1) * sa + wa), eb = pb + 2 * ((tokens - 1) * sb + wb);
  if (ea <= pb || eb <= pa) return false;
  if (sa != sb) return true;
  int64_t delta = (pb - pa) % (2 * sa);
  if (delta < 0) delta += 2 * sa;
  return delta < 2 * wa || delta + 2 * wb > 2 * sa;
}

bsa_status check_cache(const bsa_cache_shape *s, bsa::CacheDims *c) {
  if (s == nullptr) return BSA_ERR_INVALID_ARG;
  if (s->pages < 1 || s->page < 1 || s->hkv < 1 || s->head_dim < 1) return BSA_ERR_SHAPE;
  if (s->head_dim != 64 && s->head_dim != 128) return BSA_ERR_UNSUPPORTED;
  if (s->page != 64 && s->page != 128 && s->page != 256) return BSA_ERR_UNSUPPORTED;
  if (s->format != BSA_CACHE_BF16 && s->format != BSA_CACHE_E4M3 && s->format != BSA_CACHE_E2M1)
    return BSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(s->pages) * s->page > INT32_MAX || s->hkv > 4096) return BSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(s->pages) * s->hkv > INT32_MAX) return BSA_ERR_UNSUPPORTED;
  c->pages = s->pages;
  c->page = s->page;
  c->page_shift = s->page == 64 ? 6 : s->page == 128 ? 7 : 8;
  c->hkv = s->hkv;
  c->d = s->head_dim;
  c->format = s->format;
  c->row = s->format == BSA_CACHE_BF16 ? 2 * c->d : s->format == BSA_CACHE_E4M3 ? c->d : c->d / 2;
  c->per_row = s->format == BSA_CACHE_BF16 ? 0 : s->format == BSA_CACHE_E4M3 ? 1 : 1 + c->d / 16;
  return BSA_OK;
}

bool cache_pointers_ok(const bsa::CacheDims &c, const void *kc, const void *ks, const void *vc, const void *vs) {
  return good(kc) && good(vc) && (c.per_row == 0 || (good(ks) && good(vs)));
}

bsa_status check_tree(const bsa_tree_shape *s, const bsa::CacheDims &c, int *group) {
  if (s == nullptr) return BSA_ERR_INVALID_ARG;
  if (s->batch < 1 || s->total_draft < 1 || s->max_draft < 1 || s->max_cached < 0 || s->hq < 1 || s->table_stride < 1)
    return BSA_ERR_SHAPE;
  if (s->max_draft > s->total_draft || s->hq % c.hkv != 0) return BSA_ERR_SHAPE;
  const int pages = static_cast<int>((static_cast<long long>(s->max_cached) + c.page - 1) / c.page);
  if (pages > s->table_stride) return BSA_ERR_SHAPE;
  const int g = s->hq / c.hkv;
  if (g != 1 && g != 2 && g != 4 && g != 8 && g != 16) return BSA_ERR_UNSUPPORTED;
  if (s->max_draft > 256 || pages > bsa::kMaxBlocks) return BSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(s->batch) * c.hkv > bsa::kMaxDecodeRows) return BSA_ERR_UNSUPPORTED;
  // the units of a plan are counted in 32 bits: at most these, of 64 keys and 16 rows
  const long long tiles = (static_cast<long long>(s->max_draft) * g + 15) / 16;
  const long long units = static_cast<long long>(pages) * (c.page / 64) + 4;
  if (tiles * units * s->batch * c.hkv > INT32_MAX) return BSA_ERR_UNSUPPORTED;
  *group = g;
  return BSA_OK;
}

const uint8_t *u8(const void *p) { return static_cast<const uint8_t *>(p); }
const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }
cudaStream_t cu_stream(bsa_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

bsa_status bsa_qk_norm_rope(const bsa_rope_shape *shape, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, const void *q_weight, const void *k_weight,
                            const int32_t *positions, const float *inv_freq, void *q_out,
                            int64_t q_out_stride, void *k_out, int64_t k_out_stride, bsa_stream_t stream) {
  if (shape == nullptr) return BSA_ERR_INVALID_ARG;
  const bsa_rope_shape &s = *shape;
  if (s.tokens < 0 || s.hq < 1 || s.hkv < 1 || s.rotary_dim < 0 || s.rotary_dim > s.head_dim) return BSA_ERR_SHAPE;
  if ((s.head_dim != 64 && s.head_dim != 128) || s.rotary_dim % 16 != 0) return BSA_ERR_UNSUPPORTED;
  if (s.hq > 65536 || s.hkv > 65536) return BSA_ERR_UNSUPPORTED;
  if ((s.flags & ~(BSA_ROPE_PAIRS | BSA_ROPE_NO_NORM)) != 0) return BSA_ERR_INVALID_ARG;
  if (!(s.eps >= 0.f) || isinf(s.eps)) return BSA_ERR_INVALID_ARG;
  const int64_t wq = static_cast<int64_t>(s.hq) * s.head_dim, wk = static_cast<int64_t>(s.hkv) * s.head_dim;
  if (!stride_ok(q_stride, wq) || !stride_ok(q_out_stride, wq) || !stride_ok(k_stride, wk) ||
      !stride_ok(k_out_stride, wk))
    return BSA_ERR_INVALID_ARG;
  if (s.tokens == 0) return BSA_OK;
  if (!good(q) || !good(k) || !good(q_out) || !good(k_out) || !good4(positions)) return BSA_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return BSA_ERR_INVALID_ARG;
  if (s.rotary_dim > 0 && !good4(inv_freq)) return BSA_ERR_INVALID_ARG;
  const bool q_same = q_out == q && q_out_stride == q_stride, k_same = k_out == k && k_out_stride == k_stride;
  if ((!q_same && rows_overlap(q_out, q_out_stride, wq, q, q_stride, wq, s.tokens)) ||
      (!k_same && rows_overlap(k_out, k_out_stride, wk, k, k_stride, wk, s.tokens)) ||
      rows_overlap(q_out, q_out_stride, wq, k, k_stride, wk, s.tokens) ||
      rows_overlap(k_out, k_out_stride, wk, q, q_stride, wq, s.tokens) ||
      rows_overlap(q_out, q_out_stride, wq, k_out, k_out_stride, wk, s.tokens))
    return BSA_ERR_INVALID_ARG;
  const bsa::RopeArgs a{u16(q), u16(k), u16(q_weight), u16(k_weight), static_cast<uint16_t *>(q_out),
                        static_cast<uint16_t *>(k_out), positions, inv_freq, q_stride, k_stride, q_out_stride,
                        k_out_stride, s.tokens, s.hq, s.hkv, s.rotary_dim, s.eps};
  if (bsa::launch_rope(a, s.head_dim, (s.flags & BSA_ROPE_PAIRS) != 0, (s.flags & BSA_ROPE_NO_NORM) == 0,
                       cu_stream(stream)) != cudaSuccess)
    return BSA_ERR_CUDA;
  return BSA_OK;
}

size_t bsa_cache_code_bytes(const bsa_cache_shape *shape) {
  bsa::CacheDims c;
  if (check_cache(shape, &c) != BSA_OK) return 0;
  return static_cast<size_t>(c.pages) * c.hkv * c.page * c.row;
}

size_t bsa_cache_scale_bytes(const bsa_cache_shape *shape) {
  bsa::CacheDims c;
  if (check_cache(shape, &c) != BSA_OK) return 0;
  return static_cast<size_t>(c.pages) * c.hkv * c.page * c.per_row;
}

bsa_status bsa_cache_write(const bsa_cache_shape *shape, int32_t tokens, const void *k, int64_t k_stride,
                           const void *v, int64_t v_stride, const int32_t *slots, void *k_codes,
                           void *k_scales, void *v_codes, void *v_scales, int32_t *dev_status,
                           bsa_stream_t stream) {
  bsa::CacheWriteArgs a{};
  const bsa_status st = check_cache(shape, &a.c);
  if (st != BSA_OK) return st;
  if (tokens < 0) return BSA_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(a.c.hkv) * a.c.d;
  if (!stride_ok(k_stride, width) || !stride_ok(v_stride, width)) return BSA_ERR_INVALID_ARG;
  if (!cache_pointers_ok(a.c, k_codes, k_scales, v_codes, v_scales) || !status_ok(dev_status))
    return BSA_ERR_INVALID_ARG;
  if (tokens == 0) return BSA_OK;
  if (bsa::cache_ctas(a.c, tokens) > INT32_MAX) return BSA_ERR_UNSUPPORTED;
  if (!good(k) || !good(v) || !good4(slots)) return BSA_ERR_INVALID_ARG;
  a.k = u16(k);
  a.v = u16(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.tokens = tokens;
  a.k_codes = static_cast<uint8_t *>(k_codes);
  a.k_scales = static_cast<uint8_t *>(k_scales);
  a.v_codes = static_cast<uint8_t *>(v_codes);
  a.v_scales = static_cast<uint8_t *>(v_scales);
  a.status = dev_status;
  return bsa::launch_cache_write(a, cu_stream(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_cache_read(const bsa_cache_shape *shape, int32_t batch, int32_t total_tokens,
                          int32_t max_seqlen, const int32_t *cu_seqlens, const int32_t *block_table,
                          int32_t table_stride, const void *k_codes, const void *k_scales,
                          const void *v_codes, const void *v_scales, void *k_out, void *v_out,
                          int32_t *dev_status, bsa_stream_t stream) {
  bsa::CacheReadArgs a{};
  const bsa_status st = check_cache(shape, &a.c);
  if (st != BSA_OK) return st;
  if (batch < 1 || total_tokens < 1 || max_seqlen < 1 || table_stride < 1 || max_seqlen > total_tokens)
    return BSA_ERR_SHAPE;
  if ((static_cast<long long>(max_seqlen) + a.c.page - 1) / a.c.page > table_stride) return BSA_ERR_SHAPE;
  if (bsa::cache_ctas(a.c, total_tokens) > INT32_MAX) return BSA_ERR_UNSUPPORTED;
  if (!cache_pointers_ok(a.c, k_codes, k_scales, v_codes, v_scales) || !good4(cu_seqlens) || !good4(block_table) ||
      !good(k_out) || !good(v_out) || !status_ok(dev_status))
    return BSA_ERR_INVALID_ARG;
  a.k_codes = u8(k_codes);
  a.k_scales = u8(k_scales);
  a.v_codes = u8(v_codes);
  a.v_scales = u8(v_scales);
  a.cu = cu_seqlens;
  a.table = block_table;
  a.batch = batch;
  a.total = total_tokens;
  a.max_seqlen = max_seqlen;
  a.table_stride = table_stride;
  a.k = static_cast<uint16_t *>(k_out);
  a.v = static_cast<uint16_t *>(v_out);
  a.status = dev_status;
  return bsa::launch_cache_read(a, cu_stream(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

size_t bsa_tree_workspace_bytes(const bsa_tree_shape *shape, const bsa_cache_shape *cache) {
  bsa::CacheDims c;
  int group;
  if (check_cache(cache, &c) != BSA_OK || check_tree(shape, c, &group) != BSA_OK) return 0;
  return bsa::tree_workspace_bytes(c, shape->batch, shape->hq, shape->max_draft);
}

bsa_status bsa_tree_fwd(const bsa_tree_shape *shape, const bsa_cache_shape *cache, const int32_t *cu_draft,
                        const int32_t *cached, const int32_t *block_table, const int32_t *parents,
                        const void *q, const void *k_new, const void *v_new, const void *k_codes,
                        const void *k_scales, const void *v_codes, const void *v_scales,
                        const int32_t *kv_idx, const int32_t *kv_cnt, float softmax_scale, void *o,
                        float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                        bsa_stream_t stream) {
  bsa::TreeArgs a{};
  bsa_status st = check_cache(cache, &a.c);
  if (st != BSA_OK) return st;
  st = check_tree(shape, a.c, &a.group);
  if (st != BSA_OK) return st;
  if (!good4(cu_draft) || !good4(cached) || !good4(block_table) || !aligned(parents, 4) || !good(q) || !good(k_new) ||
      !good(v_new) || !good(o) || !aligned(lse, 16) || !status_ok(dev_status) ||
      !cache_pointers_ok(a.c, k_codes, k_scales, v_codes, v_scales))
    return BSA_ERR_INVALID_ARG;
  if ((kv_idx == nullptr) != (kv_cnt == nullptr) || !aligned(kv_idx, 16) || !aligned(kv_cnt, 16))
    return BSA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || isinf(softmax_scale)) return BSA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16) ||
      workspace_bytes < bsa::tree_workspace_bytes(a.c, shape->batch, shape->hq, shape->max_draft))
    return BSA_ERR_WORKSPACE;
  a.cu = cu_draft;
  a.cached = cached;
  a.table = block_table;
  a.parents = parents;
  a.kv_idx = kv_idx;
  a.kv_cnt = kv_cnt;
  a.q = u16(q);
  a.k_new = u16(k_new);
  a.v_new = u16(v_new);
  a.k_codes = u8(k_codes);
  a.k_scales = u8(k_scales);
  a.v_codes = u8(v_codes);
  a.v_scales = u8(v_scales);
  a.o = static_cast<uint16_t *>(o);
  a.lse = lse;
  a.batch = shape->batch;
  a.total = shape->total_draft;
  a.max_draft = shape->max_draft;
  a.max_cached = shape->max_cached;
  a.hq = shape->hq;
  a.table_stride = shape->table_stride;
  a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  a.status = dev_status;
  return bsa::launch_tree(a, workspace, cu_stream(stream));
}

}  // extern "C"
