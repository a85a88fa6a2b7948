"""Python binding of the libbsa C ABI, on torch CUDA tensors.

The functions carry the C entry points' names without the ``bsa_`` prefix and
do argument marshalling only (dtype / device / contiguity checks, pointers,
the current CUDA stream); every step of the path runs in libbsa's kernels.
PyTorch provides device memory and streams.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib

__all__ = [
    "Shape", "SelectParams", "SELECT_TOKEN_MAX", "make_shape", "block_meta", "select_workspace_bytes", "select_mask", "mask_build_workspace_bytes", "mask_build", "prefill_fwd",
    "prefill_dense_fwd", "prefill_layer", "prefill_layer_workspace_bytes", "layer_views",
    "alloc_meta", "alloc_select", "alloc_layer_workspace", "status_string", "version",
    "selftest_wait_timeout",
    "VarlenShape", "make_varlen_shape", "varlen_block_stride", "varlen_block_meta",
    "varlen_select_workspace_bytes", "varlen_select_mask", "varlen_prefill_fwd",
    "varlen_prefill_dense_fwd", "alloc_varlen_meta", "alloc_varlen_select",
    "decode_workspace_bytes", "decode_select", "decode_fwd", "decode_step",
    "block_meta_fp8", "select_mask_fp8", "prefill_fwd_fp8", "prefill_dense_fwd_fp8",
    "prefill_fp8_workspace_bytes",
    "RopeShape", "make_rope_shape", "ROPE_PAIRS", "ROPE_NO_NORM", "qk_norm_rope",
    "CacheShape", "make_cache_shape", "CACHE_BF16", "CACHE_E4M3", "CACHE_E2M1", "cache_code_bytes",
    "cache_scale_bytes", "alloc_cache", "cache_write", "cache_read",
    "TreeShape", "make_tree_shape", "tree_workspace_bytes", "tree_fwd",
    "SharedShape", "make_shared_shape", "shared_workspace_bytes", "shared_fwd",
    "cache_fork", "cache_trim", "cache_grow_workspace_bytes", "cache_grow", "cache_compact_workspace_bytes",
    "cache_compact", "VerifyShape", "make_verify_shape", "verify",
]

Shape = _lib.Shape
SelectParams = _lib.SelectParams
SELECT_TOKEN_MAX = _lib.SELECT_TOKEN_MAX
VarlenShape = _lib.VarlenShape
RopeShape = _lib.RopeShape
ROPE_PAIRS, ROPE_NO_NORM = _lib.ROPE_PAIRS, _lib.ROPE_NO_NORM
CacheShape = _lib.CacheShape
CACHE_BF16, CACHE_E4M3, CACHE_E2M1 = _lib.CACHE_BF16, _lib.CACHE_E4M3, _lib.CACHE_E2M1
TreeShape = _lib.TreeShape
SharedShape = _lib.SharedShape
VerifyShape = _lib.VerifyShape


def make_shape(batch: int, seq: int, hq: int, hkv: int, head_dim: int, block: int) -> Shape:
    return Shape(batch, seq, hq, hkv, head_dim, block)


def _ptr(t, name, dtype=None, numel=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dims(s: Shape):
    nb = s.seq // s.block
    return s.batch, s.seq, s.hq, s.hkv, s.head_dim, nb


def block_meta(shape: Shape, k, centroid, radius, quant, alpha, dev_status=None, stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    _lib.check("bsa_block_meta", lib.bsa_block_meta(
        ctypes.byref(shape), _ptr(k, "k", torch.bfloat16, b * n * hkv * d),
        _ptr(centroid, "centroid", torch.float32, b * hkv * d * nb),
        _ptr(radius, "radius", torch.float32, b * hkv * nb),
        _ptr(quant, "quant", torch.float32, b * hkv * 2),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nb),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def select_workspace_bytes(shape: Shape) -> int:
    return int(_lib.load().bsa_select_workspace_bytes(ctypes.byref(shape)))


def select_mask(shape: Shape, params: SelectParams, q, centroid, radius, alpha, kv_idx, kv_cnt,
                mask=None, workspace=None, dev_status=None, stream=None):
    """bsa_select_mask.  ``workspace``: uint8 CUDA tensor of select_workspace_bytes(shape)
    bytes (allocated here on the current device if None)."""
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(select_workspace_bytes(shape), dtype=torch.uint8, device=q.device)
    _lib.check("bsa_select_mask", lib.bsa_select_mask(
        ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16, b * n * hq * d),
        _ptr(centroid, "centroid", torch.float32, b * hkv * d * nb),
        _ptr(radius, "radius", torch.float32, b * hkv * nb),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nb),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nb * nb),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv * nb),
        _ptr(mask, "mask", torch.uint8, b * hkv * nb * nb),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def mask_build_workspace_bytes(shape: Shape) -> int:
    return int(_lib.load().bsa_mask_build_workspace_bytes(ctypes.byref(shape)))


def mask_build(shape: Shape, params: SelectParams, q, k, centroid, radius, quant, alpha, kv_idx, kv_cnt,
               mask=None, workspace=None, dev_status=None, stream=None):
    """bsa_mask_build (bsa_block_meta then bsa_select_mask in three launches).  ``workspace``:
    uint8 CUDA tensor of mask_build_workspace_bytes(shape) bytes (allocated here if None)."""
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(mask_build_workspace_bytes(shape), dtype=torch.uint8, device=q.device)
    _lib.check("bsa_mask_build", lib.bsa_mask_build(
        ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16, b * n * hq * d),
        _ptr(k, "k", torch.bfloat16, b * n * hkv * d),
        _ptr(centroid, "centroid", torch.float32, b * hkv * d * nb),
        _ptr(radius, "radius", torch.float32, b * hkv * nb),
        _ptr(quant, "quant", torch.float32, b * hkv * 2),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nb),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nb * nb),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv * nb),
        _ptr(mask, "mask", torch.uint8, b * hkv * nb * nb),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def prefill_fwd(shape: Shape, q, k, v, kv_idx, kv_cnt, softmax_scale, o, lse=None,
                dev_status=None, stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    _lib.check("bsa_prefill_fwd", lib.bsa_prefill_fwd(
        ctypes.byref(shape), _ptr(q, "q", torch.bfloat16, b * n * hq * d),
        _ptr(k, "k", torch.bfloat16, b * n * hkv * d), _ptr(v, "v", torch.bfloat16, b * n * hkv * d),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nb * nb),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv * nb), ctypes.c_float(softmax_scale),
        _ptr(o, "o", torch.bfloat16, b * n * hq * d), _ptr(lse, "lse", torch.float32, b * hq * n),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def prefill_dense_fwd(shape: Shape, q, k, v, softmax_scale, o, lse=None, dev_status=None,
                      stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    _lib.check("bsa_prefill_dense_fwd", lib.bsa_prefill_dense_fwd(
        ctypes.byref(shape), _ptr(q, "q", torch.bfloat16, b * n * hq * d),
        _ptr(k, "k", torch.bfloat16, b * n * hkv * d), _ptr(v, "v", torch.bfloat16, b * n * hkv * d),
        ctypes.c_float(softmax_scale), _ptr(o, "o", torch.bfloat16, b * n * hq * d),
        _ptr(lse, "lse", torch.float32, b * hq * n),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def prefill_layer_workspace_bytes(shape: Shape) -> int:
    return int(_lib.load().bsa_prefill_layer_workspace_bytes(ctypes.byref(shape)))


def prefill_layer(shape: Shape, params: SelectParams, q, k, v, softmax_scale, o, lse, workspace,
                  dev_status=None, stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    _lib.check("bsa_prefill_layer", lib.bsa_prefill_layer(
        ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16, b * n * hq * d),
        _ptr(k, "k", torch.bfloat16, b * n * hkv * d), _ptr(v, "v", torch.bfloat16, b * n * hkv * d),
        ctypes.c_float(softmax_scale), _ptr(o, "o", torch.bfloat16, b * n * hq * d),
        _ptr(lse, "lse", torch.float32, b * hq * n), _ptr(workspace, "workspace", torch.uint8),
        ctypes.c_size_t(workspace.numel()), _ptr(dev_status, "dev_status", torch.int32),
        _stream(stream)))


def layer_views(shape: Shape, workspace: torch.Tensor) -> dict:
    """Tensor views of the intermediates bsa_prefill_layer leaves in its workspace."""
    b, n, hq, hkv, d, nb = _dims(shape)
    offs = (ctypes.c_size_t * 6)()
    _lib.check("bsa_prefill_layer_views", _lib.load().bsa_prefill_layer_views(ctypes.byref(shape), offs))

    def view(i, dtype, shp):
        cnt = math.prod(shp)
        return workspace[offs[i]:offs[i] + cnt * 4].view(dtype).view(*shp)

    return {
        "centroid": view(0, torch.float32, (b, hkv, nb, d)),
        "radius": view(1, torch.float32, (b, hkv, nb)),
        "quant": view(2, torch.float32, (b, hkv, 2)),
        "alpha": view(3, torch.float32, (b, hkv, nb)),
        "kv_idx": view(4, torch.int32, (b, hkv, nb, nb)),
        "kv_cnt": view(5, torch.int32, (b, hkv, nb)),
    }


def alloc_meta(shape: Shape, device="cuda") -> dict:
    b, n, hq, hkv, d, nb = _dims(shape)
    f32 = dict(dtype=torch.float32, device=device)
    return {"centroid": torch.empty(b, hkv, nb, d, **f32), "radius": torch.empty(b, hkv, nb, **f32),
            "quant": torch.empty(b, hkv, 2, **f32), "alpha": torch.empty(b, hkv, nb, **f32)}


def alloc_select(shape: Shape, device="cuda", with_mask: bool = True) -> dict:
    b, n, hq, hkv, d, nb = _dims(shape)
    out = {"kv_idx": torch.empty(b, hkv, nb, nb, dtype=torch.int32, device=device),
           "kv_cnt": torch.empty(b, hkv, nb, dtype=torch.int32, device=device)}
    out["mask"] = torch.empty(b, hkv, nb, nb, dtype=torch.uint8, device=device) if with_mask else None
    return out


def alloc_layer_workspace(shape: Shape, device="cuda") -> torch.Tensor:
    return torch.empty(prefill_layer_workspace_bytes(shape), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- fp8 (e4m3) inputs
# q, k, v: uint8 CUDA tensors of e4m3 codes in the bf16 layouts; value = code * scale.

def block_meta_fp8(shape: Shape, k, k_scale, centroid, radius, quant, alpha, dev_status=None,
                   stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    _lib.check("bsa_block_meta_fp8", lib.bsa_block_meta_fp8(
        ctypes.byref(shape), _ptr(k, "k", torch.uint8, b * n * hkv * d), ctypes.c_float(k_scale),
        _ptr(centroid, "centroid", torch.float32, b * hkv * d * nb),
        _ptr(radius, "radius", torch.float32, b * hkv * nb),
        _ptr(quant, "quant", torch.float32, b * hkv * 2),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nb),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def select_mask_fp8(shape: Shape, params: SelectParams, q, q_scale, centroid, radius, alpha, kv_idx,
                    kv_cnt, mask=None, workspace=None, dev_status=None, stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(select_workspace_bytes(shape), dtype=torch.uint8, device=q.device)
    _lib.check("bsa_select_mask_fp8", lib.bsa_select_mask_fp8(
        ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.uint8, b * n * hq * d),
        ctypes.c_float(q_scale),
        _ptr(centroid, "centroid", torch.float32, b * hkv * d * nb),
        _ptr(radius, "radius", torch.float32, b * hkv * nb),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nb),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nb * nb),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv * nb),
        _ptr(mask, "mask", torch.uint8, b * hkv * nb * nb),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def prefill_fp8_workspace_bytes(shape: Shape) -> int:
    return int(_lib.load().bsa_prefill_fp8_workspace_bytes(ctypes.byref(shape)))


def _fp8_ws(shape, workspace, like):
    if workspace is None:
        workspace = torch.empty(prefill_fp8_workspace_bytes(shape), dtype=torch.uint8, device=like.device)
    return workspace


def prefill_fwd_fp8(shape: Shape, q, k, v, q_scale, k_scale, v_scale, kv_idx, kv_cnt, softmax_scale,
                    o, lse=None, workspace=None, dev_status=None, stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    workspace = _fp8_ws(shape, workspace, q)
    _lib.check("bsa_prefill_fwd_fp8", lib.bsa_prefill_fwd_fp8(
        ctypes.byref(shape), _ptr(q, "q", torch.uint8, b * n * hq * d),
        _ptr(k, "k", torch.uint8, b * n * hkv * d), _ptr(v, "v", torch.uint8, b * n * hkv * d),
        ctypes.c_float(q_scale), ctypes.c_float(k_scale), ctypes.c_float(v_scale),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nb * nb),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv * nb), ctypes.c_float(softmax_scale),
        _ptr(o, "o", torch.bfloat16, b * n * hq * d), _ptr(lse, "lse", torch.float32, b * hq * n),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def prefill_dense_fwd_fp8(shape: Shape, q, k, v, q_scale, k_scale, v_scale, softmax_scale, o,
                          lse=None, workspace=None, dev_status=None, stream=None):
    b, n, hq, hkv, d, nb = _dims(shape)
    lib = _lib.load()
    workspace = _fp8_ws(shape, workspace, q)
    _lib.check("bsa_prefill_dense_fwd_fp8", lib.bsa_prefill_dense_fwd_fp8(
        ctypes.byref(shape), _ptr(q, "q", torch.uint8, b * n * hq * d),
        _ptr(k, "k", torch.uint8, b * n * hkv * d), _ptr(v, "v", torch.uint8, b * n * hkv * d),
        ctypes.c_float(q_scale), ctypes.c_float(k_scale), ctypes.c_float(v_scale),
        ctypes.c_float(softmax_scale), _ptr(o, "o", torch.bfloat16, b * n * hq * d),
        _ptr(lse, "lse", torch.float32, b * hq * n),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


# ---------------------------------------------------------------- packed ragged batches

def make_varlen_shape(batch: int, total_tokens: int, max_seqlen: int, hq: int, hkv: int,
                      head_dim: int, block: int) -> VarlenShape:
    return VarlenShape(batch, total_tokens, max_seqlen, hq, hkv, head_dim, block)


def varlen_block_stride(shape: VarlenShape) -> int:
    """nbs: per-sequence stride of every per-block array (0 for an invalid shape)."""
    return int(_lib.load().bsa_varlen_block_stride(ctypes.byref(shape)))


def _vdims(s: VarlenShape):
    nbs = varlen_block_stride(s)
    if nbs == 0:
        raise _lib.BsaError("bsa_varlen_block_stride", 2)
    return s.batch, s.total_tokens, s.hq, s.hkv, s.head_dim, nbs


def _cu(cu_seqlens, batch):
    return _ptr(cu_seqlens, "cu_seqlens", torch.int32, batch + 1)


def varlen_block_meta(shape: VarlenShape, cu_seqlens, k, centroid, radius, quant, alpha,
                      dev_status=None, stream=None):
    b, t, hq, hkv, d, nbs = _vdims(shape)
    lib = _lib.load()
    _lib.check("bsa_varlen_block_meta", lib.bsa_varlen_block_meta(
        ctypes.byref(shape), _cu(cu_seqlens, b), _ptr(k, "k", torch.bfloat16, t * hkv * d),
        _ptr(centroid, "centroid", torch.float32, b * hkv * nbs * d),
        _ptr(radius, "radius", torch.float32, b * hkv * nbs),
        _ptr(quant, "quant", torch.float32, b * hkv * 2),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nbs),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def varlen_select_workspace_bytes(shape: VarlenShape) -> int:
    return int(_lib.load().bsa_varlen_select_workspace_bytes(ctypes.byref(shape)))


def varlen_select_mask(shape: VarlenShape, params: SelectParams, cu_seqlens, q, centroid, radius,
                       alpha, kv_idx, kv_cnt, mask=None, workspace=None, dev_status=None,
                       stream=None):
    b, t, hq, hkv, d, nbs = _vdims(shape)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(varlen_select_workspace_bytes(shape), dtype=torch.uint8,
                                device=q.device)
    _lib.check("bsa_varlen_select_mask", lib.bsa_varlen_select_mask(
        ctypes.byref(shape), ctypes.byref(params), _cu(cu_seqlens, b),
        _ptr(q, "q", torch.bfloat16, t * hq * d),
        _ptr(centroid, "centroid", torch.float32, b * hkv * nbs * d),
        _ptr(radius, "radius", torch.float32, b * hkv * nbs),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nbs),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nbs * nbs),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv * nbs),
        _ptr(mask, "mask", torch.uint8, b * hkv * nbs * nbs),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def varlen_prefill_fwd(shape: VarlenShape, cu_seqlens, q, k, v, kv_idx, kv_cnt, softmax_scale, o,
                       lse=None, dev_status=None, stream=None):
    b, t, hq, hkv, d, nbs = _vdims(shape)
    lib = _lib.load()
    _lib.check("bsa_varlen_prefill_fwd", lib.bsa_varlen_prefill_fwd(
        ctypes.byref(shape), _cu(cu_seqlens, b), _ptr(q, "q", torch.bfloat16, t * hq * d),
        _ptr(k, "k", torch.bfloat16, t * hkv * d), _ptr(v, "v", torch.bfloat16, t * hkv * d),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nbs * nbs),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv * nbs), ctypes.c_float(softmax_scale),
        _ptr(o, "o", torch.bfloat16, t * hq * d), _ptr(lse, "lse", torch.float32, hq * t),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def varlen_prefill_dense_fwd(shape: VarlenShape, cu_seqlens, q, k, v, softmax_scale, o, lse=None,
                             dev_status=None, stream=None):
    b, t, hq, hkv, d, nbs = _vdims(shape)
    lib = _lib.load()
    _lib.check("bsa_varlen_prefill_dense_fwd", lib.bsa_varlen_prefill_dense_fwd(
        ctypes.byref(shape), _cu(cu_seqlens, b), _ptr(q, "q", torch.bfloat16, t * hq * d),
        _ptr(k, "k", torch.bfloat16, t * hkv * d), _ptr(v, "v", torch.bfloat16, t * hkv * d),
        ctypes.c_float(softmax_scale), _ptr(o, "o", torch.bfloat16, t * hq * d),
        _ptr(lse, "lse", torch.float32, hq * t),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def alloc_varlen_meta(shape: VarlenShape, device="cuda") -> dict:
    b, t, hq, hkv, d, nbs = _vdims(shape)
    f32 = dict(dtype=torch.float32, device=device)
    return {"centroid": torch.empty(b, hkv, nbs, d, **f32), "radius": torch.empty(b, hkv, nbs, **f32),
            "quant": torch.empty(b, hkv, 2, **f32), "alpha": torch.empty(b, hkv, nbs, **f32)}


def alloc_varlen_select(shape: VarlenShape, device="cuda", with_mask: bool = True) -> dict:
    b, t, hq, hkv, d, nbs = _vdims(shape)
    out = {"kv_idx": torch.empty(b, hkv, nbs, nbs, dtype=torch.int32, device=device),
           "kv_cnt": torch.empty(b, hkv, nbs, dtype=torch.int32, device=device)}
    out["mask"] = (torch.empty(b, hkv, nbs, nbs, dtype=torch.uint8, device=device)
                   if with_mask else None)
    return out


# ---------------------------------------------------------------- decode

def decode_workspace_bytes(shape: VarlenShape) -> int:
    return int(_lib.load().bsa_decode_workspace_bytes(ctypes.byref(shape)))


def decode_select(shape: VarlenShape, params: SelectParams, cu_seqlens, q_new, centroid, radius,
                  alpha, kv_idx, kv_cnt, workspace=None, dev_status=None, stream=None):
    """bsa_decode_select: kept blocks of each sequence's new token (kv_idx [b, hkv, nbs],
    kv_cnt [b, hkv]).  ``workspace``: uint8 tensor of decode_workspace_bytes(shape) bytes."""
    b, t, hq, hkv, d, nbs = _vdims(shape)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(decode_workspace_bytes(shape), dtype=torch.uint8, device=q_new.device)
    _lib.check("bsa_decode_select", lib.bsa_decode_select(
        ctypes.byref(shape), ctypes.byref(params), _cu(cu_seqlens, b),
        _ptr(q_new, "q_new", torch.bfloat16, b * hq * d),
        _ptr(centroid, "centroid", torch.float32, b * hkv * nbs * d),
        _ptr(radius, "radius", torch.float32, b * hkv * nbs),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nbs),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nbs),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def decode_fwd(shape: VarlenShape, cu_seqlens, q_new, k, v, kv_idx, kv_cnt, softmax_scale, o,
               lse=None, workspace=None, dev_status=None, stream=None):
    """bsa_decode_fwd: o [b, hq, d] of each sequence's new token over its kept blocks."""
    b, t, hq, hkv, d, nbs = _vdims(shape)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(decode_workspace_bytes(shape), dtype=torch.uint8, device=q_new.device)
    _lib.check("bsa_decode_fwd", lib.bsa_decode_fwd(
        ctypes.byref(shape), _cu(cu_seqlens, b), _ptr(q_new, "q_new", torch.bfloat16, b * hq * d),
        _ptr(k, "k", torch.bfloat16, t * hkv * d), _ptr(v, "v", torch.bfloat16, t * hkv * d),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nbs),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv), ctypes.c_float(softmax_scale),
        _ptr(o, "o", torch.bfloat16, b * hq * d), _ptr(lse, "lse", torch.float32, b * hq),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


def decode_step(shape: VarlenShape, params: SelectParams, cu_seqlens, q_new, k, v, centroid, radius,
                alpha, softmax_scale, kv_idx, kv_cnt, o, lse=None, workspace=None, dev_status=None,
                stream=None):
    """bsa_decode_step: decode_select then decode_fwd in one cooperative launch."""
    b, t, hq, hkv, d, nbs = _vdims(shape)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(decode_workspace_bytes(shape), dtype=torch.uint8, device=q_new.device)
    _lib.check("bsa_decode_step", lib.bsa_decode_step(
        ctypes.byref(shape), ctypes.byref(params), _cu(cu_seqlens, b),
        _ptr(q_new, "q_new", torch.bfloat16, b * hq * d),
        _ptr(k, "k", torch.bfloat16, t * hkv * d), _ptr(v, "v", torch.bfloat16, t * hkv * d),
        _ptr(centroid, "centroid", torch.float32, b * hkv * nbs * d),
        _ptr(radius, "radius", torch.float32, b * hkv * nbs),
        _ptr(alpha, "alpha", torch.float32, b * hkv * nbs), ctypes.c_float(softmax_scale),
        _ptr(kv_idx, "kv_idx", torch.int32, b * hkv * nbs),
        _ptr(kv_cnt, "kv_cnt", torch.int32, b * hkv),
        _ptr(o, "o", torch.bfloat16, b * hq * d), _ptr(lse, "lse", torch.float32, b * hq),
        _ptr(workspace, "workspace", torch.uint8), ctypes.c_size_t(workspace.numel()),
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream)))


# ---------------------------------------------------------------- norm, rotation, paged cache, drafted tokens
#
# A step's kernels take a few microseconds each, so these bindings are kept lean: every tensor is
# checked by a handful of attribute reads and goes to ctypes as a plain address.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, dev):
    """Address of the given stream, or of the current stream of device `dev`."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(t, name, dev):
    """Refuses what is no tensor of device `dev` (the current one: the kernels are launched there)."""
    at = t.get_device() if isinstance(t, torch.Tensor) else -1
    if at < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if at != dev:
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{dev}")


def _addr(t, name, dtype, numel, dev):
    """Address of a contiguous tensor of at least numel elements; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, name, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _rows(t, name, tokens, heads, d, dev):
    """(address, elements between tokens) of bf16 rows [tokens, heads, d]; the tokens may be strided."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, name, dev)
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != (tokens, heads, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {(tokens, heads, d)}")
    st, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return t.data_ptr(), st if tokens > 1 else heads * d


def _scratch(n, stream, device):
    """n bytes, allocated on the call's stream, so that the allocator's order is that stream's."""
    with torch.cuda.stream(stream if stream is None or isinstance(stream, torch.cuda.Stream)
                           else torch.cuda.ExternalStream(int(stream))):
        return torch.empty(n, dtype=torch.uint8, device=device)


def make_rope_shape(tokens: int, hq: int, hkv: int, head_dim: int, rotary_dim: int, eps: float = 1e-6,
                    flags: int = 0) -> RopeShape:
    return RopeShape(tokens, hq, hkv, head_dim, rotary_dim, eps, flags)


def qk_norm_rope(shape: RopeShape, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, stream=None):
    """bsa_qk_norm_rope: per-head norm and rotation of q [tokens, hq, d] and k [tokens, hkv, d] (bf16, any
    stride between tokens) into q_out and k_out, which may be q and k themselves."""
    t, hq, hkv, d = shape.tokens, shape.hq, shape.hkv, shape.head_dim
    dev = torch.cuda.current_device()
    code = _lib.load().bsa_qk_norm_rope(
        ctypes.byref(shape), *_rows(q, "q", t, hq, d, dev), *_rows(k, "k", t, hkv, d, dev),
        _addr(q_weight, "q_weight", torch.bfloat16, d, dev), _addr(k_weight, "k_weight", torch.bfloat16, d, dev),
        _addr(positions, "positions", torch.int32, t, dev),
        _addr(inv_freq, "inv_freq", torch.float32, shape.rotary_dim // 2, dev),
        *_rows(q_out, "q_out", t, hq, d, dev), *_rows(k_out, "k_out", t, hkv, d, dev), _stream_of(stream, dev))
    _lib.check("bsa_qk_norm_rope", code)


def make_cache_shape(pages: int, page: int, hkv: int, head_dim: int, format: int) -> CacheShape:
    return CacheShape(pages, page, hkv, head_dim, format)


def cache_code_bytes(shape: CacheShape) -> int:
    return int(_lib.load().bsa_cache_code_bytes(ctypes.byref(shape)))


def cache_scale_bytes(shape: CacheShape) -> int:
    return int(_lib.load().bsa_cache_scale_bytes(ctypes.byref(shape)))


def alloc_cache(shape: CacheShape, device="cuda") -> dict:
    """The cache's arrays as uint8 tensors: codes "k", "v" [pages, hkv, page, row bytes] and scales "k_scale",
    "v_scale" [pages, hkv, scale bytes] (None for bf16)."""
    codes, scales = cache_code_bytes(shape), cache_scale_bytes(shape)
    if codes == 0:
        raise _lib.BsaError("bsa_cache_code_bytes", 2)
    u8 = dict(dtype=torch.uint8, device=device)
    dims = (shape.pages, shape.hkv)
    out = {}
    for name in ("k", "v"):
        out[name] = torch.empty(codes, **u8).view(*dims, shape.page, -1)
        out[name + "_scale"] = torch.empty(scales, **u8).view(*dims, -1) if scales else None
    return out


def _cache(shape, cache, dev):
    """Addresses of the cache's four arrays (no scales for bf16)."""
    d, fmt = shape.head_dim, shape.format
    rows = shape.pages * shape.hkv * shape.page
    codes, scales = ((2 * d, 0), (d, 1), (d // 2, 1 + d // 16))[fmt] if 0 <= fmt <= 2 else (0, 0)
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    if k is None or v is None or (scales and (ks is None or vs is None)):
        raise TypeError("the cache lacks codes or scales")
    u8 = torch.uint8
    if not scales:
        return _addr(k, "k", u8, rows * codes, dev), None, _addr(v, "v", u8, rows * codes, dev), None
    return (_addr(k, "k", u8, rows * codes, dev), _addr(ks, "k_scale", u8, rows * scales, dev),
            _addr(v, "v", u8, rows * codes, dev), _addr(vs, "v_scale", u8, rows * scales, dev))


def cache_write(shape: CacheShape, k, v, slots, cache: dict, dev_status=None, stream=None):
    """bsa_cache_write: rows k, v [tokens, hkv, d] (bf16, any stride between tokens) into their slots of the
    cache of alloc_cache (int32 [tokens], page index * page + row; negative: left out)."""
    dev = torch.cuda.current_device()
    at = _addr(slots, "slots", torch.int32, 0, dev)
    t, hkv, d = slots.numel(), shape.hkv, shape.head_dim
    code = _lib.load().bsa_cache_write(
        ctypes.byref(shape), t, *_rows(k, "k", t, hkv, d, dev), *_rows(v, "v", t, hkv, d, dev), at,
        *_cache(shape, cache, dev), _addr(dev_status, "dev_status", torch.int32, 1, dev), _stream_of(stream, dev))
    _lib.check("bsa_cache_write", code)


def _table(block_table, batch, dev):
    """(address, pages a sequence) of an int32 [batch, pages] table."""
    at = _addr(block_table, "block_table", torch.int32, 0, dev)
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}, needs [{batch}, pages]")
    return at, block_table.shape[1]


def cache_read(shape: CacheShape, cu_seqlens, block_table, max_seqlen: int, cache: dict, k_out, v_out,
               dev_status=None, stream=None):
    """bsa_cache_read: every sequence's cached tokens, in order, as packed bf16 rows k_out, v_out
    [total_tokens, hkv, d]."""
    dev = torch.cuda.current_device()
    cu = _addr(cu_seqlens, "cu_seqlens", torch.int32, 2, dev)
    _on(k_out, "k_out", dev)
    batch, total = cu_seqlens.numel() - 1, k_out.shape[0]
    n = total * shape.hkv * shape.head_dim
    table, stride = _table(block_table, batch, dev)
    code = _lib.load().bsa_cache_read(
        ctypes.byref(shape), batch, total, max_seqlen, cu, table, stride, *_cache(shape, cache, dev),
        _addr(k_out, "k_out", torch.bfloat16, n, dev), _addr(v_out, "v_out", torch.bfloat16, n, dev),
        _addr(dev_status, "dev_status", torch.int32, 1, dev), _stream_of(stream, dev))
    _lib.check("bsa_cache_read", code)


def make_tree_shape(batch: int, total_draft: int, max_draft: int, max_cached: int, hq: int,
                    table_stride: int) -> TreeShape:
    return TreeShape(batch, total_draft, max_draft, max_cached, hq, table_stride)


def tree_workspace_bytes(shape: TreeShape, cache_shape: CacheShape) -> int:
    return int(_lib.load().bsa_tree_workspace_bytes(ctypes.byref(shape), ctypes.byref(cache_shape)))


def tree_fwd(shape: TreeShape, cache_shape: CacheShape, cu_draft, cached, block_table, parents, q, k_new, v_new,
             cache: dict, kv_idx, kv_cnt, softmax_scale, o, lse=None, workspace=None, dev_status=None, stream=None):
    """bsa_tree_fwd: drafted tokens q [total_draft, hq, d] over the cached tokens (of the listed pages, or of
    all when kv_idx and kv_cnt are None) and over their own path of the draft tree (parents None: a chain).
    ``workspace``: uint8 tensor of tree_workspace_bytes bytes (allocated here if None)."""
    b, t, hq, hkv, d = shape.batch, shape.total_draft, shape.hq, cache_shape.hkv, cache_shape.head_dim
    dev = torch.cuda.current_device()
    i32, bf16 = torch.int32, torch.bfloat16
    table, stride = _table(block_table, b, dev)
    if stride != shape.table_stride:
        raise ValueError(f"block_table has {stride} pages a sequence, the shape says {shape.table_stride}")
    args = (_addr(cu_draft, "cu_draft", i32, b + 1, dev), _addr(cached, "cached", i32, b, dev), table,
            _addr(parents, "parents", i32, t, dev), _addr(q, "q", bf16, t * hq * d, dev),
            _addr(k_new, "k_new", bf16, t * hkv * d, dev), _addr(v_new, "v_new", bf16, t * hkv * d, dev),
            *_cache(cache_shape, cache, dev), _addr(kv_idx, "kv_idx", i32, b * hkv * stride, dev),
            _addr(kv_cnt, "kv_cnt", i32, b * hkv, dev), softmax_scale, _addr(o, "o", bf16, t * hq * d, dev),
            _addr(lse, "lse", torch.float32, t * hq, dev))
    status = _addr(dev_status, "dev_status", i32, 1, dev)
    if workspace is None:
        workspace = _scratch(tree_workspace_bytes(shape, cache_shape), stream, q.device)
    code = _lib.load().bsa_tree_fwd(
        ctypes.byref(shape), ctypes.byref(cache_shape), *args, _addr(workspace, "workspace", torch.uint8, 0, dev),
        workspace.numel(), status, _stream_of(stream, dev))
    _lib.check("bsa_tree_fwd", code)


# ---------------------------------------------------------------- shared pages, page tables, verification

def make_shared_shape(groups: int, batch: int, total_draft: int, max_draft: int, max_cached: int, hq: int,
                      table_stride: int) -> SharedShape:
    return SharedShape(groups, batch, total_draft, max_draft, max_cached, hq, table_stride)


def shared_workspace_bytes(shape: SharedShape, cache_shape: CacheShape) -> int:
    return int(_lib.load().bsa_shared_workspace_bytes(ctypes.byref(shape), ctypes.byref(cache_shape)))


def shared_fwd(shape: SharedShape, cache_shape: CacheShape, cu_group, shared_pages, cu_draft, cached, block_table,
               parents, q, k_new, v_new, cache: dict, softmax_scale, o, lse=None, workspace=None, dev_status=None,
               stream=None):
    """bsa_shared_fwd: tree_fwd over every cached token, for sequences whose tables begin with the same pages:
    group y is the sequences cu_group[y] .. cu_group[y + 1] - 1 and shares its first shared_pages[y] pages."""
    b, t, hq, hkv, d = shape.batch, shape.total_draft, shape.hq, cache_shape.hkv, cache_shape.head_dim
    dev = torch.cuda.current_device()
    i32, bf16 = torch.int32, torch.bfloat16
    table, stride = _table(block_table, b, dev)
    if stride != shape.table_stride:
        raise ValueError(f"block_table has {stride} pages a sequence, the shape says {shape.table_stride}")
    args = (_addr(cu_group, "cu_group", i32, shape.groups + 1, dev),
            _addr(shared_pages, "shared_pages", i32, shape.groups, dev), _addr(cu_draft, "cu_draft", i32, b + 1, dev),
            _addr(cached, "cached", i32, b, dev), table, _addr(parents, "parents", i32, t, dev),
            _addr(q, "q", bf16, t * hq * d, dev), _addr(k_new, "k_new", bf16, t * hkv * d, dev),
            _addr(v_new, "v_new", bf16, t * hkv * d, dev), *_cache(cache_shape, cache, dev), softmax_scale,
            _addr(o, "o", bf16, t * hq * d, dev), _addr(lse, "lse", torch.float32, t * hq, dev))
    status = _addr(dev_status, "dev_status", i32, 1, dev)
    if workspace is None:
        workspace = _scratch(shared_workspace_bytes(shape, cache_shape), stream, q.device)
    code = _lib.load().bsa_shared_fwd(
        ctypes.byref(shape), ctypes.byref(cache_shape), *args, _addr(workspace, "workspace", torch.uint8, 0, dev),
        workspace.numel(), status, _stream_of(stream, dev))
    _lib.check("bsa_shared_fwd", code)


def cache_fork(shape: CacheShape, source, cached, block_table, refs, cached_out, table_out, dev_status=None, stream=None):
    """bsa_cache_fork: row j of table_out (and cached_out) becomes row source[j] of block_table (-1: empty); the new
    rows take the old ones' place in refs (int32 [pages])."""
    dev = torch.cuda.current_device()
    i32 = torch.int32
    at = _addr(source, "source", i32, 1, dev)
    held = _addr(cached, "cached", i32, 1, dev)
    batch, out = cached.numel(), source.numel()
    table, stride = _table(block_table, batch, dev)
    to, stride_out = _table(table_out, out, dev)
    if stride_out != stride:
        raise ValueError(f"table_out has {stride_out} pages a sequence, block_table {stride}")
    code = _lib.load().bsa_cache_fork(
        ctypes.byref(shape), batch, out, stride, at, held, table, _addr(refs, "refs", i32, shape.pages, dev),
        _addr(cached_out, "cached_out", i32, out, dev), to, _addr(dev_status, "dev_status", i32, 1, dev),
        _stream_of(stream, dev))
    _lib.check("bsa_cache_fork", code)


def cache_trim(shape: CacheShape, keep, cached, block_table, refs, dev_status=None, stream=None):
    """bsa_cache_trim: sequence b keeps its first keep[b] tokens; the pages behind them are given up."""
    dev = torch.cuda.current_device()
    i32 = torch.int32
    at = _addr(keep, "keep", i32, 1, dev)
    batch = keep.numel()
    table, stride = _table(block_table, batch, dev)
    code = _lib.load().bsa_cache_trim(
        ctypes.byref(shape), batch, stride, at, _addr(cached, "cached", i32, batch, dev), table,
        _addr(refs, "refs", i32, shape.pages, dev), _addr(dev_status, "dev_status", i32, 1, dev), _stream_of(stream, dev))
    _lib.check("bsa_cache_trim", code)


def cache_grow_workspace_bytes(batch: int) -> int:
    return int(_lib.load().bsa_cache_grow_workspace_bytes(batch))


def cache_grow(shape: CacheShape, cu_new, rank, grow, cached, block_table, refs, cache: dict, slots, workspace=None,
               dev_status=None, stream=None):
    """bsa_cache_grow: pages and slots (int32 [total_new]) for the tokens cu_new[b] .. cu_new[b + 1] - 1 of every
    sequence, all of them or, with rank and grow (of verify), the grow[b] whose rank says so."""
    dev = torch.cuda.current_device()
    i32 = torch.int32
    cu = _addr(cu_new, "cu_new", i32, 2, dev)
    to = _addr(slots, "slots", i32, 0, dev)
    batch, total = cu_new.numel() - 1, slots.numel()
    table, stride = _table(block_table, batch, dev)
    args = (cu, _addr(rank, "rank", i32, total, dev), _addr(grow, "grow", i32, batch, dev),
            _addr(cached, "cached", i32, batch, dev), table, _addr(refs, "refs", i32, shape.pages, dev),
            *_cache(shape, cache, dev), to)
    status = _addr(dev_status, "dev_status", i32, 1, dev)
    if workspace is None:
        workspace = _scratch(cache_grow_workspace_bytes(batch), stream, slots.device)
    code = _lib.load().bsa_cache_grow(
        ctypes.byref(shape), batch, total, stride, *args, _addr(workspace, "workspace", torch.uint8, 0, dev),
        workspace.numel(), status, _stream_of(stream, dev))
    _lib.check("bsa_cache_grow", code)


def cache_compact_workspace_bytes(shape: CacheShape) -> int:
    return int(_lib.load().bsa_cache_compact_workspace_bytes(ctypes.byref(shape)))


def cache_compact(shape: CacheShape, cached, block_table, refs, cache: dict, live, workspace=None, dev_status=None,
                  stream=None):
    """bsa_cache_compact: the pages in use move to the front of the pool, and live (int32 [1]) says how many there
    are."""
    dev = torch.cuda.current_device()
    i32 = torch.int32
    held = _addr(cached, "cached", i32, 1, dev)
    batch = cached.numel()
    table, stride = _table(block_table, batch, dev)
    args = (held, table, _addr(refs, "refs", i32, shape.pages, dev), *_cache(shape, cache, dev),
            _addr(live, "live", i32, 1, dev))
    status = _addr(dev_status, "dev_status", i32, 1, dev)
    if workspace is None:
        workspace = _scratch(cache_compact_workspace_bytes(shape), stream, refs.device)
    code = _lib.load().bsa_cache_compact(
        ctypes.byref(shape), batch, stride, *args, _addr(workspace, "workspace", torch.uint8, 0, dev),
        workspace.numel(), status, _stream_of(stream, dev))
    _lib.check("bsa_cache_compact", code)


def make_verify_shape(batch: int, total_draft: int, max_draft: int, vocab: int) -> VerifyShape:
    return VerifyShape(batch, total_draft, max_draft, vocab)


def _probs(t, name, rows, vocab, dtype, dev):
    """(address, elements between rows) of [rows, vocab] probabilities; the rows may be strided."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, name, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, vocab):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {(rows, vocab)}")
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return t.data_ptr(), t.stride(0) if rows > 1 else vocab


def verify(shape: VerifyShape, cu_draft, parents, tokens, p, q, u_accept, u_sample, count, rank, next_token,
           dev_status=None, stream=None):
    """bsa_verify: the drafted tokens that stand against the target's probabilities p [total_draft, vocab] (fp32 or
    bf16, any stride between rows; q likewise, or None for tokens that were not drawn), and the token behind them."""
    b, t, vocab = shape.batch, shape.total_draft, shape.vocab
    dev = torch.cuda.current_device()
    i32, f32 = torch.int32, torch.float32
    dtype = p.dtype if isinstance(p, torch.Tensor) and p.dtype is torch.bfloat16 else f32
    code = _lib.load().bsa_verify(
        ctypes.byref(shape), _addr(cu_draft, "cu_draft", i32, b + 1, dev), _addr(parents, "parents", i32, t, dev),
        _addr(tokens, "tokens", i32, t, dev), *_probs(p, "p", t, vocab, dtype, dev),
        *((None, 0) if q is None else _probs(q, "q", t, vocab, dtype, dev)),
        _lib.PROBS_F32 if dtype is f32 else _lib.PROBS_BF16, _addr(u_accept, "u_accept", f32, t, dev),
        _addr(u_sample, "u_sample", f32, b, dev), _addr(count, "count", i32, b, dev), _addr(rank, "rank", i32, t, dev),
        _addr(next_token, "next_token", i32, b, dev), _addr(dev_status, "dev_status", i32, 1, dev),
        _stream_of(stream, dev))
    _lib.check("bsa_verify", code)


def selftest_wait_timeout(dev_status, limit_ns: int, ctas: int = 1, stream=None):
    """bsa_selftest_wait_timeout: CTAs that wait on a barrier nothing completes; CTA 0 gives
    up after limit_ns and writes BSA_ERR_DEVICE_TIMEOUT into dev_status, the others stop on
    seeing it."""
    lib = _lib.load()
    _lib.check("bsa_selftest_wait_timeout", lib.bsa_selftest_wait_timeout(
        _ptr(dev_status, "dev_status", torch.int32, 1), ctypes.c_uint64(limit_ns), ctypes.c_int32(ctas),
        _stream(stream)))


def status_string(code: int) -> str:
    return _lib.load().bsa_status_string(code).decode()


def version() -> int:
    return int(_lib.load().bsa_version())
