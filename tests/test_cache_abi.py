"""Refusals of the norm / rotation, paged cache and drafted-token entry points: every bad argument is
returned on the host before anything is launched (no GPU needed)."""
import ctypes

import pytest

FAKE, MIS = 0x10000, 0x10004        # never dereferenced; MIS is 4-byte aligned only
INVALID, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
f, m = ctypes.c_void_p(FAKE), ctypes.c_void_p(MIS)
i64 = ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    from block_sparse_long_kv_gb300 import build, _lib
    build.build()
    return _lib.load()


def far(n):
    """Pointers a terabyte apart, so that no two arrays overlap."""
    return ctypes.c_void_p(FAKE + (n << 40))


def rope(lib, stride_q=512, stride_k=256, q=None, k=None, qo=None, ko=None, sqo=512, sko=256, w=(None, None), pos=f,
         freq=f, **kw):
    from block_sparse_long_kv_gb300 import _lib
    base = dict(tokens=7, hq=4, hkv=2, head_dim=128, rotary_dim=128, eps=1e-6, flags=0)
    base.update(kw)
    s = _lib.RopeShape(**base)
    return lib.bsa_qk_norm_rope(ctypes.byref(s), q or far(1), i64(stride_q), k or far(2), i64(stride_k), *w, pos, freq,
                                qo or far(3), i64(sqo), ko or far(4), i64(sko), None)


def test_rope_refusals(lib):
    assert rope(lib, tokens=0) == 0                                  # nothing to do, nothing launched
    assert rope(lib, tokens=-1) == SHAPE and rope(lib, hq=0) == SHAPE and rope(lib, hkv=0) == SHAPE
    assert rope(lib, rotary_dim=144) == SHAPE and rope(lib, rotary_dim=-16) == SHAPE
    assert rope(lib, head_dim=96, rotary_dim=32) == UNSUPPORTED and rope(lib, rotary_dim=24) == UNSUPPORTED
    assert rope(lib, flags=4) == INVALID and rope(lib, eps=-1.0) == INVALID and rope(lib, eps=float("nan")) == INVALID
    assert rope(lib, eps=float("inf")) == INVALID
    for kw in (dict(stride_q=511), dict(stride_q=508), dict(sqo=504), dict(stride_k=248), dict(sko=260)):
        assert rope(lib, **kw) == INVALID, kw
    for kw in (dict(q=m), dict(k=m), dict(qo=m), dict(ko=m), dict(pos=None), dict(freq=None), dict(w=(m, None)),
               dict(w=(None, m)), dict(pos=ctypes.c_void_p(FAKE + 2))):
        assert rope(lib, **kw) == INVALID, kw
    from block_sparse_long_kv_gb300 import _lib
    assert lib.bsa_qk_norm_rope(None, f, i64(512), f, i64(256), None, None, f, f, f, i64(512), f, i64(256), None) == INVALID
    assert _lib.ROPE_PAIRS == 1 and _lib.ROPE_NO_NORM == 2


def test_rope_overlaps(lib):
    at = lambda b: ctypes.c_void_p(FAKE + (5 << 40) + b)
    # an output shifted into its own input, and over the other tensor's input or output
    assert rope(lib, q=at(0), qo=at(16)) == INVALID
    assert rope(lib, q=at(0), qo=at(0), sqo=520) == INVALID          # the same start at another stride
    assert rope(lib, k=at(0), qo=at(0)) == INVALID
    assert rope(lib, q=at(0), ko=at(512)) == INVALID
    assert rope(lib, qo=at(0), ko=at(16)) == INVALID
    # columns of one fused row (q | k, 768 elements): k_out over k's neighbour q is refused
    assert rope(lib, q=at(0), k=at(1024), stride_q=768, stride_k=768, qo=at(0), sqo=768, ko=at(1008), sko=768) == INVALID


def cshape(**kw):
    from block_sparse_long_kv_gb300 import _lib
    base = dict(pages=10, page=128, hkv=4, head_dim=128, format=1)
    base.update(kw)
    return _lib.CacheShape(**base)


def test_cache_sizes(lib):
    for fmt, row, per in ((0, 256, 0), (1, 128, 1), (2, 64, 9)):
        s = cshape(format=fmt)
        assert lib.bsa_cache_code_bytes(ctypes.byref(s)) == 10 * 4 * 128 * row
        assert lib.bsa_cache_scale_bytes(ctypes.byref(s)) == 10 * 4 * 128 * per
    big = cshape(pages=(1 << 24) - 1, hkv=8)                         # sizes past 32 bits
    assert lib.bsa_cache_code_bytes(ctypes.byref(big)) == ((1 << 24) - 1) * 8 * 128 * 128


BAD_CACHE = [(dict(pages=0), SHAPE), (dict(page=0), SHAPE), (dict(hkv=0), SHAPE), (dict(head_dim=0), SHAPE),
             (dict(head_dim=96), UNSUPPORTED), (dict(page=32), UNSUPPORTED), (dict(format=3), UNSUPPORTED),
             (dict(format=-1), UNSUPPORTED), (dict(pages=1 << 24), UNSUPPORTED), (dict(hkv=4097), UNSUPPORTED)]


def write(lib, s, tokens=3, k=f, ks=512, v=f, vs=512, slots=f, kc=f, ksc=f, vc=f, vsc=f, st=None):
    return lib.bsa_cache_write(None if s is None else ctypes.byref(s), tokens, k, i64(ks), v, i64(vs), slots, kc, ksc, vc,
                               vsc, st, None)


def read(lib, s, batch=2, total=50, most=30, cu=f, table=f, stride=1, kc=f, ksc=f, vc=f, vsc=f, k=f, v=f, st=None):
    return lib.bsa_cache_read(None if s is None else ctypes.byref(s), batch, total, most, cu, table, stride, kc, ksc, vc,
                              vsc, k, v, st, None)


@pytest.mark.parametrize("kw, code", BAD_CACHE)
def test_cache_shapes(lib, kw, code):
    s = cshape(**kw)
    assert lib.bsa_cache_code_bytes(ctypes.byref(s)) == 0 and lib.bsa_cache_scale_bytes(ctypes.byref(s)) == 0
    assert write(lib, s) == code and read(lib, s) == code


def test_cache_refusals(lib):
    s = cshape()
    two = ctypes.c_void_p(FAKE + 2)
    assert write(lib, None) == INVALID and read(lib, None) == INVALID
    assert write(lib, s, tokens=-1) == SHAPE and write(lib, s, tokens=0) == 0
    for kw in (dict(k=None), dict(v=m), dict(ks=511), dict(vs=516), dict(slots=two), dict(kc=m), dict(ksc=None),
               dict(vc=None), dict(vsc=m), dict(st=two)):
        assert write(lib, s, **kw) == INVALID, kw
    for kw in (dict(batch=0), dict(total=0), dict(most=0), dict(most=51), dict(stride=0), dict(total=300, most=129)):
        assert read(lib, s, **kw) == SHAPE, kw
    for kw in (dict(cu=None), dict(cu=two), dict(table=None), dict(kc=None), dict(ksc=m), dict(vc=m), dict(vsc=None),
               dict(k=m), dict(v=None), dict(st=two)):
        assert read(lib, s, **kw) == INVALID, kw


def tree(lib, c=None, ws=f, nbytes=1 << 40, scale=0.1, idx=None, cnt=None, lse=None, st=None, ptr=None, bad=f, **kw):
    from block_sparse_long_kv_gb300 import _lib
    base = dict(batch=2, total_draft=9, max_draft=5, max_cached=1000, hq=16, table_stride=8)
    base.update(kw)
    s = _lib.TreeShape(**base)
    c = c or cshape()
    names = ["cu", "cached", "table", "parents", "q", "k_new", "v_new", "kc", "ksc", "vc", "vsc"]
    p = [bad if n == ptr else f for n in names]
    return lib.bsa_tree_fwd(ctypes.byref(s), ctypes.byref(c), *p, idx, cnt, ctypes.c_float(scale), bad if ptr == "o" else f,
                            lse, ws, ctypes.c_size_t(nbytes), st, None)


def test_tree_refusals(lib):
    from block_sparse_long_kv_gb300 import _lib
    two = ctypes.c_void_p(FAKE + 2)
    for kw, code in BAD_CACHE:
        assert tree(lib, c=cshape(**kw)) == code
    for kw in (dict(batch=0), dict(total_draft=0), dict(max_draft=0), dict(max_draft=10), dict(max_cached=-1), dict(hq=0),
               dict(table_stride=0), dict(hq=18), dict(table_stride=7)):
        assert tree(lib, **kw) == SHAPE, kw
    for kw in (dict(hq=12), dict(hq=128), dict(max_draft=257, total_draft=600),
               dict(max_cached=4097 * 128, table_stride=5000), dict(batch=1025)):
        assert tree(lib, **kw) == UNSUPPORTED, kw
    for name in ("cu", "cached", "table", "parents"):
        assert tree(lib, ptr=name, bad=two) == INVALID, name
    for name in ("cu", "cached", "table", "q", "k_new", "v_new", "kc", "ksc", "vc", "vsc", "o"):
        assert tree(lib, ptr=name, bad=None) == INVALID, name
    for name in ("q", "k_new", "v_new", "kc", "ksc", "vc", "vsc", "o"):
        assert tree(lib, ptr=name, bad=m) == INVALID, name
    assert tree(lib, lse=m) == INVALID and tree(lib, st=two) == INVALID
    assert tree(lib, idx=f) == INVALID and tree(lib, cnt=f) == INVALID and tree(lib, idx=m, cnt=f) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert tree(lib, scale=scale) == INVALID
    s, c = _lib.TreeShape(2, 9, 5, 1000, 16, 8), cshape()
    need = lib.bsa_tree_workspace_bytes(ctypes.byref(s), ctypes.byref(c))
    assert need > 0
    assert tree(lib, ws=None) == WORKSPACE and tree(lib, ws=m) == WORKSPACE and tree(lib, nbytes=need - 1) == WORKSPACE
    bad = _lib.TreeShape(0, 9, 5, 1000, 16, 8)
    assert lib.bsa_tree_workspace_bytes(ctypes.byref(bad), ctypes.byref(c)) == 0


def test_strides_past_the_limit(lib):
    """Strides whose spans would not fit 64 bits for the largest token counts are refused."""
    for big in ((1 << 30) + 8, 1 << 40, (1 << 62)):
        assert rope(lib, stride_q=big) == INVALID and rope(lib, sko=big) == INVALID
        assert write(lib, cshape(), ks=big) == INVALID and write(lib, cshape(), vs=big) == INVALID


def test_grids_past_the_limit(lib):
    """A CTA is 64 threads: D / 16 of them to a row of one head.  Calls of more than 2^31 - 1 CTAs are refused."""
    big = (1 << 31) - 1
    for d, hkv, tokens in ((64, 16, big), (128, 8, big), (64, 4096, 1 << 24), (128, 4096, 1 << 22)):
        s = cshape(head_dim=d, hkv=hkv, pages=10)
        width = hkv * d
        assert write(lib, s, tokens=tokens, ks=width, vs=width) == UNSUPPORTED, (d, hkv)
        assert read(lib, s, total=tokens, most=30) == UNSUPPORTED, (d, hkv)
