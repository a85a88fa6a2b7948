"""Refusals of attention over shared pages, of the page tables and of verification: every bad argument is returned on
the host before anything is launched (no GPU needed)."""
import ctypes

import pytest

FAKE = 0x10000                      # never dereferenced
INVALID, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
i32, i64, size_t = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
BAD_CACHE = [(dict(pages=0), SHAPE), (dict(page=0), SHAPE), (dict(hkv=0), SHAPE), (dict(head_dim=0), SHAPE),
             (dict(head_dim=96), UNSUPPORTED), (dict(page=32), UNSUPPORTED), (dict(format=7), UNSUPPORTED),
             (dict(pages=1 << 25), UNSUPPORTED)]


def at(n, off=0):
    """Pointers a terabyte apart, so that no two arrays overlap."""
    return ctypes.c_void_p(FAKE + (n << 40) + off)


@pytest.fixture(scope="module")
def lib():
    from block_sparse_long_kv_gb300 import build, _lib
    build.build()
    return _lib.load()


def cshape(**kw):
    from block_sparse_long_kv_gb300 import _lib
    base = dict(pages=100, page=128, hkv=4, head_dim=128, format=_lib.CACHE_E4M3)
    base.update(kw)
    return _lib.CacheShape(**base)


def pointers(names, ptr, bad):
    return [bad if n == ptr else at(i + 1) for i, n in enumerate(names)]


SHARED = ["cu_group", "shared_pages", "cu", "cached", "table", "parents", "q", "k_new", "v_new", "kc", "ksc", "vc", "vsc"]


def shared(lib, c=None, ws=at(40), nbytes=1 << 40, scale=0.1, lse=None, st=None, ptr=None, bad=None, shape=None, **kw):
    from block_sparse_long_kv_gb300 import _lib
    base = dict(groups=2, batch=3, total_draft=9, max_draft=5, max_cached=1000, hq=16, table_stride=8)
    base.update(kw)
    s = _lib.SharedShape(**base)
    c = c or cshape()
    return lib.bsa_shared_fwd(ctypes.byref(s) if shape is None else shape, ctypes.byref(c), *pointers(SHARED, ptr, bad),
                              ctypes.c_float(scale), bad if ptr == "o" else at(30), lse, ws, size_t(nbytes), st, None)


def test_shared_refusals(lib):
    from block_sparse_long_kv_gb300 import _lib
    for kw, code in BAD_CACHE:
        assert shared(lib, c=cshape(**kw)) == code, kw
    for kw in (dict(groups=0), dict(batch=0), dict(total_draft=0), dict(max_draft=0), dict(max_draft=10),
               dict(max_cached=-1), dict(hq=0), dict(hq=18), dict(table_stride=0), dict(table_stride=7)):
        assert shared(lib, **kw) == SHAPE, kw
    for kw in (dict(hq=12), dict(hq=128), dict(max_draft=257, total_draft=600), dict(batch=1025), dict(groups=4097),
               dict(total_draft=1 << 28, hq=16), dict(max_cached=(1 << 31) - 1, table_stride=1 << 24, batch=1000)):
        assert shared(lib, **kw) == UNSUPPORTED, kw
    for name in ("cu_group", "shared_pages", "cu", "cached", "table", "parents"):
        assert shared(lib, ptr=name, bad=at(50, 2)) == INVALID, name
    for name in [n for n in SHARED if n != "parents"] + ["o"]:
        assert shared(lib, ptr=name, bad=None) == INVALID, name
    for name in SHARED[6:] + ["o"]:
        assert shared(lib, ptr=name, bad=at(50, 4)) == INVALID, name
    assert shared(lib, lse=at(31, 4)) == INVALID and shared(lib, st=at(32, 2)) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert shared(lib, scale=scale) == INVALID
    s, c = _lib.SharedShape(2, 3, 9, 5, 1000, 16, 8), cshape()
    need = lib.bsa_shared_workspace_bytes(ctypes.byref(s), ctypes.byref(c))
    assert need > 0
    assert shared(lib, ws=None) == WORKSPACE and shared(lib, ws=at(40, 4)) == WORKSPACE
    assert shared(lib, nbytes=need - 1) == WORKSPACE
    bad = _lib.SharedShape(0, 3, 9, 5, 1000, 16, 8)
    assert lib.bsa_shared_workspace_bytes(ctypes.byref(bad), ctypes.byref(c)) == 0
    assert lib.bsa_shared_workspace_bytes(None, ctypes.byref(c)) == 0
    assert lib.bsa_shared_workspace_bytes(ctypes.byref(s), None) == 0
    assert lib.bsa_shared_fwd(None, ctypes.byref(c), *pointers(SHARED, None, None), ctypes.c_float(0.1), at(30), None, at(40),
                              size_t(1 << 40), None, None) == INVALID


FORK = ["source", "cached", "table", "refs", "cached_out", "table_out"]


def fork(lib, c=None, batch=3, out=4, stride=8, ptr=None, bad=None, st=None):
    c = c or cshape()
    return lib.bsa_cache_fork(ctypes.byref(c), i32(batch), i32(out), i32(stride), *pointers(FORK, ptr, bad), st, None)


def test_fork_refusals(lib):
    for kw, code in BAD_CACHE:
        assert fork(lib, c=cshape(**kw)) == code, kw
    for kw in (dict(batch=0), dict(out=0), dict(stride=0)):
        assert fork(lib, **kw) == SHAPE, kw
    for name in FORK:
        assert fork(lib, ptr=name, bad=None) == INVALID and fork(lib, ptr=name, bad=at(50, 2)) == INVALID, name
    assert fork(lib, st=at(51, 2)) == INVALID
    for name in ("cached_out", "table_out"):                       # outputs over inputs
        for i in range(4):
            assert fork(lib, ptr=name, bad=at(i + 1)) == INVALID, (name, i)
    assert fork(lib, ptr="table_out", bad=at(3, 4 * 23)) == INVALID   # the last entry of the old table
    assert fork(lib, ptr="table_out", bad=at(5, 12)) == INVALID       # cached_out's last


TRIM = ["keep", "cached", "table", "refs"]


def trim(lib, c=None, batch=3, stride=8, ptr=None, bad=None, st=None):
    c = c or cshape()
    return lib.bsa_cache_trim(ctypes.byref(c), i32(batch), i32(stride), *pointers(TRIM, ptr, bad), st, None)


def test_trim_refusals(lib):
    for kw, code in BAD_CACHE:
        assert trim(lib, c=cshape(**kw)) == code, kw
    assert trim(lib, batch=0) == SHAPE and trim(lib, stride=0) == SHAPE
    for name in TRIM:
        assert trim(lib, ptr=name, bad=None) == INVALID and trim(lib, ptr=name, bad=at(50, 2)) == INVALID, name
    assert trim(lib, st=at(51, 2)) == INVALID


GROW = ["cu", "rank", "grow", "cached", "table", "refs", "kc", "ksc", "vc", "vsc", "slots"]


def grow(lib, c=None, batch=3, total=9, stride=8, ws=at(40), nbytes=1 << 30, ptr=None, bad=None, st=None):
    c = c or cshape()
    return lib.bsa_cache_grow(ctypes.byref(c), i32(batch), i32(total), i32(stride), *pointers(GROW, ptr, bad), ws,
                              size_t(nbytes), st, None)


def test_grow_refusals(lib):
    for kw, code in BAD_CACHE:
        assert grow(lib, c=cshape(**kw)) == code, kw
    for kw in (dict(batch=0), dict(total=-1), dict(stride=0)):
        assert grow(lib, **kw) == SHAPE, kw
    assert grow(lib, total=0) == 0                                 # nothing to do, nothing launched
    assert grow(lib, batch=4097) == UNSUPPORTED
    for name in GROW:
        if name not in ("rank", "grow"):
            assert grow(lib, ptr=name, bad=None) == INVALID, name
        assert grow(lib, ptr=name, bad=at(50, 2)) == INVALID, name
    for name in ("kc", "ksc", "vc", "vsc"):
        assert grow(lib, ptr=name, bad=at(50, 4)) == INVALID, name
    assert grow(lib, st=at(51, 2)) == INVALID
    need = lib.bsa_cache_grow_workspace_bytes(i32(3))
    assert need > 0 and lib.bsa_cache_grow_workspace_bytes(i32(0)) == 0
    assert grow(lib, ws=None) == WORKSPACE and grow(lib, ws=at(40, 4)) == WORKSPACE and grow(lib, nbytes=need - 1) == WORKSPACE


COMPACT = ["cached", "table", "refs", "kc", "ksc", "vc", "vsc", "live"]


def compact(lib, c=None, batch=3, stride=8, ws=at(40), nbytes=1 << 30, ptr=None, bad=None, st=None):
    c = c or cshape()
    return lib.bsa_cache_compact(ctypes.byref(c), i32(batch), i32(stride), *pointers(COMPACT, ptr, bad), ws, size_t(nbytes),
                                 st, None)


def test_compact_refusals(lib):
    for kw, code in BAD_CACHE:
        assert compact(lib, c=cshape(**kw)) == code, kw
    assert compact(lib, batch=0) == SHAPE and compact(lib, stride=0) == SHAPE
    for name in COMPACT:
        assert compact(lib, ptr=name, bad=None) == INVALID and compact(lib, ptr=name, bad=at(50, 2)) == INVALID, name
    assert compact(lib, st=at(51, 2)) == INVALID
    c = cshape()
    need = lib.bsa_cache_compact_workspace_bytes(ctypes.byref(c))
    assert need > 0 and lib.bsa_cache_compact_workspace_bytes(None) == 0
    assert compact(lib, ws=None) == WORKSPACE and compact(lib, ws=at(40, 4)) == WORKSPACE
    assert compact(lib, nbytes=need - 1) == WORKSPACE


def verify(lib, ptr=None, bad=None, p_stride=1000, q_stride=1000, kind=0, q=at(5), st=None, **kw):
    from block_sparse_long_kv_gb300 import _lib
    base = dict(batch=2, total_draft=9, max_draft=5, vocab=1000)
    base.update(kw)
    s = _lib.VerifyShape(**base)
    n = lambda name, i: bad if ptr == name else at(i)
    return lib.bsa_verify(ctypes.byref(s), n("cu", 1), n("parents", 2), n("tokens", 3), n("p", 4), i64(p_stride),
                          bad if ptr == "q" else q, i64(q_stride), i32(kind), n("ua", 6), n("us", 7), n("count", 8),
                          n("rank", 9), n("next", 10), st, None)


def test_verify_refusals(lib):
    from block_sparse_long_kv_gb300 import _lib
    for kw in (dict(batch=0), dict(total_draft=0), dict(max_draft=0), dict(max_draft=10), dict(vocab=0)):
        assert verify(lib, **kw) == SHAPE, kw
    for kw in (dict(max_draft=257, total_draft=300), dict(batch=65536), dict(kind=2),
               dict(vocab=(1 << 22) + 1, p_stride=1 << 23, q_stride=1 << 23)):
        assert verify(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(p_stride=999), dict(q_stride=999), dict(p_stride=(1 << 30) + 1), dict(q_stride=-1)):
        assert verify(lib, **kw) == INVALID, kw
    for name in ("cu", "tokens", "p", "ua", "us", "count", "rank", "next"):
        assert verify(lib, ptr=name, bad=None) == INVALID, name
    for name in ("cu", "parents", "tokens", "p", "q", "ua", "us", "count", "rank", "next"):
        assert verify(lib, ptr=name, bad=at(50, 2)) == INVALID, name
    assert verify(lib, kind=_lib.PROBS_BF16, ptr="p", bad=at(50, 1)) == INVALID
    assert verify(lib, st=at(51, 2)) == INVALID
    assert lib.bsa_verify(None, *[at(1)] * 4, i64(10), at(1), i64(10), i32(0), *[at(1)] * 5, None, None) == INVALID
