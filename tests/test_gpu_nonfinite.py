"""Infinities and NaN go where the formulas take them: to every row that uses them, whatever the batch around
it, and to no other.  Everything else keeps the bits that it has with zeros in their place."""
import math

import pytest
import torch

from oracle import cache_oracle as C
from test_gpu_tree import FMTS, Case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_kv_gb300 import build
    build.build()


def same(a, b):
    """Equal bits, NaN equal to NaN."""
    return torch.equal(torch.nan_to_num(a.float(), 12345.0, 23456.0, -23456.0), torch.nan_to_num(b.float(), 12345.0, 23456.0, -23456.0))


# one row tile in one CTA, and tiles shared by many CTAs; few rows, up to 128 rows, more
SPLITS = [[40], [9000], [700, 3000]]
DRAFTS = [4, 20, 70]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lengths", SPLITS)
@pytest.mark.parametrize("drafts", DRAFTS)
def test_a_query_with_nan_gives_nan_however_its_tile_is_split(fmt, lengths, drafts):
    c = Case(fmt, lengths, [drafts] * len(lengths), 8, 2, 128, 64, seed=drafts)
    bad = [(1, 0, NAN), (2, 5, INF), (drafts * len(lengths) - 1, 7, NAN)]
    for t, h, _ in bad:
        c.q[t, h] = 0
    o, lse = c.run()
    for t, h, value in bad:
        c.q[t, h, 3] = value
    got, gl = c.run()
    for t, h, _ in bad:
        assert torch.isnan(got[t, h].float()).all() and torch.isnan(gl[t, h]), (t, h)
        got[t, h], gl[t, h] = o[t, h], lse[t, h]
    assert torch.equal(got, o) and torch.equal(gl, lse)


def descends(parents, j):
    """The tokens that attend to drafted token j."""
    out = []
    for i in range(len(parents)):
        p = i
        while p > j:
            p = parents[p]
        if p == j:
            out.append(i)
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("length", [0, 40, 9000])
@pytest.mark.parametrize("drafts", [4, 20, 70, 200])
def test_a_drafted_value_with_inf_or_nan_reaches_those_that_attend_to_it(fmt, length, drafts):
    """v_new of two tokens: the dimensions that hold Inf or NaN come out as the formula gives them, the others and
    lse as with zeros there."""
    c = Case(fmt, [length], [drafts], 8, 2, 128, 64, seed=drafts)
    c.parents[0][1] = c.parents[0][2] = 0
    tokens = [(1, slice(0, 128, 5), NAN), (drafts // 2, slice(2, 128, 7), INF), (drafts - 1, slice(3, 128, 11), -INF)]
    for j, dims, _ in tokens:
        c.v_new[j, 1, dims] = 0
    want, wl = c.run()
    want = want.float()
    for j, dims, value in tokens:
        c.v_new[j, 1, dims] = value
        for i in descends(c.parents[0], j):
            want[i, 4:, dims] += value
    got, gl = c.run()
    assert torch.isnan(want).any() and torch.isinf(want).any()
    assert same(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("length", [0, 40, 9000])
@pytest.mark.parametrize("drafts", [4, 20, 70, 200])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_drafted_key_with_inf_or_nan_reaches_those_that_attend_to_it(fmt, length, drafts, value):
    """A key whose logit is NaN or +Inf makes its rows NaN; no other row changes."""
    c = Case(fmt, [length], [drafts], 8, 2, 128, 64, seed=drafts)
    c.parents[0][1] = c.parents[0][2] = 0
    j = drafts // 2
    c.k_new[j, 0, 9] = 0
    c.q[:, :4, 9] = c.q[:, :4, 9].abs() + 1
    want, wl = c.run()
    c.k_new[j, 0, 9] = value
    got, gl = c.run()
    for i in descends(c.parents[0], j):
        assert torch.isnan(got[i, :4].float()).all() and torch.isnan(gl[i, :4]).all(), i
        got[i, :4], gl[i, :4] = want[i, :4], wl[i, :4]
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("n", [40, 9000])
@pytest.mark.parametrize("group", [1, 8])
def test_decode_of_a_query_with_nan(n, group):
    """One decode row of NaN, in one CTA's run or split over many, in two calls and in the one-launch step."""
    import block_sparse_long_kv_gb300 as bsa
    hkv, d, block = 2, 128, 128
    hq = hkv * group
    g = torch.Generator().manual_seed(n)
    s = bsa.make_varlen_shape(2, 2 * n, n, hq, hkv, d, block)
    nbs = bsa.varlen_block_stride(s)
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    rnd = lambda *shape: torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()
    q, k, v = rnd(2, hq, d), rnd(2 * n, hkv, d), rnd(2 * n, hkv, d)
    meta = bsa.alloc_varlen_meta(s)
    bsa.varlen_block_meta(s, cu, k, meta["centroid"], meta["radius"], meta["quant"], meta["alpha"])
    used = -(-n // block)
    idx = torch.arange(nbs, dtype=torch.int32, device="cuda").expand(2, hkv, nbs).contiguous()
    cnt = torch.full((2, hkv), used, dtype=torch.int32, device="cuda")

    def run(q):
        o, lse = torch.zeros(2, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, hq, device="cuda")
        bsa.decode_fwd(s, cu, q, k, v, idx, cnt, 1 / math.sqrt(d), o, lse)
        o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
        bsa.decode_step(s, bsa.SelectParams(0.5, 0.1, 0), cu, q, k, v, meta["centroid"], meta["radius"], meta["alpha"],
                        1 / math.sqrt(d), idx.clone(), cnt.clone(), o2, lse2)
        torch.cuda.synchronize()
        return o, lse, o2, lse2

    want = run(q)
    h = hq - 1
    q[1, h, 5] = NAN
    got = run(q)
    for x in got:
        assert torch.isnan(x[1, h].float()).all()
    for x, w in zip(got[:2], want[:2]):                        # (the step's selection sees the NaN too)
        x[1, h] = w[1, h]
        assert torch.equal(x, w)
    for x, w in zip(got[2:], want[2:]):
        assert torch.equal(x[0], w[0]) and torch.isfinite(x[0].float()).all()


# ---------------------------------------------------------------- held in the cache

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_cache_holds_inf_and_nan_as_documented(fmt, d):
    """Written and read back: BF16 as they are; E4M3 as NaN; E2M1 as NaN for the 16 dimensions of their group.
    The other elements have the bytes of a row with zeros in their place."""
    import block_sparse_long_kv_gb300 as bsa
    n, hkv = 90, 2
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(n, hkv, d, generator=g) * 10.0 ** torch.randint(-3, 3, (n, hkv, 1), generator=g)).to(torch.bfloat16)
    bad = torch.zeros(n, hkv, d, dtype=torch.bool)
    for t in range(n):
        kind = t % 6
        if kind < 3:
            bad[t, t % hkv, torch.randperm(d, generator=g)[:1 + 3 * kind]] = True
        elif kind == 3:
            bad[t] = True                                      # nothing but Inf and NaN
        elif kind == 4:
            bad[t, :, 16:32] = True
    clean = torch.where(bad, torch.zeros_like(x), x)
    x = torch.where(bad, torch.tensor([NAN, INF, -INF]).to(torch.bfloat16)[torch.randint(0, 3, x.shape, generator=g)], x)
    cs = bsa.make_cache_shape(2, 64, hkv, d, fmt)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    out = []
    for rows in (x, clean):
        cache = bsa.alloc_cache(cs)
        for t in cache.values():
            if t is not None:
                t.fill_(0xA7)
        bsa.cache_write(cs, rows.cuda(), -rows.cuda(), slots, cache)
        ko, vo = torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda")
        bsa.cache_read(cs, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                       torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), n, cache, ko, vo)
        torch.cuda.synchronize()
        out.append((cache, ko.cpu(), vo.cpu()))
    (got, gk, gv), (want, wk, wv) = out
    if fmt == C.BF16:
        assert same(gk, x) and same(gv, -x)
        return
    lost = bad if fmt == C.E4M3 else bad.view(n, hkv, d // 16, 16).any(-1, keepdim=True).expand(n, hkv, d // 16, 16).reshape(n, hkv, d)
    for a, b in ((gk, wk), (gv, wv)):
        assert torch.isnan(a[lost].float()).all()
        # in E2M1 the lost group's finite elements do not count in the row's exponent either
        clear = ~lost if fmt == C.E4M3 else ~lost & ~lost.any(-1, keepdim=True)
        assert torch.equal(a[clear], b[clear])
    whole = bad.any(-1) & ~bad.all(-1) if fmt == C.E2M1 else torch.zeros(n, hkv, dtype=torch.bool)
    if whole.any():                                            # those rows: as written with the whole group zero
        zero = torch.where(lost, torch.zeros_like(x), x)
        held = torch.from_numpy(C.held(zero.double().numpy(), fmt))
        assert torch.equal(gk[~lost].double(), held[~lost])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("drafts", DRAFTS)
def test_attention_over_held_nan(fmt, drafts):
    """A cached key of NaN makes its head's rows NaN; a cached value of NaN the dimensions it is held in."""
    c = Case(fmt, [300], [drafts], 8, 2, 128, 64, seed=drafts)
    slots = c.table[0].numpy()[torch.arange(300).numpy() // 64] * 64 + torch.arange(300).numpy() % 64
    c.v[100, 1, 20] = 0
    if fmt == C.E2M1:
        c.v[100, 1, 16:32] = 0
    write = lambda: c.bsa.cache_write(c.cs, c.k.cuda(), c.v.cuda(), torch.from_numpy(slots.astype("int32")).cuda(), c.cache)
    write()
    want, wl = c.run()
    c.k[200, 0, 7] = NAN
    c.v[100, 1, 20] = NAN
    write()
    got, gl = c.run()
    assert torch.isnan(got[:, :4].float()).all() and torch.isnan(gl[:, :4]).all()
    assert torch.equal(gl[:, 4:], wl[:, 4:])
    lost = torch.zeros(128, dtype=torch.bool)
    lost[slice(16, 32) if fmt == C.E2M1 else 20] = True
    assert torch.isnan(got[:, 4:][..., lost].float()).all()
    assert torch.equal(got[:, 4:][..., ~lost], want[:, 4:][..., ~lost])
