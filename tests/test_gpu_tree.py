"""bsa_tree_fwd on the GPU against the float64 reference.

Tolerance, before the first run.  Logits: exact products summed in fp32, off by at most
delta = (d + 8) 2^-24 max_s scale sum_x |q_x k_x| (+ 2^-20 in log units for the exponentials), and as
much again for an f16 query element that lies 2^28 below its row's largest.  P is rounded to bf16
(2^-8 of each term) or f16 (2^-11), sums are fp32, and O is rounded to bf16: with
A = sum p |v| / sum p,  |O - ref| <= (2^-8 + 4 delta + 2^-18) A + 2^-8 |ref|,  and
|lse - ref| <= 2 delta + 2^-20 (1 + |ref|).
An 8- or 4-bit cache is computed in f16, whose smallest step is 2^-24, so small terms keep an absolute
error.  With few rows P' = p 2^(e - eref + 11), p <= 16: a key's term is off by at most 2^-25-11 |code|
2^eref, a code is at most 448 (2688) and the row that set eref has its largest value above half of that
times 2^eref, so by 2^-35 vmax, vmax the largest |v|.  With many rows P' = p 2^11 with p <= 16, off by 2^-36 of
values up to vmax, and V' holds vmax above 2^13, so it is off by 2^-38 vmax itself.  p of the largest
logit is at least 1, hence sum p >= 1, and n keys add at most n 2^-35 vmax (a softmax so sharp that A
itself is below 2^-28 meets it).
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu
FMTS = [C.BF16, C.E4M3, C.E2M1]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_kv_gb300 import build
    build.build()


def bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


class Case:
    """A batch: cached tokens in shuffled pages of a cache full of garbage, and its drafts."""

    def __init__(self, fmt, lengths, drafts, hq, hkv, d, page, chain=False, keep=None, seed=0, spread=0, deep=False):
        import block_sparse_long_kv_gb300 as bsa
        self.bsa, self.fmt, self.lengths, self.drafts = bsa, fmt, lengths, drafts
        self.hq, self.hkv, self.d, self.page, self.group = hq, hkv, d, page, hq // hkv
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.rng = rng
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + 2
        self.stride = max(max(need), 1) + 1
        self.cs = bsa.make_cache_shape(pages, page, hkv, d, fmt)
        self.cache = bsa.alloc_cache(self.cs)
        for t in self.cache.values():
            if t is not None:
                t.fill_(0xFF)                                 # NaN codes and scales wherever nobody writes
        order = rng.permutation(pages)
        self.table = torch.full((len(lengths), self.stride), -7, dtype=torch.int32)
        slots, at = [], 0
        for b, n in enumerate(lengths):
            self.table[b, :need[b]] = torch.from_numpy(order[at:at + need[b]].astype(np.int32))
            at += need[b]
            i = np.arange(n)
            slots.append(self.table[b].numpy()[i // page] * page + i % page)
        slots = np.concatenate(slots).astype(np.int32)
        n = len(slots)
        # rows of different sizes, so that the row exponents differ by up to `spread` powers of ten
        mul = lambda m: torch.from_numpy(10.0 ** rng.uniform(-spread, 0, size=(m, hkv, 1))).float()
        self.k = (bf(g, n, hkv, d).float() * mul(n)).to(torch.bfloat16)
        self.v = (bf(g, n, hkv, d).float() * mul(n)).to(torch.bfloat16)
        if n:
            bsa.cache_write(self.cs, self.k.cuda(), self.v.cuda(), torch.from_numpy(slots).cuda(), self.cache)
        t = sum(drafts)
        self.q, self.k_new, self.v_new = bf(g, t, hq, d), bf(g, t, hkv, d), bf(g, t, hkv, d)
        self.parents = [[] for _ in drafts]
        for b, m in enumerate(drafts):
            self.parents[b] = [(i - 1 if chain or deep else int(max(-1, i - 1 - rng.integers(0, 4)))) for i in range(m)]
        self.chain = chain
        self.lists = None
        if keep is not None:
            self.lists = [[sorted(set(rng.permutation(max(c, 1))[:max(1, int(keep * c))].tolist()) if c else [])
                           for _ in range(hkv)] for c in need]

    def run(self, lse=True, workspace=None, stream=None, out=None):
        bsa, b, t = self.bsa, len(self.lengths), sum(self.drafts)
        cu = torch.tensor([0] + np.cumsum(self.drafts).tolist(), dtype=torch.int32, device="cuda")
        par = None if self.chain else torch.tensor(sum(self.parents, []), dtype=torch.int32, device="cuda")
        idx = cnt = None
        if self.lists is not None:
            idx = torch.full((b, self.hkv, self.stride), 1 << 20, dtype=torch.int32)
            cnt = torch.zeros(b, self.hkv, dtype=torch.int32)
            for x in range(b):
                for g in range(self.hkv):
                    row = self.lists[x][g]
                    idx[x, g, :len(row)] = torch.tensor(row, dtype=torch.int32)
                    cnt[x, g] = len(row)
            idx, cnt = idx.cuda(), cnt.cuda()
        ts = bsa.make_tree_shape(b, t, max(max(self.drafts), 1), max(self.lengths), self.hq, self.stride)
        o = torch.full((t, self.hq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
        l = torch.full((t, self.hq), float("nan"), device="cuda") if lse else None
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        if workspace is None:
            workspace = torch.full((bsa.tree_workspace_bytes(ts, self.cs),), 0xFF, dtype=torch.uint8, device="cuda")
        bsa.tree_fwd(ts, self.cs, cu, torch.tensor(self.lengths, dtype=torch.int32, device="cuda"), self.table.cuda(), par,
                     self.q.cuda(), self.k_new.cuda(), self.v_new.cuda(), self.cache, idx, cnt, 1 / math.sqrt(self.d), o, l,
                     workspace, st, stream)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return o, l

    def check(self, o, lse, parents=None):
        parents = parents or self.parents
        hk, hv = C.held(self.k.double().numpy(), self.fmt), C.held(self.v.double().numpy(), self.fmt)
        got, gl = o.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
        f0 = t0 = 0
        scale, worst = 1 / math.sqrt(self.d), 0.0
        for b, (n, t) in enumerate(zip(self.lengths, self.drafts)):
            for g in range(self.hkv):
                at = np.arange(n)
                if self.lists is not None:
                    at = at[np.isin(at // self.page, self.lists[b][g])]
                hs = slice(g * self.group, (g + 1) * self.group)
                want, wl, a, reach = C.tree_attention(
                    self.q[t0:t0 + t, hs].double().numpy(), self.k_new[t0:t0 + t, g].double().numpy(),
                    self.v_new[t0:t0 + t, g].double().numpy(), hk[f0:f0 + n, g][at], hv[f0:f0 + n, g][at], parents[b], scale)
                delta = 2 * (self.d + 8) * 2.0 ** -24 * reach + 2.0 ** -20
                tol = (2.0 ** -8 + 4 * delta[..., None] + 2.0 ** -18) * a + 2.0 ** -8 * np.abs(want)
                if self.fmt != C.BF16 and at.size:
                    vmax = max(np.abs(hv[f0:f0 + n, g][at]).max(), self.v_new[t0:t0 + t, g].abs().max().item() if t else 0.0)
                    tol = tol + (at.size + t) * 2.0 ** -35 * vmax
                err = np.abs(got[t0:t0 + t, hs] - want)
                assert (err <= tol).all(), (b, g, float((err / np.maximum(tol, 1e-30)).max()))
                worst = max(worst, float((err / np.maximum(tol, 1e-30)).max()) if err.size else 0.0)
                if gl is not None:
                    assert (np.abs(gl[t0:t0 + t, hs] - wl) <= 2 * delta + 2.0 ** -20 * (1 + np.abs(wl))).all()
            f0 += n
            t0 += t
        return worst


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths, drafts, hq, hkv, page", [
    ([1], [1], 1, 1, 64), ([63], [1], 4, 2, 64), ([64], [2], 8, 1, 64), ([129], [3], 16, 1, 128),
    ([0], [5], 4, 2, 64), ([700], [1], 32, 4, 128)])
def test_small_steps(fmt, d, lengths, drafts, hq, hkv, page):
    c = Case(fmt, lengths, drafts, hq, hkv, d, page)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_batches(fmt, d, group):
    c = Case(fmt, [513, 0, 130, 1000, 64], [7, 3, 0, 1, 16], 2 * group, 2, d, 128, seed=group)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("drafts, chain, deep", [([64], False, False), ([65], True, False), ([130], False, True),
                                                 ([256], False, False), ([256, 3], True, False)])
def test_wide_and_deep_trees(fmt, drafts, chain, deep):
    c = Case(fmt, [300] * len(drafts), drafts, 8, 2, 128, 64, chain=chain, deep=deep)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [64, 128, 256])
def test_kept_pages(fmt, page):
    c = Case(fmt, [3000, 77, 0, 1025], [5, 2, 1, 9], 8, 2, 128, page, keep=0.4, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_empty_lists_leave_the_drafts(fmt):
    c = Case(fmt, [500, 200], [4, 3], 8, 2, 64, 64, keep=0.5)
    c.lists = [[[], [0, 7]], [[], []]]
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_many_splits_and_a_long_cache(fmt, d):
    c = Case(fmt, [40000, 9000], [2, 1], 16, 2, d, 256, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [C.E4M3, C.E2M1])
def test_rows_of_very_different_sizes(fmt):
    """Row exponents that differ by up to 2^13 between the keys of one softmax."""
    c = Case(fmt, [900], [6], 8, 2, 128, 64, spread=4, seed=5)
    c.check(*c.run())
    c.v[:, :, :] = 0                                            # all value rows zero, one huge at the end
    c.v[-1] = 3.0e4
    slots = c.table[0].numpy()[np.arange(900) // 64] * 64 + np.arange(900) % 64
    c.bsa.cache_write(c.cs, c.k.cuda(), c.v.cuda(), torch.from_numpy(slots.astype(np.int32)).cuda(), c.cache)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_large_logits(fmt):
    c = Case(fmt, [400], [4], 4, 1, 64, 64, seed=6)
    c.q = (c.q.float() * 30).to(torch.bfloat16)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_twice_the_same_bits_and_without_lse(fmt):
    c = Case(fmt, [5000, 300, 1], [5, 17, 2], 8, 2, 128, 128, keep=0.5)
    o, lse = c.run()
    o2, lse2 = c.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, _ = c.run(lse=False)
    assert torch.equal(o, o3)


def test_rows_behind_the_last_sequence_stay():
    c = Case(C.E4M3, [300, 10], [3, 2], 8, 2, 128, 128)
    bsa = c.bsa
    o = torch.full((9, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 8), 5.0, device="cuda")
    pad = lambda t: torch.cat([t, torch.full((4, *t.shape[1:]), float("nan"), dtype=t.dtype)]).cuda()
    ts = bsa.make_tree_shape(2, 9, 3, 300, 8, c.stride)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.tree_fwd(ts, c.cs, torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda"),
                 torch.tensor(c.lengths, dtype=torch.int32, device="cuda"), c.table.cuda(),
                 torch.tensor(sum(c.parents, []) + [99] * 4, dtype=torch.int32, device="cuda"), pad(c.q), pad(c.k_new),
                 pad(c.v_new), c.cache, None, None, 1 / math.sqrt(128), o, lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert (o[5:] == 5).all() and (lse[5:] == 5).all()
    c.check(o[:5], lse[:5])


def test_bad_device_arguments_are_reported_and_left_out():
    c = Case(C.E4M3, [300], [4], 8, 2, 128, 128)
    bsa = c.bsa
    ts = bsa.make_tree_shape(1, 4, 4, 300, 8, c.stride)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def run(cu=(0, 4), cached=(300,), table=None, parents=None):
        o = torch.full((4, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, 8), 5.0, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        bsa.tree_fwd(ts, c.cs, dev(cu), dev(cached), c.table.cuda() if table is None else table.cuda(),
                     dev(c.parents[0] if parents is None else parents), c.q.cuda(), c.k_new.cuda(), c.v_new.cuda(), c.cache,
                     None, None, 1 / math.sqrt(128), o, lse, dev_status=st)
        torch.cuda.synchronize()
        return o, lse, int(st.item())

    o, lse, code = run()
    assert code == 0
    c.check(o, lse)
    for cu in ((0, 5), (-1, 4), (3, 1)):
        o, lse, code = run(cu=cu)
        assert code == 1 and (o == 5).all() and (lse == 5).all()
    # an impossible cache length reads as an empty cache: the drafts alone
    for n in (-1, 301):
        o, lse, code = run(cached=(n,))
        assert code == 1
        keep, c.lists = c.lists, [[[], []]]
        c.check(o, lse)
        c.lists = keep
    # a bad page is left out
    for bad in (-1, c.cs.pages, 1 << 30):
        t = c.table.clone()
        t[0, 1] = bad
        o, lse, code = run(table=t)
        assert code == 1
        c.lists = [[[0, 2], [0, 2]]]
        c.check(o, lse)
        c.lists = None
    # a parent that is no earlier token reads as a root
    for bad in (2, 3, 1 << 30, -2):
        par = list(c.parents[0])
        par[2] = bad
        o, lse, code = run(parents=par)
        assert code == 1
        par[2] = -1
        c.check(o, lse, [par])


def test_two_streams_with_their_own_workspaces():
    a, b = Case(C.E4M3, [5000], [5], 16, 2, 128, 128, seed=1), Case(C.BF16, [4000], [3], 16, 2, 128, 128, seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            oa, la = a.run(stream=s1)
        with torch.cuda.stream(s2):
            ob, lb = b.run(stream=s2)
    a.check(oa, la)
    b.check(ob, lb)


def test_captured_step_follows_its_inputs():
    """One captured graph: lengths, table, drafts and cache contents change between replays."""
    import block_sparse_long_kv_gb300 as bsa
    cases = [Case(C.E2M1, [900, 300], [5, 2], 8, 2, 128, 64, seed=s) for s in (1, 2)]
    c = cases[0]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t = 7
    ts = bsa.make_tree_shape(2, t, 6, 1000, 8, 17)
    cs = c.cs
    cu, cached = dev([0, 5, 7]), dev([900, 300])
    table = torch.zeros(2, 17, dtype=torch.int32, device="cuda")
    par = dev([0] * t)
    q, kn, vn = (torch.zeros_like(x).cuda() for x in (c.q, c.k_new, c.v_new))
    o, lse = torch.zeros(t, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(t, 8, device="cuda")
    ws = torch.empty(bsa.tree_workspace_bytes(ts, cs), dtype=torch.uint8, device="cuda")
    cache = {n: x.clone() for n, x in c.cache.items()}
    st = dev([0])
    call = lambda: bsa.tree_fwd(ts, cs, cu, cached, table, par, q, kn, vn, cache, None, None, 1 / math.sqrt(128), o, lse, ws, st)
    call()
    torch.cuda.synchronize()
    st.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in cases:
        table[:, :x.stride] = x.table.cuda()
        par.copy_(dev(sum(x.parents, [])))
        for dst, src in ((q, x.q), (kn, x.k_new), (vn, x.v_new)):
            dst.copy_(src)
        for n in cache:
            cache[n].copy_(x.cache[n])
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        x.check(o, lse)


def test_serving_run():
    """The operators together, as a server runs them: norm and rotate a prompt, write its keys and values,
    read them back for the block summaries, select, and verify a tree of drafts over the kept pages; then
    accept one path into the cache and take a plain step over the longer sequence."""
    import block_sparse_long_kv_gb300 as bsa
    hq, hkv, d, page, n, t = 8, 2, 128, 64, 1000, 6
    g = torch.Generator().manual_seed(0)
    row = bf(g, n + t, (hq + 2 * hkv) * d).cuda()
    q, k, v = (row[:, a * d:b * d].view(n + t, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    par = [-1, 0, 0, 1, 1, 3]
    depth = [0, 1, 1, 2, 2, 3]
    pos = torch.tensor(list(range(n)) + [n + x for x in depth], dtype=torch.int32, device="cuda")
    freq = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    qr, kr = torch.empty(n + t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(n + t, hkv, d, dtype=torch.bfloat16, device="cuda")
    bsa.qk_norm_rope(bsa.make_rope_shape(n + t, hq, hkv, d, d), q, k, None, None, pos, freq, qr, kr)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for fmt in FMTS:
        cs = bsa.make_cache_shape(20, page, hkv, d, fmt)
        cache = bsa.alloc_cache(cs)
        table = torch.randperm(20, generator=g)[None].int().cuda()
        slot = lambda i: (table[0, i // page] * page + i % page).int()
        st = dev([0])
        bsa.cache_write(cs, kr[:n], v[:n], slot(torch.arange(n, device="cuda")), cache, st)
        ko, vo = torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda")
        cu = dev([0, n])
        bsa.cache_read(cs, cu, table, n, cache, ko, vo, st)
        vs = bsa.make_varlen_shape(1, n, n, hq, hkv, d, page)
        nbs = bsa.varlen_block_stride(vs)
        meta = bsa.alloc_varlen_meta(vs)
        bsa.varlen_block_meta(vs, cu, ko, meta["centroid"], meta["radius"], meta["quant"], meta["alpha"], st)
        idx, cnt = torch.zeros(1, hkv, nbs, dtype=torch.int32, device="cuda"), torch.zeros(1, hkv, dtype=torch.int32, device="cuda")
        bsa.decode_select(vs, bsa.SelectParams(0.3, 0.1, 0), cu, qr[n:n + 1], meta["centroid"], meta["radius"], meta["alpha"],
                          idx, cnt, dev_status=st)
        ts = bsa.make_tree_shape(1, t, t, n, hq, nbs)
        o, lse = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hq, device="cuda")
        bsa.tree_fwd(ts, cs, dev([0, t]), dev([n]), table[:, :nbs].contiguous(), dev(par), qr[n:], kr[n:], v[n:].contiguous(),
                     cache, idx, cnt, 1 / math.sqrt(d), o, lse, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        kept = [idx[0, x, :int(cnt[0, x])].tolist() for x in range(hkv)]
        assert all(r == sorted(set(r)) and r[0] == 0 and r[-1] == (n - 1) // page and len(r) < 16 for r in kept)
        hk, hv = C.held(kr[:n].double().cpu().numpy(), fmt), C.held(v[:n].double().cpu().numpy(), fmt)
        np.testing.assert_array_equal(ko.double().cpu().numpy(), hk)

        def check(o, lse, q0, q1, parents, length, lists, keys, vals):
            for x in range(hkv):
                at = np.arange(length)
                at = at if lists is None else at[np.isin(at // page, lists[x])]
                hs = slice(x * 4, x * 4 + 4)
                want, wl, a, reach = C.tree_attention(
                    qr[q0:q1, hs].double().cpu().numpy(), kr[q0:q1, x].double().cpu().numpy(),
                    v[q0:q1, x].double().cpu().numpy(), keys[at, x], vals[at, x], parents, 1 / math.sqrt(d))
                delta = 2 * (d + 8) * 2.0 ** -24 * reach + 2.0 ** -20
                tol = (2.0 ** -8 + 4 * delta[..., None] + 2.0 ** -18) * a + 2.0 ** -8 * np.abs(want)
                tol = tol + ((len(at) + 6) * 2.0 ** -35 * max(np.abs(vals[at, x]).max(), v[n:].abs().max().item()) if fmt != C.BF16 else 0.0)
                assert (np.abs(o[:, hs].double().cpu().numpy() - want) <= tol).all()
                assert (np.abs(lse[:, hs].double().cpu().numpy() - wl) <= 2 * delta + 2.0 ** -20 * (1 + np.abs(wl))).all()

        check(o, lse, n, n + t, par, n, kept, hk, hv)
        # the path 0, 1, 3 is accepted: its tokens follow the prompt in the cache, the others are left out
        slots = dev([-1] * t)
        take = [0, 1, 3]
        slots[take] = slot(n + torch.arange(3, device="cuda"))
        bsa.cache_write(cs, kr[n:], v[n:], slots, cache, st)
        ts = bsa.make_tree_shape(1, 1, 1, n + 3, hq, 20)
        o, lse = torch.empty(1, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, hq, device="cuda")
        bsa.tree_fwd(ts, cs, dev([0, 1]), dev([n + 3]), table, None, qr[n + 5:], kr[n + 5:], v[n + 5:].contiguous(), cache,
                     None, None, 1 / math.sqrt(d), o, lse, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        at = [n + x for x in take]
        hk = np.concatenate([hk, C.held(kr[at].double().cpu().numpy(), fmt)])
        hv = np.concatenate([hv, C.held(v[at].double().cpu().numpy(), fmt)])
        check(o, lse, n + 5, n + 6, [-1], n + 3, None, hk, hv)


def test_python_refusals():
    c = Case(C.BF16, [300], [4], 8, 2, 128, 128)
    bsa = c.bsa
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ts = bsa.make_tree_shape(1, 4, 4, 300, 8, c.stride)
    o = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    base = dict(cu=dev([0, 4]), cached=dev([300]), table=c.table.cuda(), parents=None, q=c.q.cuda(), k=c.k_new.cuda(),
                v=c.v_new.cuda(), o=o, lse=None, ts=ts, ws=None)

    def call(**kw):
        a = dict(base, **kw)
        bsa.tree_fwd(a["ts"], c.cs, a["cu"], a["cached"], a["table"], a["parents"], a["q"], a["k"], a["v"], c.cache, None,
                     None, 0.1, a["o"], a["lse"], a["ws"])

    call()
    for kw, err in ((dict(q=c.q.cuda().float()), TypeError), (dict(k=c.k_new), TypeError), (dict(cached=dev([300]).long()), TypeError),
                    (dict(o=o[:3]), ValueError), (dict(table=c.table[:, :1].contiguous().cuda()), ValueError),
                    (dict(parents=dev([0])), ValueError), (dict(lse=torch.zeros(4, 4, device="cuda")), ValueError),
                    (dict(q=c.q.cuda().transpose(0, 1)), ValueError), (dict(cu=dev([0])), ValueError),
                    (dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")), RuntimeError),
                    (dict(ts=bsa.make_tree_shape(1, 4, 4, 300 * 128, 8, c.stride)), RuntimeError)):
        with pytest.raises(err):
            call(**kw)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- many query rows (drafted tokens x heads > 16)

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [64, 128, 256])
def test_kept_pages_with_many_rows(fmt, page):
    c = Case(fmt, [3000, 77, 0, 1025], [40, 33, 18, 64], 8, 2, 128, page, keep=0.4, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("drafts", [20, 40])
def test_bad_device_arguments_with_many_rows(drafts):
    c = Case(C.E4M3, [300], [drafts], 8, 2, 128, 128)
    bsa = c.bsa
    ts = bsa.make_tree_shape(1, drafts, drafts, 300, 8, c.stride)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def run(cu=(0, drafts), cached=(300,), table=None, parents=None):
        o = torch.full((drafts, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((drafts, 8), 5.0, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        bsa.tree_fwd(ts, c.cs, dev(cu), dev(cached), c.table.cuda() if table is None else table.cuda(),
                     dev(c.parents[0] if parents is None else parents), c.q.cuda(), c.k_new.cuda(), c.v_new.cuda(), c.cache,
                     None, None, 1 / math.sqrt(128), o, lse, dev_status=st)
        torch.cuda.synchronize()
        return o, lse, int(st.item())

    o, lse, code = run()
    assert code == 0
    c.check(o, lse)
    for cu in ((0, drafts + 1), (-1, drafts), (3, 1)):
        o, lse, code = run(cu=cu)
        assert code == 1 and (o == 5).all() and (lse == 5).all()
    for n in (-1, 301):                                         # reads as an empty cache
        o, lse, code = run(cached=(n,))
        assert code == 1
        keep, c.lists = c.lists, [[[], []]]
        c.check(o, lse)
        c.lists = keep
    for bad in (-1, c.cs.pages, 1 << 30):                       # a page that is left out
        t = c.table.clone()
        t[0, 1] = bad
        o, lse, code = run(table=t)
        assert code == 1
        c.lists = [[[0, 2], [0, 2]]]
        c.check(o, lse)
        c.lists = None
    for bad in (2, 3, 1 << 30, -2):                             # a parent that reads as a root
        par = list(c.parents[0])
        par[2] = bad
        o, lse, code = run(parents=par)
        assert code == 1
        par[2] = -1
        c.check(o, lse, [par])


@pytest.mark.parametrize("first", [19, 50])
def test_rows_behind_the_last_sequence_stay_with_many_rows(first):
    c = Case(C.E2M1, [300, 10], [first, 18], 8, 2, 128, 128)
    bsa, t = c.bsa, first + 18
    o = torch.full((t + 4, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((t + 4, 8), 5.0, device="cuda")
    pad = lambda x: torch.cat([x, torch.full((4, *x.shape[1:]), float("nan"), dtype=x.dtype)]).cuda()
    ts = bsa.make_tree_shape(2, t + 4, first, 300, 8, c.stride)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.tree_fwd(ts, c.cs, torch.tensor([0, first, t], dtype=torch.int32, device="cuda"),
                 torch.tensor(c.lengths, dtype=torch.int32, device="cuda"), c.table.cuda(),
                 torch.tensor(sum(c.parents, []) + [99] * 4, dtype=torch.int32, device="cuda"), pad(c.q), pad(c.k_new),
                 pad(c.v_new), c.cache, None, None, 1 / math.sqrt(128), o, lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert (o[t:] == 5).all() and (lse[t:] == 5).all()
    c.check(o[:t], lse[:t])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("drafts", [4, 20, 70])
def test_a_branch_with_nan_and_inf_does_not_reach_the_others(fmt, drafts):
    """Drafted tokens that nobody descends from hold infinities and NaN; every other token's result is that with
    zeros in their place, bit for bit."""
    c = Case(fmt, [200], [drafts], 8, 2, 128, 64)
    leaves = [i for i in range(drafts) if i not in c.parents[0]][:3] if drafts > 4 else [3]
    if drafts == 4:
        c.parents[0] = [-1, 0, 1, 0]
    bad = [float("nan"), float("inf"), -float("inf")]
    clean = []
    for x, poison in ((c.k_new, bad), (c.v_new, bad[::-1])):
        for i, leaf in enumerate(leaves):
            x[leaf] = 0
            clean.append((x, leaf, poison[i]))
    want, wl = c.run()
    for x, leaf, value in clean:
        x[leaf, :, ::3] = value
    got, gl = c.run()
    keep = [i for i in range(drafts) if i not in leaves]
    assert torch.equal(got[keep], want[keep]) and torch.equal(gl[keep], wl[keep])
    assert torch.isfinite(got[keep].float()).all() and torch.isfinite(gl[keep]).all()


@pytest.mark.parametrize("fmt, batch, hkv, drafts", [(C.E4M3, 300, 4, 17), (C.BF16, 300, 4, 17), (C.E2M1, 1024, 4, 3),
                                                     (C.E4M3, 1024, 4, 1)])
def test_very_many_short_sequences(fmt, batch, hkv, drafts):
    """Runs of a CTA that cross many row tiles, some of one unit only, up to the largest number of groups."""
    lengths = [(7 * b) % 70 if b % 11 else 0 for b in range(batch)]
    c = Case(fmt, lengths, [max(0, drafts - b % 3) for b in range(batch)], 8 * hkv, hkv, 64, 64, seed=batch)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch, drafts", [(38, 8), (3, 256)])
def test_runs_of_many_units(fmt, batch, drafts):
    """Every CTA walks more than 128 units: one row tile of 128 rows each, and sixteen tiles of 256."""
    import block_sparse_long_kv_gb300 as bsa
    hkv, group, d, page, pages, n = 2, 16, 64, 256, 40, 33000
    hq, scale = hkv * group, 0.125
    g = torch.Generator().manual_seed(drafts)
    cs = bsa.make_cache_shape(pages, page, hkv, d, fmt)
    cache = bsa.alloc_cache(cs)
    k, v = bf(g, pages * page, hkv, d), bf(g, pages * page, hkv, d)
    bsa.cache_write(cs, k.cuda(), v.cuda(), torch.arange(pages * page, dtype=torch.int32, device="cuda"), cache)
    hk, hv = (torch.from_numpy(C.held(x.double().numpy(), fmt)).cuda() for x in (k, v))
    stride = -(-n // page)
    table = torch.randint(0, pages, (batch, stride), generator=g, dtype=torch.int32)
    lengths = [n - 77 * b for b in range(batch)]
    t = batch * drafts
    q, kn, vn = bf(g, t, hq, d), bf(g, t, hkv, d), bf(g, t, hkv, d)
    par = torch.tensor([max(-1, i - 1 - i % 3) for i in range(drafts)], dtype=torch.int32)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ts = bsa.make_tree_shape(batch, t, drafts, n, hq, stride)
    o, lse = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hq, device="cuda")
    st = dev([0])
    bsa.tree_fwd(ts, cs, dev([drafts * b for b in range(batch + 1)]), dev(lengths), table.cuda(), par.repeat(batch).cuda(),
                 q.cuda(), kn.cuda(), vn.cuda(), cache, None, None, scale, o, lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    sees = torch.zeros(drafts, drafts, dtype=torch.bool)
    for i in range(drafts):
        p = i
        while p >= 0:
            sees[i, p] = True
            p = int(par[p])
    hidden = ~sees.cuda().repeat_interleave(group, 0)
    for b in range(batch):
        i = torch.arange(lengths[b])
        at = (table[b].long()[i // page] * page + i % page).cuda()
        rows = slice(b * drafts, (b + 1) * drafts)
        for x in range(hkv):
            qq = q[rows, x * group:(x + 1) * group].double().cuda().reshape(-1, d)
            kk = torch.cat([hk[at, x], kn[rows, x].double().cuda()])
            vv = torch.cat([hv[at, x], vn[rows, x].double().cuda()])
            s = scale * qq @ kk.T
            s[:, lengths[b]:].masked_fill_(hidden, -math.inf)
            reach = (scale * qq.abs() @ kk.abs().T).amax(-1)
            wl = torch.logsumexp(s, -1)
            p = torch.exp(s - wl[:, None])
            want, a = p @ vv, p @ vv.abs()
            delta = 2 * (d + 8) * 2.0 ** -24 * reach + 2.0 ** -20
            tol = (2.0 ** -8 + 4 * delta[:, None] + 2.0 ** -18) * a + 2.0 ** -8 * want.abs()
            if fmt != C.BF16:
                tol = tol + len(kk) * 2.0 ** -35 * vv.abs().max()
            got = o[rows, x * group:(x + 1) * group].double().reshape(-1, d)
            assert ((got - want).abs() <= tol).all(), (b, x)
            gl = lse[rows, x * group:(x + 1) * group].double().reshape(-1)
            assert ((gl - wl).abs() <= 2 * delta + 2.0 ** -20 * (1 + wl.abs())).all(), (b, x)


@pytest.mark.parametrize("drafts", [[20, 18], [40, 33]])
def test_two_captured_graphs_share_a_workspace(drafts):
    """Replayed one after the other on one stream, each gives its eager call's bits."""
    cases = [Case(f, [900, 300], drafts, 8, 2, 128, 64, seed=s) for f, s in ((C.E2M1, 1), (C.BF16, 2))]
    bsa = cases[0].bsa
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ts = bsa.make_tree_shape(2, sum(drafts), max(drafts), 900, 8, cases[0].stride)
    ws = torch.empty(max(bsa.tree_workspace_bytes(ts, c.cs) for c in cases), dtype=torch.uint8, device="cuda")
    graphs, outs, held, want = [], [], [], [c.run() for c in cases]
    for c in cases:
        o, lse, st = torch.zeros(sum(drafts), 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(sum(drafts), 8, device="cuda"), dev([0])
        args = (ts, c.cs, dev([0, drafts[0], sum(drafts)]), dev([900, 300]), c.table.cuda(), dev(sum(c.parents, [])), c.q.cuda(),
                c.k_new.cuda(), c.v_new.cuda(), c.cache, None, None, 1 / math.sqrt(128), o, lse, ws, st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bsa.tree_fwd(*args)
        graphs.append(graph)
        outs.append((o, lse, st))
        held.append(args)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (o, lse, st), (wo, wl) in zip(outs, want):
        assert int(st.item()) == 0 and torch.equal(o, wo) and torch.equal(lse, wl)


def test_calls_from_two_threads_with_different_batches():
    """The library is called without Python's lock: a small batch and one whose plan takes more shared memory."""
    import threading
    cases = [Case(C.E4M3, [300], [20], 8, 2, 128, 64, seed=1),
             Case(C.E4M3, [10] * 400, [5] * 400, 8, 2, 128, 64, seed=2),
             Case(C.E4M3, [300], [2], 8, 2, 128, 64, seed=3),
             Case(C.E4M3, [10] * 400, [1] * 400, 8, 2, 128, 64, seed=4)]
    want, got, failed = [c.run() for c in cases], [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = cases[i].run(stream=torch.cuda.current_stream())
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for (o, lse), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("fmt, pages", [(C.BF16, 150000), (C.E4M3, 300000), (C.E2M1, 600000)])
@pytest.mark.parametrize("drafts", [2, 20, 40])
def test_pages_past_32_bit_offsets(fmt, pages, drafts):
    c = Case(fmt, [500, 70], [drafts, 1], 8, 2, 128, 64, seed=drafts)
    few = c.cs.pages
    cs = c.bsa.make_cache_shape(pages, 64, 2, 128, fmt)
    assert c.bsa.cache_code_bytes(cs) > 1 << 32
    big = c.bsa.alloc_cache(cs)
    for name, x in c.cache.items():
        if x is not None:
            big[name][pages - few:] = x
    c.cs, c.cache = cs, big
    c.table = torch.where(c.table >= 0, c.table + (pages - few), c.table)
    c.check(*c.run())
