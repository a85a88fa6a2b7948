"""bsa_shared_fwd on the GPU against the float64 reference.

Tolerance, before the first run.  Logits: exact products summed in fp32, off by at most
delta = (d + 8) 2^-24 max_s scale sum_x |q_x k_x| (+ 2^-20 in log units for the exponentials), and as much again for an
f16 query element that lies 2^28 below its row's largest.  P is rounded to bf16 (2^-8 of each term) or f16 (2^-11), sums
are fp32, and O is rounded to bf16: with A = sum p |v| / sum p,
|O - ref| <= (2^-8 + 4 delta + 2^-18) A + 2^-8 |ref|,  and  |lse - ref| <= 2 delta + 2^-20 (1 + |ref|).
An 8- or 4-bit cache is computed in f16: P' = p 2^11 with p <= 16 is off by at most 2^-36 of values up to vmax, and V' holds
vmax above 2^13, so it is off by 2^-38 vmax itself, where vmax is the largest |v| of the sequences computed together: those of
a group.  p of the largest logit is at least 1, hence sum p >= 1, and n keys add at most n 2^-35 vmax.
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Groups of (shared pages, tails, drafts): sequences of shared pages * page + tail cached tokens, in shuffled pages of
    a cache full of garbage, and their drafts."""

    def __init__(self, fmt, groups, hq, hkv, d, page, chain=False, seed=0, extra=0, first_page=0):
        import block_sparse_long_kv_gb300 as bsa
        self.bsa, self.fmt, self.groups, self.hq, self.hkv, self.d, self.page = bsa, fmt, groups, hq, hkv, d, page
        self.group, self.chain, self.extra = hq // hkv, chain, extra
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lengths = [p * page + t for p, tails, _ in groups for t in tails]
        self.drafts = [t for _, _, drafts in groups for t in drafts]
        self.of = [y for y, (_, tails, _) in enumerate(groups) for _ in tails]
        pages = sum(p + sum(-(-t // page) for t in tails) for p, tails, _ in groups) + 2
        self.stride = max(-(-n // page) for n in self.lengths) + 1
        self.cs = bsa.make_cache_shape(first_page + pages, page, hkv, d, fmt)
        self.cache = bsa.alloc_cache(self.cs)
        for t in self.cache.values():
            if t is not None:
                t.fill_(0xFF)                                 # NaN codes and scales wherever nobody writes
        order = first_page + rng.permutation(pages)
        self.table = torch.full((len(self.lengths), self.stride), -7, dtype=torch.int32)
        at, b, slots, self.rows, n_rows = 0, 0, [], [], 0     # rows: of k and v that a sequence holds
        for p, tails, _ in groups:
            common = order[at:at + p]
            at += p
            slots.append((common[:, None] * page + np.arange(page)).reshape(-1))
            shared_rows = np.arange(n_rows, n_rows + p * page)
            n_rows += p * page
            for tail in tails:
                mine = order[at:at + -(-tail // page)]
                at += len(mine)
                self.table[b, :p] = torch.from_numpy(common.astype(np.int32))
                self.table[b, p:p + len(mine)] = torch.from_numpy(mine.astype(np.int32))
                i = np.arange(tail)
                slots.append(mine[i // page] * page + i % page if tail else i)
                self.rows.append(np.concatenate([shared_rows, np.arange(n_rows, n_rows + tail)]))
                n_rows += tail
                b += 1
        slots = np.concatenate(slots).astype(np.int32)
        bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
        self.k, self.v = bf(n_rows, hkv, d), bf(n_rows, hkv, d)
        self.slots = torch.from_numpy(slots).cuda()
        self.write()
        t = sum(self.drafts)
        self.q, self.k_new, self.v_new = bf(t + extra, hq, d), bf(t + extra, hkv, d), bf(t + extra, hkv, d)
        self.parents = [[i - 1 if chain else int(max(-1, i - 1 - rng.integers(0, 4))) for i in range(m)] for m in self.drafts]
        self.cu_group = [0] + np.cumsum([len(tails) for _, tails, _ in groups]).tolist()
        self.shared = [p for p, _, _ in groups]

    def write(self):
        if len(self.slots):
            self.bsa.cache_write(self.cs, self.k.cuda(), self.v.cuda(), self.slots, self.cache)

    def args(self, **over):
        bsa, t = self.bsa, sum(self.drafts) + self.extra
        a = dict(cu_group=i32(self.cu_group), shared_pages=i32(self.shared), cu_draft=i32([0] + np.cumsum(self.drafts).tolist()),
                 cached=i32(self.lengths), block_table=self.table.cuda(),
                 parents=None if self.chain else i32(sum(self.parents, []) + [0] * self.extra), q=self.q.cuda(),
                 k_new=self.k_new.cuda(), v_new=self.v_new.cuda())
        a.update(over)
        shape = bsa.make_shared_shape(len(self.groups), len(self.lengths), t, max(max(self.drafts), 1), max(self.lengths),
                                      self.hq, self.stride)
        return shape, a

    def run(self, want_status=0, lse=True, workspace=None, **over):
        shape, a = self.args(**over)
        t = sum(self.drafts) + self.extra
        o = torch.full((t, self.hq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        l = torch.full((t, self.hq), float("nan"), device="cuda") if lse else None
        st = i32([0])
        if workspace is None:
            workspace = torch.full((self.bsa.shared_workspace_bytes(shape, self.cs),), 0xFF, dtype=torch.uint8, device="cuda")
        self.bsa.shared_fwd(shape, self.cs, a["cu_group"], a["shared_pages"], a["cu_draft"], a["cached"], a["block_table"],
                            a["parents"], a["q"], a["k_new"], a["v_new"], self.cache, 1 / math.sqrt(self.d), o, l, workspace, st)
        torch.cuda.synchronize()
        assert int(st.item()) == want_status
        return o, l

    def check(self, o, lse, skip=(), drop=None, only=None):
        """skip: drafted tokens that are not looked at; drop(b): kept rows of the sequence's cached ones."""
        hk, hv = C.held(self.k.double().numpy(), self.fmt), C.held(self.v.double().numpy(), self.fmt)
        got, gl = o.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
        t0, scale, worst = 0, 1 / math.sqrt(self.d), 0.0
        vmax = [0.0] * len(self.groups)
        for b, y in enumerate(self.of):
            t1 = t0 + self.drafts[b]
            for x in (hv[self.rows[b]], self.v_new[t0:t1].double().numpy()):
                x = np.abs(x[np.isfinite(x)])
                vmax[y] = max(vmax[y], x.max() if x.size else 0.0)
            t0 = t1
        t0 = 0
        for b, t in enumerate(self.drafts):
            rows = self.rows[b] if drop is None else self.rows[b][drop(b)]
            look = [i for i in range(t) if t0 + i not in skip]
            if only is not None and b not in only:
                look = []
            for g in range(self.hkv):
                if not look:
                    break
                hs = slice(g * self.group, (g + 1) * self.group)
                clean = lambda x: np.nan_to_num(x.double().numpy(), nan=0.0, posinf=0.0, neginf=0.0)
                want, wl, a, reach = C.tree_attention(
                    clean(self.q[t0:t0 + t, hs]), clean(self.k_new[t0:t0 + t, g]), clean(self.v_new[t0:t0 + t, g]),
                    np.nan_to_num(hk[rows, g], nan=0.0, posinf=0.0, neginf=0.0),
                    np.nan_to_num(hv[rows, g], nan=0.0, posinf=0.0, neginf=0.0), self.parents[b], scale)
                delta = 2 * (self.d + 8) * 2.0 ** -24 * reach + 2.0 ** -20
                tol = (2.0 ** -8 + 4 * delta[..., None] + 2.0 ** -18) * a + 2.0 ** -8 * np.abs(want)
                if self.fmt != C.BF16:
                    tol = tol + (len(rows) + t) * 2.0 ** -35 * vmax[self.of[b]]
                err = np.abs(got[t0:t0 + t, hs] - want)[look] / np.maximum(tol, 1e-30)[look]
                assert (err <= 1).all(), (b, g, float(np.nanmax(err)), np.argwhere(~(err <= 1))[:4].tolist())
                worst = max(worst, float(err.max()))
                if gl is not None:
                    assert (np.abs(gl[t0:t0 + t, hs] - wl) <= 2 * delta + 2.0 ** -20 * (1 + np.abs(wl)))[look].all(), (b, g)
            t0 += t
        return worst


ONE = [(2, [0, 1, 130], [1, 1, 1])]
SOME = [(0, [70, 0], [2, 3]), (3, [0, 5, 64, 65], [1, 4, 0, 2]), (1, [200], [7])]
MANY = [(1, [(37 * i) % 151 for i in range(40)], [1 + (i % 5 == 0) for i in range(40)])]
HEADS = [(64, 1, 64), (128, 2, 128), (64, 4, 256), (128, 8, 64), (128, 16, 128), (64, 16, 64)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d, group, page", HEADS)
@pytest.mark.parametrize("groups", [ONE, SOME, MANY], ids=["one", "some", "many"])
def test_groups(fmt, d, group, page, groups):
    c = Case(fmt, groups, 2 * group, 2, d, page, seed=d + group)
    o, lse = c.run()
    c.check(o, lse)
    again, lse2 = c.run()
    assert torch.equal(o.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)     # the same bits


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [1, 4, 16])
@pytest.mark.parametrize("chain", [True, False])
def test_many_drafts(fmt, group, chain):
    """Up to 256 drafted tokens: a sequence of several row tiles, tiles of several sequences, tokens behind the last."""
    c = Case(fmt, [(1, [3, 100, 0], [256, 1, 100]), (2, [64], [129])], group, 1, 128, 64, chain=chain, seed=7, extra=5)
    o, lse = c.run()
    c.check(o, lse)
    assert torch.isnan(o[-5:]).all() and torch.isnan(lse[-5:]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_many_units_of_one_head(fmt):
    """Runs that end inside a group, at its own keys and at its drafts; without lse."""
    c = Case(fmt, [(70, [900, 5, 0], [3, 1, 2]), (33, [129, 640], [1, 1])], 8, 1, 128, 64, seed=3)
    c.check(c.run(lse=False)[0], None)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hkv", [1, 8])
def test_few_units(fmt, hkv):
    """Fewer units than CTAs: runs of a single place."""
    c = Case(fmt, [(1, [1, 700, 33, 0], [1, 1, 1, 1]), (0, [1], [1]), (0, [0], [1])], 2 * hkv, hkv, 64, 64, seed=9)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_empty_groups_and_sequences(fmt):
    c = Case(fmt, [(0, [], []), (1, [3, 9], [0, 2]), (0, [], []), (2, [1], [1]), (4, [10, 0], [0, 0]), (0, [], [])], 4, 2, 64,
             64, seed=4)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_the_same_as_without_sharing(fmt):
    """Groups of one sequence, groups that share fewer pages than they could, and none: all within the limits."""
    c = Case(fmt, [(3, [10, 0, 70], [2, 1, 4])], 8, 2, 128, 64, seed=5)
    o, lse = c.run()
    c.check(o, lse)
    c.check(*c.run(shared_pages=i32([1])))
    c.check(*c.run(shared_pages=i32([0])))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [2, 16])
@pytest.mark.parametrize("what", ["inf", "-inf", "nan"])
def test_values_that_are_not_finite(fmt, group, what):
    """Of drafted and own values, keys and queries: into the rows that see them and into no others."""
    c = Case(fmt, [(1, [70, 3, 0, 129], [4, 1, 5, 2])], 2 * group, 2, 64, 64, seed=6)
    t0 = [0] + np.cumsum(c.drafts).tolist()
    bad = float(what)
    path = lambda b, i: {i} | (path(b, c.parents[b][i]) if c.parents[b][i] >= 0 else set())
    sees = lambda b, j: [t0[b] + i for i in range(c.drafts[b]) if j in path(b, i)]
    c.v_new[t0[2] + 1, 0, 5] = bad                              # a drafted value
    c.k_new[t0[3], 1, 7] = float("nan")                         # a drafted key
    c.q[t0[0] + 1, group + 1, 3] = float("nan")                 # a query of the second KV head
    own = int(c.rows[0][64 + 69])                               # an own value of sequence 0 (its last key)
    c.v[own, 1, 9] = bad
    c.write()
    o, lse = c.run()
    drafted, keyed, asked, owned = sees(2, 1), sees(3, 0), [t0[0] + 1], list(range(t0[0], t0[1]))
    assert drafted and keyed
    c.check(o, lse, skip=set(drafted + keyed + asked + owned))
    # a drafted value: that dimension of the first KV head, what the formula says; all others as without it
    head = o[drafted, :group].float()
    want = bad if math.isnan(bad) or math.isinf(bad) else 0
    assert (torch.isnan(head[..., 5]) if math.isnan(want) else head[..., 5] == want).all()
    assert torch.isfinite(head[..., [x for x in range(64) if x != 5]]).all() and torch.isfinite(o[drafted, group:].float()).all()
    # a drafted key: all dimensions of the second head
    assert torch.isnan(o[keyed, group:].float()).all() and torch.isfinite(o[keyed, :group].float()).all()
    # a query: its own row alone
    assert torch.isnan(o[asked, group + 1].float()).all()
    rest = [t for t in owned if t not in asked]
    mine = o[rest, group:].float()
    dims = [9] if fmt != C.E2M1 else list(range(16))            # 4 bits: Inf and NaN take their group of 16 along
    others = [x for x in range(64) if x not in dims]
    if fmt == C.BF16 and not math.isnan(bad):
        assert (mine[..., 9] == bad).all()
    else:
        assert torch.isnan(mine[..., dims]).all()               # 8 and 4 bits hold NaN for either
    assert torch.isfinite(mine[..., others]).all() and torch.isfinite(o[rest, :group].float()).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """Pages whose bytes begin past 2^32."""
    page_bytes = {C.BF16: 2 * 128, C.E4M3: 128, C.E2M1: 64}[fmt] * 128 * 8
    c = Case(fmt, [(2, [130, 7], [2, 1])], 16, 8, 128, 128, seed=8, first_page=(1 << 32) // page_bytes + 3)
    c.check(*c.run())


def test_bad_groups_compute_nothing():
    c = Case(C.BF16, SOME, 4, 2, 64, 64, seed=10)
    n = len(c.lengths)
    for cu in ([0, 2, 6, n - 1], [1, 2, 6, n], [0, 6, 2, n], [0, 2, n + 1, n], [-1, 2, 6, n], [0, 2, 6, n + 5]):
        o, lse = c.run(want_status=1, cu_group=i32(cu))
        assert torch.isnan(o).all() and torch.isnan(lse).all(), cu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("pages", [-1, 1 << 20, -(1 << 31), (1 << 31) - 1])
def test_bad_shared_pages_share_nothing(fmt, pages):
    c = Case(fmt, SOME, 4, 2, 64, 64, seed=11)
    c.check(*c.run(want_status=1, shared_pages=i32([0, pages, 1])))


@pytest.mark.parametrize("fmt", FMTS)
def test_bad_entries_are_left_out(fmt):
    c = Case(fmt, [(3, [70, 10], [2, 3]), (0, [130], [1])], 4, 2, 64, 64, seed=12)
    table = c.table.clone()
    table[0, 1] = c.cs.pages                                    # of a shared page, in the table that is read
    table[1, 3] = -1                                            # an own page
    table[2, 1] = 1 << 30
    o, lse = c.run(want_status=1, block_table=table.cuda())
    kept = {0: [0, 2, 3, 4], 1: [0, 2], 2: [0, 2]}
    c.check(o, lse, drop=lambda b: np.isin(np.arange(c.lengths[b]) // 64, kept[b]))


def test_bad_lengths_and_offsets():
    c = Case(C.E4M3, [(1, [70, 10, 5], [2, 3, 1])], 4, 2, 64, 64, seed=13)
    # fewer tokens than the group's pages: the group's are attended to
    o, lse = c.run(want_status=1, cached=i32([c.lengths[0], 3, c.lengths[2]]))
    c.check(o, lse, drop=lambda b: np.arange(c.lengths[b]) < (64 if b == 1 else 1 << 30))
    # a length past max_cached reads as an empty cache, which lacks those pages
    o, lse = c.run(want_status=1, cached=i32([c.lengths[0], 1 << 30, c.lengths[2]]))
    c.check(o, lse, drop=lambda b: np.arange(c.lengths[b]) < (64 if b == 1 else 1 << 30))
    # offsets that do not follow one another: nothing is computed
    for cu in ([0, 2, 1, 6], [0, 2, 7, 6], [0, -1, 5, 6], [0, 2, 1 << 30, 6], [0, 2, 5, 7], [-(1 << 31), 2, 5, 6]):
        o, lse = c.run(want_status=1, cu_draft=i32(cu))
        assert torch.isnan(o).all() and torch.isnan(lse).all(), cu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [1, 16])
def test_a_sequence_with_more_drafts_than_the_shape_allows(fmt, group):
    """It reads as without drafts, and its tokens' rows stay as they were; those before and behind it are computed."""
    c = Case(fmt, [(1, [3, 70, 10], [2, 300, 3])], group, 1, 64, 64, seed=17)
    shape, a = c.args()
    shape = c.bsa.make_shared_shape(1, 3, 305, 3, max(c.lengths), group, c.stride)
    o = torch.full((305, group, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = i32([0])
    ws = torch.full((c.bsa.shared_workspace_bytes(shape, c.cs),), 0xFF, dtype=torch.uint8, device="cuda")
    c.bsa.shared_fwd(shape, c.cs, a["cu_group"], a["shared_pages"], a["cu_draft"], a["cached"], a["block_table"], a["parents"],
                     a["q"], a["k_new"], a["v_new"], c.cache, 0.125, o, None, ws, st)
    torch.cuda.synchronize()
    assert st.item() == 1 and torch.isnan(o[2:302]).all()
    c.check(o, None, only=[0, 2])


def test_a_parent_that_is_none():
    c = Case(C.BF16, [(1, [3], [4])], 4, 2, 64, 64, seed=14)
    c.parents = [[-1, 0, 1, 1]]
    bad = i32([-1, 0, 2, 1])                                    # token 2 is its own parent: a root
    o, lse = c.run(want_status=1, parents=bad)
    c.parents = [[-1, 0, -1, 1]]
    c.check(o, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_another_stream_and_two_graphs(fmt):
    """Captured on streams of their own with workspaces of their own, replayed at the same time over new inputs."""
    c = Case(fmt, [(5, [70, 3, 0], [2, 1, 3]), (2, [1, 90], [1, 1])], 8, 2, 128, 64, seed=15)
    shape, a = c.args()
    bsa, t = c.bsa, sum(c.drafts)
    nbytes = bsa.shared_workspace_bytes(shape, c.cs)
    sides = []
    for _ in range(2):
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        q = a["q"].clone()
        o = torch.empty(t, c.hq, c.d, dtype=torch.bfloat16, device="cuda")
        ws, st = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), i32([0])
        call = lambda q=q, o=o, ws=ws, st=st: bsa.shared_fwd(
            shape, c.cs, a["cu_group"], a["shared_pages"], a["cu_draft"], a["cached"], a["block_table"], a["parents"], q,
            a["k_new"], a["v_new"], c.cache, 1 / math.sqrt(c.d), o, None, ws, st)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            call()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            call()
        sides.append((s, g, q, o, st, ws))                    # (a graph works in its workspace as long as it lives)
    for i, (s, g, q, o, st, _) in enumerate(sides):
        q.copy_(a["q"] * (1.0 if i == 0 else -0.5))
        o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, g, q, o, st, _ in sides:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for s, g, q, o, st, _ in sides:
        assert int(st.item()) == 0
        want, _ = c.run(lse=False, q=q)
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


def test_captured_lengths_change():
    """One graph over a batch whose lengths, drafts and shared pages move between replays, all within the shape."""
    c = Case(C.BF16, [(3, [100, 64], [4, 3])], 8, 2, 64, 64, seed=16, extra=2)
    shape, a = c.args()
    o = torch.empty(9, 8, 64, dtype=torch.bfloat16, device="cuda")
    st, ws = i32([0]), torch.empty(c.bsa.shared_workspace_bytes(shape, c.cs), dtype=torch.uint8, device="cuda")
    call = lambda: c.bsa.shared_fwd(shape, c.cs, a["cu_group"], a["shared_pages"], a["cu_draft"], a["cached"],
                                    a["block_table"], a["parents"], a["q"], a["k_new"], a["v_new"], c.cache, 0.125, o, None,
                                    ws, st)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        call()
    for lengths, drafts, shared in (([292, 256], [4, 3], 3), ([192, 256], [1, 4], 3), ([193, 200], [0, 2], 2), ([64, 0], [3, 1], 0)):
        a["cached"].copy_(i32(lengths))
        a["cu_draft"].copy_(i32([0] + np.cumsum(drafts).tolist()))
        a["shared_pages"].copy_(i32([shared]))
        a["parents"].copy_(i32(sum([list(range(-1, n - 1)) for n in drafts], []) + [0] * (9 - sum(drafts))))
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        keep, c.drafts, c.parents = c.drafts, drafts, [list(range(-1, n - 1)) for n in drafts]
        c.check(o, None, drop=lambda b: np.arange(len(c.rows[b])) < lengths[b])
        assert torch.isnan(o[sum(drafts):]).all()
        c.drafts = keep


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("what", ["no drafts", "too many drafts", "bad groups"])
def test_steps_that_write_no_row_between_others_in_one_workspace(fmt, what):
    """Queued one behind the other: a step in which no sequence has rows, then a whole one, in the same workspace."""
    c = Case(fmt, [(70, [900, 5, 0], [3, 1, 2]), (33, [129, 640], [1, 1])], 8, 2, 128, 64, seed=18)
    shape, a = c.args()
    bsa, t = c.bsa, sum(c.drafts)
    ws = torch.full((bsa.shared_workspace_bytes(shape, c.cs),), 0xFF, dtype=torch.uint8, device="cuda")
    empty = dict(a)
    if what == "no drafts":
        empty["cu_draft"] = i32([0] * 6)
    elif what == "too many drafts":
        empty["cu_draft"] = i32([0, 4, 4, 8, 8, 8])             # of 3
    else:
        empty["cu_group"] = i32([0, 6, 5])

    def call(x, o, lse, st):
        bsa.shared_fwd(shape, c.cs, x["cu_group"], x["shared_pages"], x["cu_draft"], x["cached"], x["block_table"],
                       x["parents"], x["q"], x["k_new"], x["v_new"], c.cache, 1 / math.sqrt(c.d), o, lse, ws, st)

    def outs(n):
        return ([torch.full((t, c.hq, c.d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(n)],
                [torch.full((t, c.hq), float("nan"), device="cuda") for _ in range(n)])
    n = 20
    (o, lse), (none, no_lse), st, st_none = outs(n), outs(n), i32([0]), i32([0])
    torch.cuda.synchronize()
    for i in range(n):
        call(empty, none[i], no_lse[i], st_none)
        call(a, o[i], lse[i], st)
    torch.cuda.synchronize()
    assert st.item() == 0 and st_none.item() == (0 if what == "no drafts" else 1)
    c.check(o[0], lse[0])
    for i in range(n):
        assert torch.isnan(none[i]).all() and torch.isnan(no_lse[i]).all()
        assert torch.equal(o[i].view(torch.int16), o[0].view(torch.int16)) and torch.equal(lse[i], lse[0]), i


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups", [[(456, [70, 0, 130], [4, 3, 3])], [(150, [3, 70], [5, 4]), (140, [1], [9]), (160, [64, 0], [6, 3])]],
                         ids=["one run", "segments"])
def test_a_dozen_units_a_run_in_two_row_tiles(fmt, groups):
    """Every place of the rings of tiles, codes, records and signs is used several times, each in its turn."""
    c = Case(fmt, groups, 128, 8, 64, 64, seed=19)
    o, lse = c.run()
    c.check(o, lse)
    for _ in range(3):
        again, lse2 = c.run()
        assert torch.equal(o.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_refusals_of_the_binding():
    c = Case(C.BF16, ONE, 4, 2, 64, 64)
    for over, kind in ((dict(cu_group=i32([0])), ValueError), (dict(shared_pages=torch.zeros(1, device="cuda")), TypeError),
                       (dict(block_table=c.table.cuda()[:, :2].contiguous()), ValueError),
                       (dict(q=c.q.cuda().float()), TypeError), (dict(cached=torch.tensor(c.lengths).int()), TypeError)):
        with pytest.raises(kind):
            c.run(**over)
