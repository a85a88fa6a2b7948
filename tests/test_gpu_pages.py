"""Page tables on the GPU (fork, growth, trim, compaction) against a model on the host: integers and bytes, all exact."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu
INVALID, WORKSPACE = 1, 4


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_kv_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """The model: tables, lengths, counts, and for every page and row of it what is stored there."""

    def __init__(self, pages, page, stride):
        self.pages, self.page, self.stride = pages, page, stride
        self.refs = [0] * pages
        self.cached, self.table = [], []
        self.data = {}                                        # page -> bytes of its rows, per array

    def have(self, n):
        return -(-n // self.page)

    def fork(self, source):
        rows = [(0, []) if s < 0 else (self.cached[s], self.table[s][:self.have(self.cached[s])]) for s in source]
        old = [p for n, t in zip(self.cached, self.table) for p in t[:self.have(n)]]
        for p in old:
            self.refs[p] -= 1
        self.cached = [n for n, _ in rows]
        self.table = [list(t) + [-1] * (self.stride - len(t)) for _, t in rows]
        for _, t in rows:
            for p in t:
                self.refs[p] += 1

    def grow(self, cu, grow, rank=None):
        """None if the pool lacks pages, else (slots, copies): copies of (from, to, rows)."""
        refs, cached, table = list(self.refs), list(self.cached), [list(t) for t in self.table]
        slots, copies = [None] * cu[-1], []
        take = iter([p for p in range(self.pages) if refs[p] == 0])
        for b, n in enumerate(cached):
            g = cu[b + 1] - cu[b] if grow is None else grow[b]
            if g > 0:
                used = n % self.page
                try:
                    if used and refs[table[b][n // self.page]] > 1:
                        old, new = table[b][n // self.page], next(take)
                        refs[old] -= 1
                        refs[new] = 1
                        table[b][n // self.page] = new
                        copies.append((old, new, used))
                    for j in range(self.have(n), self.have(n + g)):
                        table[b][j] = next(take)
                        refs[table[b][j]] = 1
                except StopIteration:
                    return None
            for i in range(cu[b + 1] - cu[b]):
                r = i if rank is None else rank[cu[b] + i]
                at = n + r
                slots[cu[b] + i] = table[b][at // self.page] * self.page + at % self.page if 0 <= r < g else -1
            cached[b] = n + g
        self.refs, self.cached, self.table = refs, cached, table
        return slots, copies

    def trim(self, keep):
        for b, k in enumerate(keep):
            for j in range(self.have(k), self.have(self.cached[b])):
                self.refs[self.table[b][j]] -= 1
                self.table[b][j] = -1
            self.cached[b] = k

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        moves = list(zip([p for p in range(live, self.pages) if self.refs[p] > 0],
                         [p for p in range(live) if self.refs[p] == 0]))
        to = dict(moves)
        for src, dst in moves:
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for b, n in enumerate(self.cached):
            for j in range(self.have(n)):
                self.table[b][j] = to.get(self.table[b][j], self.table[b][j])
        return live, moves


class Gpu:
    def __init__(self, pool, fmt=C.BF16, hkv=2, d=64, seed=0):
        import block_sparse_long_kv_gb300 as bsa
        self.bsa, self.pool, self.hkv = bsa, pool, hkv
        self.cs = bsa.make_cache_shape(pool.pages, pool.page, hkv, d, fmt)
        self.cache = bsa.alloc_cache(self.cs)
        g = torch.Generator().manual_seed(seed)
        for t in self.cache.values():
            if t is not None:
                t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, dtype=torch.uint8))
        self.refs = i32(pool.refs)
        self.status = i32([0])
        self.load()

    def load(self):
        self.cached, self.table = i32(self.pool.cached or [0]), i32(self.pool.table or [[-1] * self.pool.stride])

    def bytes(self):
        """name -> [pages, hkv, bytes of a page and head] on the host"""
        return {k: t.view(torch.uint8).reshape(self.pool.pages, self.hkv, -1).cpu().numpy().copy()
                for k, t in self.cache.items() if t is not None}

    def same(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        assert self.refs.tolist() == self.pool.refs
        assert self.cached.tolist() == self.pool.cached
        got = self.table.tolist()
        for b, n in enumerate(self.pool.cached):
            assert got[b][:self.pool.have(n)] == self.pool.table[b][:self.pool.have(n)], b

    def fork(self, source):
        out = (torch.full((len(source),), -9, dtype=torch.int32, device="cuda"),
               torch.full((len(source), self.pool.stride), -9, dtype=torch.int32, device="cuda"))
        self.bsa.cache_fork(self.cs, i32(source), self.cached, self.table, self.refs, *out, self.status)
        self.cached, self.table = out

    def grow(self, cu, grow=None, rank=None, extra=0, batch_cu=None):
        slots = torch.full((cu[-1] + extra,), -9, dtype=torch.int32, device="cuda")
        ranks = None if rank is None else i32(list(rank) + [0] * extra)
        self.bsa.cache_grow(self.cs, i32(batch_cu or cu), ranks, None if grow is None else i32(grow), self.cached, self.table,
                            self.refs, self.cache, slots, None, self.status)
        return slots.tolist()

    def trim(self, keep):
        self.bsa.cache_trim(self.cs, i32(keep), self.cached, self.table, self.refs, self.status)

    def compact(self):
        live = i32([-9])
        self.bsa.cache_compact(self.cs, self.cached, self.table, self.refs, self.cache, live, None, self.status)
        return int(live.item())


def rows_of(fmt, name, page, x):
    """[hkv, rows] bytes of an array's page x [hkv, bytes], by row: codes and exponents in order, group scales after."""
    hkv = x.shape[0]
    if name in ("k", "v") or fmt == C.E4M3:
        return x.reshape(hkv, page, -1)
    return np.concatenate([x[:, :page, None], x[:, page:].reshape(hkv, page, -1)], 2)


def copied(fmt, page, before, after, copies):
    """The copies' rows hold what the old pages' did, and nothing else has changed."""
    for name, a in after.items():
        b = before[name]
        want = b.copy()
        for old, new, rows in copies:
            w, o = rows_of(fmt, name, page, want[new]).copy(), rows_of(fmt, name, page, b[old])
            w[:, :rows] = o[:, :rows]
            got = rows_of(fmt, name, page, a[new])
            assert (got == w).all(), (name, old, new)
        untouched = [p for p in range(len(a)) if p not in {n for _, n, _ in copies}]
        assert (a[untouched] == want[untouched]).all(), name


FMTS = [C.BF16, C.E4M3, C.E2M1]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [64, 128, 256])
@pytest.mark.parametrize("seed", range(4))
def test_a_life_of_a_pool(fmt, page, seed):
    """Random forks, growths, trims and compactions, one after the other, from an empty pool."""
    rng = np.random.default_rng(seed)
    pool = Pool(int(rng.integers(40, 90)), page, 12)
    pool.cached, pool.table = [0] * 3, [[-1] * 12 for _ in range(3)]
    dev = Gpu(pool, fmt, hkv=int(rng.integers(1, 4)), d=[64, 128][seed % 2], seed=seed)
    for step in range(14):
        what = ["grow", "fork", "grow", "trim", "compact"][step % 5]
        batch = len(pool.cached)
        before = dev.bytes()
        if what == "grow":
            room = [min(12 * page - n, 3 * page) for n in pool.cached]
            new = [int(rng.choice([0, 1, 5, page - 1, page, 2 * page + 3])) for _ in range(batch)]
            new = [min(x, r) for x, r in zip(new, room)]
            x = int(rng.integers(batch))
            new[x] = min(1, room[x])
            if sum(new) == 0:
                continue
            cu = [0] + np.cumsum(new).tolist()
            grow = rank = None
            if step % 2 == 0 and step:                       # some of the tokens, in another order
                grow = [int(rng.integers(0, x + 1)) for x in new]
                rank = np.concatenate([rng.permutation(x) for x in new if x]).tolist()
                rank = [r if r < g else -1 for r, g in zip(rank, np.repeat(grow, new))]
            made = pool.grow(cu, grow, rank)
            slots = dev.grow(cu, grow, rank, extra=2)
            assert slots[-2:] == [-9, -9]
            if made is None:
                dev.same(WORKSPACE)
                assert set(slots[:-2]) <= {-1}
                dev.status.zero_()
                copied(fmt, page, before, dev.bytes(), [])
                pool.fork([0, -1])                            # make room
                dev.fork([0, -1])
                dev.same()
                continue
            assert slots[:-2] == made[0]
            dev.same()
            copied(fmt, page, before, dev.bytes(), made[1])
        elif what == "fork":
            source = [int(x) for x in rng.integers(-1, batch, size=int(rng.integers(1, 7)))]
            source[0] = max(source[0], 0)
            pool.fork(source)
            dev.fork(source)
            dev.same()
            assert dev.table.tolist() == pool.table           # to the end of every row
        elif what == "trim":
            keep = [int(rng.choice([0, n // 2, max(0, n - 1), n, n - n % page])) for n in pool.cached]
            pool.trim(keep)
            dev.trim(keep)
            dev.same()
        else:
            live, moves = pool.compact()
            assert dev.compact() == live
            dev.same()
            after = dev.bytes()
            for name, a in after.items():
                want = before[name].copy()
                for src, dst in moves:
                    want[dst] = before[name][src]
                in_use = [p for p in range(pool.pages) if pool.refs[p] > 0]
                assert (a[in_use] == want[in_use]).all(), name
        assert all(r >= 0 for r in pool.refs)


def shared_rows(n, lengths, page=64, pages=40, stride=8):
    """n sequences that all begin with the pages of the longest."""
    pool = Pool(pages, page, stride)
    need = pool.have(max(lengths))
    row = list(range(3, 3 + need))
    pool.cached = list(lengths)
    pool.table = [row[:pool.have(x)] + [-1] * (stride - pool.have(x)) for x in lengths]
    for t, x in zip(pool.table, lengths):
        for p in t[:pool.have(x)]:
            pool.refs[p] += 1
    return pool


@pytest.mark.parametrize("growing", [[1, 1, 1, 1], [1, 0, 1, 0], [0, 0, 0, 1], [64, 65, 0, 1]])
@pytest.mark.parametrize("lengths", [[70, 70, 70, 70], [70, 90, 100, 127], [64, 70, 128, 65], [0, 1, 63, 64]])
def test_who_copies_a_shared_last_page(growing, lengths):
    """All but the last that holds it, whoever grows and wherever their tokens end."""
    pool = shared_rows(4, lengths)
    dev = Gpu(pool, C.E2M1)
    before = dev.bytes()
    cu = [0] + np.cumsum(growing).tolist()
    slots, copies = pool.grow(cu, None)
    assert dev.grow(cu) == slots
    dev.same()
    copied(C.E2M1, 64, before, dev.bytes(), copies)


@pytest.mark.parametrize("short", [0, 1])
def test_all_or_nobody(short):
    """A pool with just enough pages, and one with one page less."""
    pool = shared_rows(3, [70, 70, 128], pages=8 - short)
    dev = Gpu(pool, C.BF16)
    before = dev.bytes()
    cu = [0, 1, 130, 200]                                     # a copy; a copy and two pages; two pages
    made = pool.grow(cu, None)
    slots = dev.grow(cu)
    if made is None:
        dev.same(WORKSPACE)
        assert set(slots) == {-1}
        copied(C.BF16, 64, before, dev.bytes(), [])
    else:
        assert slots == made[0]
        dev.same()
    assert (made is None) == (short == 1)


@pytest.mark.parametrize("pages, batch", [(1, 1), (5000, 3), (9001, 1500)])
def test_pools_and_batches_of_several_rounds(pages, batch):
    """More pages than a planning CTA takes at a time (4096), and more sequences (1024)."""
    rng = np.random.default_rng(pages)
    pool = Pool(pages, 64, 6)
    pool.cached, pool.table = [0] * batch, [[-1] * 6 for _ in range(batch)]
    dev = Gpu(pool, C.E2M1, hkv=1)
    new = rng.integers(0, 129, size=batch).tolist() if batch > 1 else [64]
    for _ in range(2 if batch > 1 else 1):
        cu = [0] + np.cumsum(new).tolist()
        assert dev.grow(cu) == pool.grow(cu, None)[0]
        dev.same()
    if batch == 1:
        assert pool.grow([0, 1], None) is None and dev.grow([0, 1]) == [-1]
        dev.same(WORKSPACE)
        return
    source = rng.integers(0, batch, size=batch).tolist()
    pool.fork(source)
    dev.fork(source)
    dev.same()
    cu = list(range(batch + 1))
    assert dev.grow(cu) == pool.grow(cu, None)[0]
    dev.same()
    live, _ = pool.compact()
    assert dev.compact() == live
    dev.same()


def test_bad_entries_are_reported_and_left_out():
    def fresh():
        pool = shared_rows(3, [70, 90, 128])
        return pool, Gpu(pool)
    # fork: sources outside the batch are empty rows
    pool, dev = fresh()
    dev.fork([0, 3, -2, 1 << 30])
    pool.fork([0, -1, -1, -1])
    dev.same(INVALID)
    # a page that is none: not counted
    pool, dev = fresh()
    dev.table[0, 0] = 40
    pool.table[0][0] = 40
    dev.fork([0, 0, 1, 2])
    torch.cuda.synchronize()
    assert int(dev.status.item()) == INVALID and dev.refs.tolist()[:6] == [0, 0, 0, 3, 4, 0]
    # lengths that the row cannot hold
    for n in (-1, 8 * 64 + 1, -(1 << 31), (1 << 31) - 1):
        pool, dev = fresh()
        dev.cached[1] = n
        assert dev.grow([0, 1, 2, 3])[1] == -1
        assert int(dev.status.item()) == INVALID and dev.cached.tolist() == [71, n, 129]
    # growth past the row, tokens outside the total, a last page that is none: the others grow
    for over in (dict(cu=[0, 1, 500, 501]), dict(cu=[0, 1, 2, 3], batch_cu=[0, 1, 9, 3]), dict(cu=[0, 1, 2, 3], batch_cu=[0, 1, -5, 3]),
                 dict(cu=[0, 1, 2, 3], grow=[1, 2, 1]), dict(cu=[0, 1, 2, 3], grow=[1, -1, 1])):
        pool, dev = fresh()
        dev.grow(**over)
        torch.cuda.synchronize()
        assert int(dev.status.item()) == INVALID and dev.cached.tolist()[:2] == [71, 90], over
    pool, dev = fresh()
    dev.table[1, 1] = -1
    slots = dev.grow([0, 1, 2, 3])
    torch.cuda.synchronize()
    assert int(dev.status.item()) == INVALID and dev.cached.tolist() == [71, 90, 129] and slots[1] == -1
    # trim to more than there is, or less than nothing
    pool, dev = fresh()
    dev.trim([71, -1, 60])
    pool.trim([70, 90, 60])
    dev.same(INVALID)
    # counts that are too small never make a page free that a row names
    pool, dev = fresh()
    dev.refs[3] = 1
    dev.trim([0, 0, 0])
    torch.cuda.synchronize()
    assert int(dev.status.item()) == INVALID
    # compaction: an entry that names a free page, or none
    for bad in (39, 40, -1):
        pool, dev = fresh()
        dev.table[1, 0] = bad
        dev.compact()
        torch.cuda.synchronize()
        assert int(dev.status.item()) == INVALID
        assert dev.table.tolist()[0][:2] == [0, 1] and dev.table.tolist()[1][:2] == [bad, 1]


@pytest.mark.parametrize("fmt", [C.BF16, C.E4M3])
def test_offsets_past_32_bits(fmt):
    """Copies and moves of pages whose bytes begin past 2^32."""
    page_bytes = {C.BF16: 2 * 128, C.E4M3: 128}[fmt] * 128 * 8
    first = (1 << 32) // page_bytes + 5
    import block_sparse_long_kv_gb300 as bsa
    cs = bsa.make_cache_shape(first + 4, 128, 8, 128, fmt)
    cache = bsa.alloc_cache(cs)
    for t in cache.values():
        if t is not None:
            t.view(torch.uint8).view(first + 4, -1)[first:].random_(0, 256)
    refs = torch.ones(first + 4, dtype=torch.int32, device="cuda")
    refs[first] = 2
    refs[first + 1:] = 0
    cached, table = i32([100, 100]), i32([[first, -1], [first, -1]])
    st, slots, live = i32([0]), i32([-9, -9]), i32([0])
    old = {k: t.view(torch.uint8).view(first + 4, -1)[first].clone() for k, t in cache.items() if t is not None}
    bsa.cache_grow(cs, i32([0, 1, 2]), None, None, cached, table, refs, cache, slots, None, st)
    assert slots.tolist() == [(first + 1) * 128 + 100, first * 128 + 100] and st.item() == 0
    for k, x in old.items():
        new = cache[k].view(torch.uint8).view(first + 4, -1)[first + 1]
        per = new.numel() // 8 // 128
        assert torch.equal(new.view(8, 128, per)[:, :100], x.view(8, 128, per)[:, :100]), k
    kept = {k: t.view(torch.uint8).view(first + 4, -1)[first + 1].clone() for k, t in cache.items() if t is not None}
    refs[2] = 0
    bsa.cache_compact(cs, cached, table, refs, cache, live, None, st)
    assert live.item() == first + 1 and table.tolist()[0][0] == 2 and table.tolist()[1][0] == first and st.item() == 0
    for k, x in kept.items():
        assert torch.equal(cache[k].view(torch.uint8).view(first + 4, -1)[2], x), k


def test_captured_on_another_stream():
    """Fork, growth, trim and compaction in one graph, replayed over a table that goes on changing."""
    pool = shared_rows(2, [70, 100], pages=60)
    dev = Gpu(pool, C.E4M3)
    bsa, cs = dev.bsa, dev.cs
    src, cu, keep = i32([0, 0, 1]), i32([0, 3, 5, 9]), i32([72, 70, 100])
    out_c, out_t = i32([0] * 3), i32([[-1] * 8] * 3)
    slots, live = i32([0] * 9), i32([0])
    wg = torch.empty(bsa.cache_grow_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    wc = torch.empty(bsa.cache_compact_workspace_bytes(cs), dtype=torch.uint8, device="cuda")

    def step():
        bsa.cache_fork(cs, src, dev.cached, dev.table, dev.refs, out_c, out_t, dev.status)
        bsa.cache_grow(cs, cu, None, None, out_c, out_t, dev.refs, dev.cache, slots, wg, dev.status)
        bsa.cache_trim(cs, keep, out_c, out_t, dev.refs, dev.status)
        bsa.cache_compact(cs, out_c, out_t, dev.refs, dev.cache, live, wc, dev.status)
        dev.cached.copy_(out_c[1:])
        dev.table.copy_(out_t[1:])

    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    start = [t.clone() for t in (dev.cached, dev.table, dev.refs)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    for t, x in zip((dev.cached, dev.table, dev.refs), start):
        t.copy_(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        step()
    for t, x in zip((dev.cached, dev.table, dev.refs), start):
        t.copy_(x)
    torch.cuda.synchronize()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        pool.fork([0, 0, 1])
        want, _ = pool.grow([0, 3, 5, 9], None)
        assert slots.tolist() == want
        pool.trim([min(k, n) for k, n in zip([72, 70, 100], pool.cached)])
        assert live.item() == pool.compact()[0]
        assert dev.refs.tolist() == pool.refs and out_c.tolist() == pool.cached
        # the first row is dropped without being given up here: count it out on both sides
        for p in pool.table[0][:pool.have(pool.cached[0])]:
            pool.refs[p] -= 1
            dev.refs[p] -= 1
        pool.cached, pool.table = pool.cached[1:], pool.table[1:]
    assert int(dev.status.item()) == 0


LENGTHS_THAT_ARE_NONE = [-1, 8 * 64 + 1, -(1 << 31), (1 << 31) - 1]


@pytest.mark.parametrize("n", LENGTHS_THAT_ARE_NONE)
@pytest.mark.parametrize("keep", [0, 5, -1])
def test_trim_of_a_length_that_is_none(n, keep):
    """Nothing of that row changes, not even where nothing is to be kept; the others are trimmed."""
    pool = shared_rows(3, [70, 90, 128])
    dev = Gpu(pool)
    dev.cached[1] = n
    dev.trim([60, keep, 128])
    pool.trim([60, 90, 128])
    pool.cached[1] = n
    torch.cuda.synchronize()
    assert int(dev.status.item()) == INVALID
    assert dev.cached.tolist() == pool.cached and dev.refs.tolist() == pool.refs and dev.table.tolist() == pool.table


@pytest.mark.parametrize("count", [1, 0, -5])
def test_counts_too_small_for_what_is_given_up(count):
    """Page 3 is named by three rows.  A count that would go below 0 stays and is reported; one that reaches 0 early is
    that of a free page, whoever still names it."""
    pool = shared_rows(3, [70, 90, 128])
    for row in ([0], [0, 1], [0, 1, 2]):                        # rows given up, one after the other
        dev = Gpu(pool)
        dev.refs[3] = count
        for x in row:
            before = int(dev.refs[3].item())
            keep = dev.cached.tolist()
            keep[x] = 0
            dev.status.zero_()
            dev.trim(keep)
            torch.cuda.synchronize()
            assert int(dev.refs[3].item()) == (before - 1 if before > 0 else before)
            assert int(dev.status.item()) == (0 if before > 0 else INVALID)
        refs = list(pool.refs)
        refs[3], refs[4] = min(count, 0), refs[4] - len(row)
        assert dev.refs.tolist() == refs
        assert [t[:2] for t in dev.table.tolist()] == [[-1, -1] if x in row else [3, 4] for x in range(3)]
        assert dev.cached.tolist() == [0 if x in row else n for x, n in enumerate([70, 90, 128])]


@pytest.mark.parametrize("count", [0, -5])
@pytest.mark.parametrize("source", [[1, 2], [0, 0, 0, 1, 2]])
def test_fork_of_a_page_whose_count_is_too_small(count, source):
    """A page that row 0 alone names, given up or taken more often: its count stays as it is, the others follow."""
    pool = shared_rows(3, [70, 90, 128])
    pool.table[0][0] = 9
    pool.refs[9], pool.refs[3] = 1, 2
    dev = Gpu(pool)
    dev.refs[9] = count
    dev.fork(source)
    pool.fork(source)
    pool.refs[9] = count
    dev.same(INVALID)


@pytest.mark.parametrize("count", [3, 2, 1, 0, -5])
@pytest.mark.parametrize("growing", [[1, 1, 1], [0, 1, 1], [1, 0, 65], [0, 0, 1]])
def test_growth_into_a_last_page_whose_count_is_too_small(count, growing):
    """One after the other: while the count is above 1 a row gets a copy, at 1 it keeps the page, and then no row does."""
    pool = shared_rows(4, [70, 90, 100, 64])
    dev = Gpu(pool)
    dev.refs[4] = count
    want, refs, short, free = [], count, False, [0, 1, 2, 5, 6]
    for b, g in enumerate(growing):
        if g and refs < 1:
            want.append(None)
            short = True
            continue
        first = 4
        if g and refs > 1:
            refs, first = refs - 1, free.pop(0)
        elif g:
            refs = 0                                          # (kept: no one else's)
        at = [70, 90, 100][b]
        pages = [3, first] + ([free.pop(0)] if at + g > 128 else [])
        want.append([pages[x // 64] * 64 + x % 64 for x in range(at, at + g)])
    want.append([free.pop(0) * 64])                           # and a row that takes no copy
    cu = [0] + np.cumsum(growing + [1]).tolist()
    slots = dev.grow(cu)
    torch.cuda.synchronize()
    assert int(dev.status.item()) == (INVALID if short else 0)
    if count != 0:                                            # (0 says that page 4 is free)
        assert slots == [s for w, g in zip(want, growing + [1]) for s in (w if w is not None else [-1] * g)]
    assert dev.cached.tolist() == [n + (g if w is not None else 0) for n, w, g in zip([70, 90, 100, 64], want, growing + [1])]


@pytest.mark.parametrize("pages, step", [(3000, 1499), ((1 << 18) + 3000, 1 << 18)])
def test_growth_of_many_rows_two_of_them_into_one_page(pages, step):
    """More rows than a planning CTA has threads: two name the same last page, which counts once.  And pages a power of two
    apart, which nobody shares."""
    pool = Pool(pages, 64, 2)
    batch = 1500
    pool.cached = [1] * batch
    pool.table = [[p, -1] for p in range(batch)]
    for b in range(0, batch, 100):
        pool.table[b][0] = (b + step) % pages if step == 1 << 18 else b
    for t in pool.table:
        pool.refs[t[0]] = 1
    pool.table[1400][0] = 7
    dev = Gpu(pool, C.E2M1, hkv=1)
    cu = list(range(batch + 1))
    want = [t[0] * 64 + 1 for t in pool.table]
    want[1400] = -1                                           # row 7 keeps it
    assert dev.grow(cu) == want
    torch.cuda.synchronize()
    assert int(dev.status.item()) == INVALID
    assert dev.cached.tolist() == [1 if b == 1400 else 2 for b in range(batch)] and dev.refs.tolist() == pool.refs


def test_growth_whose_pages_do_not_add_up_in_32_bits():
    """2048 sequences of 2^20 new pages each: offsets that descend name the same tokens again and again."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs a table of 16 GB")
    import block_sparse_long_kv_gb300 as bsa
    batch, stride, n = 4096, 1 << 20, 1 << 26
    cs = bsa.make_cache_shape(8, 64, 1, 64, C.E4M3)
    cache = bsa.alloc_cache(cs)
    cached, refs, st = torch.zeros(batch, dtype=torch.int32, device="cuda"), i32([0] * 8), i32([0])
    table = torch.full((batch, stride), -1, dtype=torch.int32, device="cuda")
    slots = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    bsa.cache_grow(cs, i32([0, n] * (batch // 2) + [0]), None, None, cached, table, refs, cache, slots, None, st)
    torch.cuda.synchronize()
    assert st.item() == INVALID                               # (of the sequences between them, which come first)
    assert not cached.any() and not refs.any() and bool((slots < 0).all())
    assert all(bool((table[i:i + 64] == -1).all()) for i in range(0, batch, 64))


@pytest.mark.parametrize("bad", [0, 1, 2, 39])
def test_compaction_reports_an_entry_that_names_a_free_page(bad):
    """One below the pages in use among them, which gets another row's page."""
    pool = shared_rows(3, [70, 90, 128])
    dev = Gpu(pool)
    dev.table[1, 0] = bad
    assert dev.compact() == 2
    torch.cuda.synchronize()
    assert int(dev.status.item()) == INVALID
    assert [t[:2] for t in dev.table.tolist()] == [[0, 1], [bad, 1], [0, 1]]
    assert dev.refs.tolist()[:6] == [3, 3, 0, 0, 0, 0]
