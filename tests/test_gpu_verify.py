"""bsa_verify on the GPU against 64-bit arithmetic.

Every decision is a comparison of values that 64 bits and integers in units of 2^-60 hold to within 2^-50: sums of up to 2^22
terms of up to 1, each off by 2^-60 (truncation) or 2^-53 of itself (64 bits).  So a decision is the same on both sides unless
the two compared values lie within MARGIN = 2^-40 of one another, which the reference asserts of no case here.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
INVALID = 1
MARGIN = 2.0 ** -40


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_kv_gb300 import build
    build.build()


def clean(row):
    """What is negative or NaN counts as 0, what is larger as 1."""
    row = np.where(np.isnan(row), 0.0, row)
    return np.clip(row, 0.0, 1.0)


def reference(p, q, tokens, parents, u, us):
    """One sequence: rows p [n, vocab], q (or None); (path ranks, count, next, how far each decision was from a tie)."""
    n, vocab = p.shape
    rank, node, depth = [-1] * n, 0, 1
    rank[0] = 0
    apart = []
    while True:
        left, mass, step = clean(p[node]), 1.0, None
        for c in [i for i in range(1, n) if parents[i] == node]:
            x = tokens[c]
            row = np.eye(1, vocab, x)[0] if q is None else clean(q[c])
            apart.append(abs(u[c] * mass * row[x] - left[x]))
            if u[c] * mass * row[x] < left[x]:
                step = c
                break
            left = np.maximum(left - mass * row, 0.0)
            mass = left.sum()
        if step is None:
            break
        rank[step], node, depth = depth, step, depth + 1
    w = left if mass > 0 else clean(p[node])
    run = np.cumsum(w)
    if run[-1] == 0:
        return rank, depth, 0, apart
    last = int(np.nonzero(w > 0)[0][-1])
    if not us < 1.0:
        return rank, depth, last, apart
    t = max(us, 0.0) * run[-1]
    nxt = min(int(np.searchsorted(run, t, side="right")), last)
    apart += [abs(run[nxt] - t)] + ([abs(run[nxt - 1] - t)] if nxt and run[nxt - 1] > 0 and t > 0 else [])
    return rank, depth, nxt, apart


class Batch:
    def __init__(self, counts, vocab, seed, parents="tree", dtype=torch.float32, drawn=True, sharp=2.5, pad=0, fresh=0.8, extra=0):
        import block_sparse_long_kv_gb300 as bsa
        self.bsa, self.counts, self.vocab, self.dtype, self.extra = bsa, counts, vocab, dtype, extra
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        t = sum(counts)
        self.cu = [0] + np.cumsum(counts).tolist()
        self.parents = []
        for n in counts:
            self.parents += {"tree": lambda: [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)],
                             "star": lambda: [-1] + [0] * (n - 1),
                             "chain": lambda: [i - 1 for i in range(n)]}[parents]()[:n]
        self.chain = parents == "chain"
        logits = sharp * torch.randn(t, vocab, generator=g)
        guess = logits + fresh * torch.randn(t, vocab, generator=g)
        start = np.repeat(self.cu[:-1], counts)
        above = torch.tensor([int(s + max(0, x)) for s, x in zip(start, self.parents)], dtype=torch.long)
        wide = lambda x: torch.cat([x.to(dtype), torch.full((t, pad), float("nan"), dtype=dtype)], 1).cuda()[:, :vocab]
        self.p = wide(torch.softmax(logits, -1))
        rows = torch.softmax(guess, -1)[above]
        self.q = wide(rows) if drawn else None
        self.tokens = torch.multinomial(rows, 1, generator=g)[:, 0].int() if drawn else rows.argmax(-1).int()
        self.u, self.us = torch.rand(t, generator=g), torch.rand(len(counts), generator=g)

    def run(self, status=0, max_draft=None, cu=None, stream=None, parents=None, batch=None):
        t, b = sum(self.counts), len(self.counts)
        tail = [0] * self.extra
        n = t + self.extra
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
        more = lambda x: x if self.extra == 0 or x is None else torch.cat([x, x[:1].expand(self.extra, -1)])
        out = (i32([-9] * b), i32([-9] * n), i32([-9] * b))
        st = i32([0])
        shape = self.bsa.make_verify_shape(b, n, max_draft or max(self.counts), self.vocab)
        par = parents if parents is not None else self.parents
        self.bsa.verify(shape, i32(cu or self.cu), None if self.chain else i32(par + tail), i32(self.tokens.tolist() + tail),
                        more(self.p), more(self.q), torch.cat([self.u, torch.zeros(self.extra)]).cuda(), self.us.cuda(), *out, st, stream)
        torch.cuda.synchronize()
        assert int(st.item()) == status
        return [x.tolist() for x in out]

    def want(self, ties=False):
        p = self.p.double().cpu().numpy()
        q = None if self.q is None else self.q.double().cpu().numpy()
        count, rank, nxt = [], [], []
        for b, n in enumerate(self.counts):
            a, e = self.cu[b], self.cu[b + 1]
            if n == 0:
                count.append(0)
                nxt.append(-1)
                continue
            r, c, x, apart = reference(p[a:e], None if q is None else q[a:e], self.tokens[a:e].tolist(), self.parents[a:e],
                                       self.u[a:e].double().tolist(), float(self.us[b]))
            assert ties or min(apart, default=1.0) > MARGIN
            rank += r
            count.append(c)
            nxt.append(x)
        return [count, rank, nxt]

    def check(self, ties=False, **kw):
        got, want = self.run(**kw), self.want(ties)
        assert got[0] == want[0] and got[1][:len(want[1])] == want[1] and got[2] == want[2]
        assert got[1][len(want[1]):] == [-9] * self.extra
        return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("parents", ["tree", "star", "chain"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 255, 256, 257, 4096, 4099, 33001])
def test_walks(dtype, drawn, parents, vocab):
    b = Batch([1, 9, 4, 0, 6, 2, 8], vocab, seed=vocab + drawn, parents=parents, dtype=dtype, drawn=drawn, extra=3)
    b.check(ties=vocab <= 2)                                  # (few tokens: nothing left, and ties at 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 1, 3, 8])
def test_rows_at_any_stride(dtype, pad):
    """Rows that begin on any boundary, NaN behind them."""
    Batch([5, 7, 3], 5003, seed=pad, dtype=dtype, pad=pad).check()
    b = Batch([5, 7, 3], 5000, seed=pad, dtype=dtype, pad=pad)
    b.q = b.q.contiguous()                                    # p and q at different strides
    b.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_refusals(dtype):
    """A star of 40 children that are nearly all refused, over slices larger than shared memory keeps (8 CTAs x 12288), one
    that fits, and one of a single CTA."""
    for vocab in (3001, 50021, 131071):
        b = Batch([41, 12], vocab, seed=vocab, parents="star", dtype=dtype)
        b.u = 0.9 + 0.1 * b.u
        got = b.check()
        assert max(got[0]) <= 2


def test_256_drafts():
    b = Batch([256, 200, 1], 300, seed=5, parents="tree")
    b.check()
    Batch([256], 97, seed=6, parents="star", drawn=False).check(ties=True)
    Batch([256], 97, seed=7, parents="chain", fresh=0.05).check()


def test_equal_distributions_take_every_first_child():
    """q = p: u M q(x) < p(x) for every u below 1."""
    b = Batch([6, 6], 501, seed=8, parents="chain", fresh=0.0)
    got = b.check()
    assert got[0] == [6, 6] and got[1] == list(range(6)) * 2


def test_the_same_token_twice():
    """Siblings with one token: refused once, nothing of it is left of a one-hot q."""
    b = Batch([5], 64, seed=9, parents="star", drawn=False)
    b.tokens[:] = 11
    b.u[:] = 0.999
    p = b.p.clone()
    p[0] = 1 / 64
    b.p = p
    assert b.run()[1] == [0, -1, -1, -1, -1] and b.check()[2][0] != 11
    b = Batch([5], 64, seed=9, parents="star", drawn=True)
    b.tokens[:] = 11
    b.check()


@pytest.mark.parametrize("us", [0.0, -1.0, float("nan"), 1.0, 2.0, float("inf"), 0.99999994, 1e-45])
def test_ends_of_the_draw(us):
    """The first token with anything left, the last one, and neither of the zeros around them."""
    b = Batch([1], 1000, seed=10)
    b.p[:, :13] = 0
    b.p[:, 990:] = 0
    b.us[:] = us
    x = b.run()[2][0]
    first, last = 13, 989
    if us == 0.0 or us == -1.0 or us == 1e-45:
        assert x == first
    elif us != 0.99999994:
        assert x == last
    else:
        assert first <= x <= last


@pytest.mark.parametrize("us", [0.0, 0.5, 1.0])
def test_rows_of_nothing(us):
    """A target row of zeros gives token 0; nothing left after refusals falls back to p."""
    b = Batch([1, 3], 300, seed=11, parents="star")
    b.p.zero_()
    b.us[:] = us
    got = b.run()
    assert got[2] == [0, 0] and got[0] == [1, 1]
    b = Batch([2], 300, seed=12, parents="star")
    q = b.q.clone()
    q[:] = 1.0                                                # above p everywhere: nothing is left
    b.q, b.u[:] = q, 1.0
    b.us[:] = us if us < 1 else 0.75
    got = b.check()
    assert got[0] == [1]


def test_values_that_are_no_probabilities():
    """NaN, negative values and values above 1, in p and in q."""
    b = Batch([4, 3], 700, seed=13, parents="star")
    b.p[:, 5::50] = float("nan")
    b.p[:, 7::50] = -0.25
    b.p[1, 300] = 7.0
    b.q[:, 9::50] = float("nan")
    b.q[2, 11] = float("inf")
    b.q[:, 12::50] = -float("inf")
    b.check()


@pytest.mark.parametrize("value", [float("nan"), -0.5, 3.0, float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["p", "q", "sibling"])
def test_a_drafted_token_without_a_probability(value, where):
    """At the drafted ids themselves: 0 for NaN and below, 1 above."""
    for seed in range(6):
        b = Batch([4, 5], 60, seed=40 + seed, parents="star")
        x = int(b.tokens[2])
        b.tokens[3] = x
        if where == "p":
            b.p[0, x] = value
        elif where == "q":
            b.q[2, x] = value
        else:
            b.q[1, x] = value                                 # of the child tried before
            b.u[1] = 1.0
        b.check(ties=True)


def test_subnormal_and_tiny_probabilities():
    b = Batch([3, 3], 400, seed=14, parents="star")
    b.p[:, ::3] = 1e-42
    b.p[:, 1::3] = 2.0 ** -59
    b.check()
    b.p[:, :] = 1e-30                                         # below every unit: the row counts as nothing
    got = b.run()
    assert got[2] == [0, 0]


def test_u_of_zero_and_one():
    """u = 0 takes a child if anything of its token is left; u = 1 only where q < what is left."""
    b = Batch([6, 6], 333, seed=15)
    b.u[:6], b.u[6:] = 0.0, 1.0
    got = b.check()
    assert got[0][0] > 1


def test_other_roots_and_bad_ids():
    b = Batch([5, 4], 100, seed=16, parents="chain")
    b.chain = False
    par = list(b.parents)
    b.u[:] = 0.0
    par[2] = -1                                               # another root: neither it nor those behind it are reached
    b.parents = par
    got = b.check()
    assert got[1][2] == -1 and got[0][0] == 2
    for bad in (2, 3, 100, -2, (1 << 31) - 1):                # no parent of token 2
        wrong = list(par)
        wrong[2] = bad
        assert b.run(status=INVALID, parents=wrong) == got
    for bad in (100, -1, 1 << 30, -(1 << 31)):                # no token
        b.parents = list(range(-1, 4)) + list(range(-1, 3))
        keep = int(b.tokens[2])
        b.tokens[2] = bad
        again = b.run(status=INVALID)
        b.tokens[2] = keep
        assert again[0] == [2, got[0][1]] and again[1][:5] == [0, 1, -1, -1, -1]
    b.parents = list(range(-1, 4)) + list(range(-1, 3))
    want = b.check()
    b.tokens[0] = -5                                          # of the first token nothing is asked
    assert b.run() == want


@pytest.mark.parametrize("cu", [[0, 5, 3], [0, 6, 9], [-1, 5, 9], [0, 5, 10], [0, 1 << 30, 9]])
def test_bad_offsets_read_as_no_drafts(cu):
    b = Batch([5, 4], 100, seed=17)
    got = b.run(status=INVALID, cu=cu, max_draft=5)
    assert 0 in got[0] and got[2][got[0].index(0)] == -1


def test_more_sequences_than_fit_at_once():
    b = Batch([1 + i % 3 for i in range(500)], 9000, seed=18, dtype=torch.bfloat16)
    b.check()


@pytest.mark.parametrize("vocab", [7, 50021])
def test_the_same_again_on_streams_and_captured(vocab):
    """Two streams at once and one graph whose inputs change: the same integers."""
    one, two = (Batch([5, 9, 1, 12], vocab, seed=s, parents="tree") for s in (19, 20))
    want = [one.check(ties=vocab < 10), two.check(ties=vocab < 10)]
    bsa, i32 = one.bsa, lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    sides = []
    for x in (one, two):
        t = sum(x.counts)
        args = [i32(x.cu), i32(x.parents), i32(x.tokens), x.p, x.q, x.u.cuda(), x.us.cuda()]
        out = [i32([-9] * 4), i32([-9] * t), i32([-9] * 4)]
        sides.append((bsa.make_verify_shape(4, t, 12, vocab), args, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for shape, args, out, s in sides:
            bsa.verify(shape, *args, *out, None, s)
    torch.cuda.synchronize()
    assert [[x.tolist() for x in side[2]] for side in sides] == want
    shape, args, out, s = sides[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bsa.verify(shape, *args, *out)
    for a, x in zip(args[1:], sides[1][1][1:]):
        a.copy_(x)
    for x in out:
        x.fill_(-9)
    g.replay()
    torch.cuda.synchronize()
    assert [x.tolist() for x in out] == want[1]


def test_the_token_is_distributed_as_p():
    """65535 sequences of one draft of three siblings over 6 tokens: whatever q is, the first new token (drafted and taken, or
    drawn behind) is of p.  A count of n draws deviates by less than 6 sqrt(n p (1 - p)) but for one case in 10^8."""
    import block_sparse_long_kv_gb300 as bsa
    b, v = 65535, 6
    g = torch.Generator().manual_seed(21)
    p = torch.tensor([0.4, 0.05, 0.25, 0.0, 0.2, 0.1])
    q = torch.tensor([0.1, 0.3, 0.05, 0.25, 0.1, 0.2])
    drawn = torch.multinomial(q, 3 * b, replacement=True, generator=g).view(b, 3)
    tokens = torch.cat([torch.zeros(b, 1, dtype=torch.long), drawn], 1).int().reshape(-1).cuda()
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    shape = bsa.make_verify_shape(b, 4 * b, 4, v)
    count, rank, nxt = i32([0] * b), i32([0] * 4 * b), i32([0] * b)
    bsa.verify(shape, i32(torch.arange(b + 1) * 4), i32([-1, 0, 0, 0]).repeat(b), tokens, p.cuda().repeat(4 * b, 1),
               q.cuda().repeat(4 * b, 1), torch.rand(4 * b, generator=g).cuda(), torch.rand(b, generator=g).cuda(), count, rank, nxt)
    took = (rank.view(b, 4) == 1)
    first = torch.where(took.any(1), (tokens.view(b, 4) * took).sum(1), nxt).cpu()
    n = torch.bincount(first, minlength=v).double()
    p = p.double()
    assert (abs(n - b * p) <= 6 * torch.sqrt(b * p * (1 - p))).all(), n
    assert int(took.any(1).sum()) > b // 2


def test_refusals_of_the_binding():
    b = Batch([3], 50, seed=22)
    keep = b.p
    for p, kind in ((b.p.double(), TypeError), (b.p[:, :49], ValueError), (b.p.t().contiguous().t(), ValueError), (b.p.cpu(), TypeError)):
        b.p = p
        with pytest.raises(kind):
            b.run()
    b.p = keep
    b.q = b.q.to(torch.bfloat16)                              # another type than p's
    with pytest.raises(TypeError):
        b.run()
