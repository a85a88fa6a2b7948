"""Several continuations of one prompt, decoded with drafted tokens from start to end: fork, attention over the shared pages,
verification, growth, write, trim and compaction on the device, each step checked against what lists on the host hold."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_kv_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Decoder:
    """What a server keeps for a batch of `batch` rows, each drafting up to `most` tokens a step; a step's kernels run on fixed
    buffers, so that they can be captured."""

    def __init__(self, fmt, batch, most, hq, hkv, d, page, vocab, pages, stride, seed):
        import block_sparse_long_kv_gb300 as bsa
        self.bsa, self.fmt, self.batch, self.most, self.hq, self.hkv, self.d, self.page = bsa, fmt, batch, most, hq, hkv, d, page
        self.g = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.cs = bsa.make_cache_shape(pages, page, hkv, d, fmt)
        self.cache = bsa.alloc_cache(self.cs)
        self.refs, self.status, self.live = i32([0] * pages), i32([0]), i32([0])
        self.cached, self.table = i32([0]), i32([[-1] * stride])
        self.pages, self.stride, self.vocab = pages, stride, vocab
        t = batch * most
        zero = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
        self.q, self.k_new, self.v_new, self.o = zero(t, hq, d), zero(t, hkv, d), zero(t, hkv, d), zero(t, hq, d)
        self.head = (torch.randn(hq * d, vocab, generator=self.g) * 2 / math.sqrt(hq * d)).cuda()
        self.cu_draft, self.parents, self.tokens, self.slots = i32([0] * (batch + 1)), i32([0] * t), i32([0] * t), i32([0] * t)
        self.cu_group, self.shared_pages = i32([0, batch]), i32([0])
        self.qp = torch.zeros(t, vocab, device="cuda")
        self.p = torch.zeros(t, vocab, device="cuda")
        self.u, self.us = torch.zeros(t, device="cuda"), torch.zeros(batch, device="cuda")
        self.count, self.rank, self.next = i32([0] * batch), i32([0] * t), i32([0] * batch)
        self.shape = bsa.make_shared_shape(1, batch, t, most, stride * page, hq, stride)
        self.vshape = bsa.make_verify_shape(batch, t, most, vocab)
        byte = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
        self.ws = byte(bsa.shared_workspace_bytes(self.shape, self.cs))
        self.wg = byte(bsa.cache_grow_workspace_bytes(batch))
        self.wc = byte(bsa.cache_compact_workspace_bytes(self.cs))
        self.host = [[]]                                       # a list of (k, v) of every row

    def bf(self, *s):
        return torch.randn(*s, generator=self.g).to(torch.bfloat16)

    def prompt(self, n):
        k, v = self.bf(n, self.hkv, self.d), self.bf(n, self.hkv, self.d)
        slots = i32([-1] * n)
        self.bsa.cache_grow(self.cs, i32([0, n]), None, None, self.cached, self.table, self.refs, self.cache, slots, None,
                            self.status)
        self.bsa.cache_write(self.cs, k.cuda(), v.cuda(), slots, self.cache)
        self.host = [[(k[i], v[i]) for i in range(n)]]
        self.shared_pages.fill_(n // self.page)
        self.prefix = n

    def fork(self, source):
        c, t = i32([0] * self.batch), i32([[-1] * self.stride] * self.batch)
        self.bsa.cache_fork(self.cs, i32(source), self.cached, self.table, self.refs, c, t, self.status)
        if self.cached.numel() == self.batch:                  # (the buffers that a graph knows)
            self.cached.copy_(c)
            self.table.copy_(t)
        else:
            self.cached, self.table = c, t
        self.host = [list(self.host[s]) if s >= 0 else [] for s in source]

    def step(self):
        b = self.bsa
        b.shared_fwd(self.shape, self.cs, self.cu_group, self.shared_pages, self.cu_draft, self.cached, self.table,
                     self.parents, self.q, self.k_new, self.v_new, self.cache, 1 / math.sqrt(self.d), self.o, None, self.ws,
                     self.status)
        torch.softmax(self.o.flatten(1).float() @ self.head, -1, out=self.p)
        b.verify(self.vshape, self.cu_draft, self.parents, self.tokens, self.p, self.qp, self.u, self.us, self.count, self.rank,
                 self.next, self.status)
        self.slots.fill_(-1)
        b.cache_grow(self.cs, self.cu_draft, self.rank, self.count, self.cached, self.table, self.refs, self.cache, self.slots,
                     self.wg, self.status)
        b.cache_write(self.cs, self.k_new, self.v_new, self.slots, self.cache)

    def draft(self):
        """New inputs of a step."""
        n = [int(self.rng.integers(1, self.most + 1)) if self.host[b] else 0 for b in range(self.batch)]
        n[0] = self.most
        self.n, t = n, sum(n)
        self.cu_draft.copy_(i32([0] + np.cumsum(n).tolist()))
        self.up = [[-1] + [int(self.rng.integers(max(0, i - 2), i)) for i in range(1, x)] for x in n]
        self.up = [x[:m] for x, m in zip(self.up, n)]
        pad = self.batch * self.most - t
        self.parents.copy_(i32(sum(self.up, []) + [0] * pad))
        for x in (self.q, self.k_new, self.v_new):
            x.copy_(self.bf(*x.shape))
        rows = torch.softmax(torch.randn(t + pad, self.vocab, generator=self.g), -1)
        self.qp.copy_(rows)
        self.tokens.copy_(torch.multinomial(rows, 1, generator=self.g)[:, 0])
        self.u.copy_(torch.rand(self.u.shape, generator=self.g))
        self.us.copy_(torch.rand(self.us.shape, generator=self.g))
        self.o.zero_()

    def check(self):
        """The step against float64: attention within its limits (as stated for bsa_shared_fwd), the walk on the same
        probabilities, and the lists follow."""
        from test_gpu_verify import MARGIN, reference
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        got = self.o.double().cpu().numpy()
        q, kn, vn = (x.double().cpu().numpy() for x in (self.q, self.k_new, self.v_new))
        p, qp, tokens = self.p.double().cpu().numpy(), self.qp.double().cpu().numpy(), self.tokens.tolist()
        u, us = self.u.double().tolist(), self.us.double().tolist()
        count, rank, nxt = self.count.tolist(), self.rank.tolist(), self.next.tolist()
        grp, scale, t0 = self.hq // self.hkv, 1 / math.sqrt(self.d), 0
        vmax = max(float(np.abs(vn).max()), max(float(v.abs().max()) for row in self.host for _, v in row))
        for b, t in enumerate(self.n):
            row = self.host[b]
            if t == 0:
                assert count[b] == 0 and nxt[b] == -1
                continue
            k = C.held(torch.stack([x for x, _ in row]).double().numpy(), self.fmt)
            v = C.held(torch.stack([x for _, x in row]).double().numpy(), self.fmt)
            for g in range(self.hkv):
                hs = slice(g * grp, (g + 1) * grp)
                want, _, a, reach = C.tree_attention(q[t0:t0 + t, hs], kn[t0:t0 + t, g], vn[t0:t0 + t, g], k[:, g], v[:, g],
                                                     self.up[b], scale)
                delta = 2 * (self.d + 8) * 2.0 ** -24 * reach + 2.0 ** -20
                tol = (2.0 ** -8 + 4 * delta[..., None] + 2.0 ** -18) * a + 2.0 ** -8 * np.abs(want)
                if self.fmt != C.BF16:
                    tol = tol + (len(row) + t) * 2.0 ** -35 * vmax
                assert (np.abs(got[t0:t0 + t, hs] - want) <= tol).all(), (b, g)
            r, c, x, apart = reference(p[t0:t0 + t], qp[t0:t0 + t], tokens[t0:t0 + t], self.up[b], u[t0:t0 + t], us[b])
            assert min(apart) > MARGIN
            assert rank[t0:t0 + t] == r and count[b] == c and nxt[b] == x
            for place in range(c):
                i = t0 + r.index(place)
                row.append((self.k_new[i].cpu(), self.v_new[i].cpu()))
            t0 += t
        assert self.cached.tolist() == [len(r) for r in self.host]
        self.counted()

    def counted(self):
        """refs is what the tables say."""
        want = [0] * self.pages
        for n, row in zip(self.cached.tolist(), self.table.tolist()):
            for p in row[:-(-n // self.page)]:
                want[p] += 1
        assert self.refs.tolist() == want

    def trim(self, keep):
        self.bsa.cache_trim(self.cs, i32(keep), self.cached, self.table, self.refs, self.status)
        self.host = [r[:k] for r, k in zip(self.host, keep)]

    def compact(self):
        self.bsa.cache_compact(self.cs, self.cached, self.table, self.refs, self.cache, self.live, self.wc, self.status)
        torch.cuda.synchronize()
        refs = self.refs.tolist()
        assert self.live.item() == sum(r > 0 for r in refs) and all(r > 0 for r in refs[:self.live.item()])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fmt", [C.BF16, C.E4M3, C.E2M1])
@pytest.mark.parametrize("n, hq, hkv, d, page", [(333, 8, 2, 64, 64), (257, 16, 1, 128, 128)])
def test_continuations_of_a_prompt(fmt, captured, n, hq, hkv, d, page):
    x = Decoder(fmt, 5, 6, hq, hkv, d, page, vocab=101, pages=40, stride=10, seed=n)
    x.prompt(n)
    x.fork([0] * 5)
    step, s = x.step, None
    if captured:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        x.draft()
        kept = [t.clone() for t in (x.cached, x.table, x.refs)] + [t.clone() for t in x.cache.values() if t is not None]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            x.step()
        torch.cuda.synchronize()
        for t, k in zip([x.cached, x.table, x.refs] + [t for t in x.cache.values() if t is not None], kept):
            t.copy_(k)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            x.step()
        step = g.replay
    for i in range(8):
        x.draft()
        torch.cuda.synchronize()
        step()
        x.check()
        if i == 2:                                             # one answer is taken back, one ends
            x.trim([x.prefix + 1, 0] + [len(r) for r in x.host[2:]])
            x.compact()
        if i == 4:                                             # beams: the best go on, one of them thrice
            x.fork([2, 2, 0, 2, 4])
        if i == 5:
            x.compact()
        x.counted()
