"""bsa_tree_fwd in all three of its forms (at most 16 query rows per KV head, up to 128, more) where one of them
alone could go wrong: maxima that grow from unit to unit, rows whose exponents lie far apart, captured steps,
concurrent calls, and batches whose plan leaves no room for two row tiles.

Tolerances as in test_gpu_tree, before the first run.  One term more where cached rows lie far apart: with more
than 16 rows over an 8- or 4-bit cache a key of a unit of 128 becomes f16 against the unit's largest row.  E4M3:
the largest row has a value above 224 units of its exponent, a key is off by half of f16's smallest step, 2^-25, in
units 2^-6 of that exponent: 2^-31 / 224 < 2^-38 of the largest |k|.  E2M1: group scale and product are each off by
half a step, the former times at most 6, in units 2^-4, against a value above 1344 units:
7 x 2^-25 x 2^-4 / 1344 < 2^-36.  So a logit moves by at most scale sum |q| 2^-36 kmax.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from test_gpu_tree import FMTS, Case

pytestmark = pytest.mark.gpu
FORMS = [("few", 2), ("one tile", 16), ("two tiles", 20)]       # drafts with G = 8: 16, 128 and 160 rows


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_kv_gb300 import build
    build.build()


def rewrite(c):
    """The case's cached rows, written again."""
    slots = []
    for b, n in enumerate(c.lengths):
        i = np.arange(n)
        slots.append(c.table[b].numpy()[i // c.page] * c.page + i % c.page)
    slots = torch.from_numpy(np.concatenate(slots).astype(np.int32)).cuda()
    c.bsa.cache_write(c.cs, c.k.cuda(), c.v.cuda(), slots, c.cache)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("form, drafts", FORMS)
@pytest.mark.parametrize("up", [True, False])
def test_maxima_that_grow_from_unit_to_unit(fmt, form, drafts, up):
    """Logits rise along the cache by more per unit than the softmax reference may lag (2^8, or 2^4 over an 8- or
    4-bit cache), and the values fall by as much, so that every unit counts in O and each rescale shows.  Falling
    logits leave the reference alone.  Enough tiles that a CTA walks whole ones and crosses into others."""
    batch, n, d, hkv = 40, 512, 64, 4
    c = Case(fmt, [n] * batch, [drafts] * batch, 8 * hkv, hkv, d, 64, seed=drafts)
    rise = 20.0 if fmt == C.BF16 else 5.0                       # log2 units per 128 keys
    g = torch.Generator().manual_seed(7)
    sign = torch.where(torch.rand(hkv, d, generator=g) < 0.5, -1.0, 1.0)
    c.q = (sign.repeat_interleave(8, 0) * (1 + 0.05 * torch.randn(*c.q.shape, generator=g).abs())).to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.float64).repeat(batch) / 128
    if not up:
        pos = 4 - pos
    per = math.sqrt(d) / (d * math.log2(math.e))                # of the key along sign, for one log2 unit
    size = (rise * per * pos)[:, None, None]
    c.k = (sign * size + 0.02 * torch.randn(*c.k.shape, generator=g)).to(torch.bfloat16)
    c.v = (c.v.double() * 2.0 ** (-rise * (pos - pos.max()))[:, None, None]).to(torch.bfloat16)
    c.v_new = (c.v_new.float() * 0.25).to(torch.bfloat16)
    c.k_new = (sign * (size.max() if up else size[n - 1, 0, 0]) + 0.02 * torch.randn(*c.k_new.shape, generator=g)).to(torch.bfloat16)
    rewrite(c)
    # the held logits do move as said: the largest of each unit of 128 keys of sequence 0
    k = C.held(c.k[:n].double().numpy(), fmt)
    s = np.einsum("thgd,nhd->thgn", c.q[:drafts].double().numpy().reshape(drafts, hkv, 8, d), k) / math.sqrt(d) * math.log2(math.e)
    top = s.reshape(drafts, hkv, 8, 4, 128).max(-1)
    step = np.diff(top, axis=-1) * (1 if up else -1)
    assert step.min() > (8 if fmt == C.BF16 else 4), step.min()
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [C.E4M3, C.E2M1])
@pytest.mark.parametrize("drafts", [4, 20, 70])
def test_row_exponents_apart(fmt, drafts):
    """Row exponents that differ by up to 2^13 between the keys of one softmax, and all values in one row."""
    c = Case(fmt, [900], [drafts], 8, 2, 128, 64, spread=4, seed=5)
    c.check(*c.run())
    c.v[:, :, :] = 0
    c.v[-1] = 3.0e4
    rewrite(c)
    c.check(*c.run())
    c.v[-1] = 0
    c.v[0] = 3.0e4
    rewrite(c)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [C.E4M3, C.E2M1])
@pytest.mark.parametrize("drafts", [4, 20, 70])
def test_rows_past_f16_apart_keep_the_stated_limits(fmt, drafts):
    """Keys and values from 1 down to 10^-12 side by side: what lies 2^20 and more below the largest loses bits or
    becomes 0, never more than the bound."""
    c = Case(fmt, [900], [drafts], 8, 2, 128, 64, spread=12, seed=9)
    c.v_new = (c.v_new.float() * 1e-6).to(torch.bfloat16)
    o, lse = c.run()
    hk, hv = C.held(c.k.double().numpy(), fmt), C.held(c.v.double().numpy(), fmt)
    scale = 1 / math.sqrt(128)
    for g in range(2):
        hs = slice(4 * g, 4 * g + 4)
        want, wl, a, reach = C.tree_attention(c.q[:, hs].double().numpy(), c.k_new[:, g].double().numpy(),
                                              c.v_new[:, g].double().numpy(), hk[:, g], hv[:, g], c.parents[0], scale)
        kmax = max(np.abs(hk[:, g]).max(), c.k_new[:, g].abs().max().item())
        vmax = max(np.abs(hv[:, g]).max(), c.v_new[:, g].abs().max().item())
        delta = 2 * (128 + 8) * 2.0 ** -24 * reach + 2.0 ** -20
        delta = delta + scale * c.q[:, hs].double().abs().sum(-1).numpy() * 2.0 ** -36 * kmax
        tol = (2.0 ** -8 + 4 * delta[..., None] + 2.0 ** -18) * a + 2.0 ** -8 * np.abs(want) + (900 + drafts) * 2.0 ** -35 * vmax
        assert (np.abs(o[:, hs].double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse[:, hs].double().cpu().numpy() - wl) <= 2 * delta + 2.0 ** -20 * (1 + np.abs(wl))).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("drafts", [4, 20, 70])
def test_large_logits_in_every_form(fmt, drafts):
    c = Case(fmt, [400], [drafts], 8, 2, 64, 64, seed=6)
    c.q = (c.q.float() * 30).to(torch.bfloat16)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("drafts", [[3, 4, 1], [20, 17, 2], [70, 33, 1]])
def test_the_same_bits_again(fmt, drafts):
    c = Case(fmt, [5000, 300, 1], drafts, 8, 2, 128, 128, keep=0.5)
    o, lse = c.run()
    o2, lse2 = c.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, _ = c.run(lse=False)
    assert torch.equal(o, o3)
    c.check(o, lse)


@pytest.mark.parametrize("drafts", [2, 20, 70])
def test_two_streams(drafts):
    a, b = Case(C.E4M3, [5000], [drafts], 16, 2, 128, 128, seed=1), Case(C.BF16, [4000], [drafts], 16, 2, 128, 128, seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    want = a.run(), b.run()
    for _ in range(3):
        with torch.cuda.stream(s1):
            oa = a.run(stream=s1)
        with torch.cuda.stream(s2):
            ob = b.run(stream=s2)
    for got, w in ((oa, want[0]), (ob, want[1])):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    a.check(*oa)
    b.check(*ob)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("drafts", [[4, 2], [70, 33]])
def test_captured_steps(fmt, drafts):
    """A captured step follows its inputs, and two graphs share a workspace."""
    cases = [Case(fmt, [900, 300], drafts, 8, 2, 128, 64, seed=s) for s in (1, 2)]
    bsa, t = cases[0].bsa, sum(drafts)
    want = [c.run() for c in cases]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ts, cs = bsa.make_tree_shape(2, t, max(drafts), 1000, 8, 17), cases[0].cs
    ws = torch.empty(bsa.tree_workspace_bytes(ts, cs), dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):
        buf = dict(cu=dev([0, drafts[0], t]), cached=dev([900, 300]), table=torch.zeros(2, 17, dtype=torch.int32, device="cuda"),
                   par=dev([0] * t), q=torch.zeros_like(cases[0].q).cuda(), k=torch.zeros_like(cases[0].k_new).cuda(),
                   v=torch.zeros_like(cases[0].v_new).cuda(), cache={n: None if x is None else x.clone() for n, x in cases[0].cache.items()},
                   o=torch.zeros(t, 8, 128, dtype=torch.bfloat16, device="cuda"), lse=torch.zeros(t, 8, device="cuda"), st=dev([0]))
        call = lambda: bsa.tree_fwd(ts, cs, buf["cu"], buf["cached"], buf["table"], buf["par"], buf["q"], buf["k"], buf["v"],
                                    buf["cache"], None, None, 1 / math.sqrt(128), buf["o"], buf["lse"], ws, buf["st"])
        call()
        torch.cuda.synchronize()
        buf["st"].zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, buf))
    for turn in range(3):
        for i, (graph, buf) in enumerate(graphs):
            x = cases[(i + turn) % 2]
            buf["table"][:, :x.stride] = x.table.cuda()
            buf["par"].copy_(dev(sum(x.parents, [])))
            for name, src in (("q", x.q), ("k", x.k_new), ("v", x.v_new)):
                buf[name].copy_(src)
            for n, src in x.cache.items():
                if src is not None:
                    buf["cache"][n].copy_(src)
            graph.replay()
        torch.cuda.synchronize()
        for i, (graph, buf) in enumerate(graphs):
            wo, wl = want[(i + turn) % 2]
            assert int(buf["st"].item()) == 0
            # the table is wider than the case's own, the plan and so the bits the same
            assert torch.equal(buf["o"], wo) and torch.equal(buf["lse"], wl)
    for c, w in zip(cases, want):
        c.check(*w)


@pytest.mark.parametrize("fmt", FMTS)
def test_more_groups_than_two_tiles_leave_room_for(fmt):
    """Over 128 rows in so many sequences that the plan does not fit beside two row tiles of d = 128."""
    batch, hkv, drafts = 1000, 4, 33
    c = Case(fmt, [(7 * b) % 40 if b % 9 else 0 for b in range(batch)], [max(0, drafts - (b % 4) * 11) for b in range(batch)],
             4 * hkv, hkv, 128, 64, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [C.BF16, C.E4M3])
@pytest.mark.parametrize("drafts", [3, 20, 40])
def test_a_negative_list_entry_is_reported(fmt, drafts):
    """Entries past the sequence's last page are left out without a word (a selection made with the new token may
    name the page that it will begin); a negative one is an error, reported, and its page left out."""
    c = Case(fmt, [300], [drafts], 8, 2, 128, 64)
    bsa = c.bsa
    ts = bsa.make_tree_shape(1, drafts, drafts, 300, 8, c.stride)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def run(row, cnt):
        idx = torch.full((1, 2, c.stride), 1 << 20, dtype=torch.int32)
        idx[:, :, :len(row)] = torch.tensor(row, dtype=torch.int32)
        o, lse = torch.zeros(drafts, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(drafts, 8, device="cuda")
        st = dev([0])
        bsa.tree_fwd(ts, c.cs, dev([0, drafts]), dev([300]), c.table.cuda(), dev(c.parents[0]), c.q.cuda(), c.k_new.cuda(),
                     c.v_new.cuda(), c.cache, idx.cuda(), dev([[cnt, cnt]]), 1 / math.sqrt(128), o, lse, dev_status=st)
        torch.cuda.synchronize()
        return o, lse, int(st.item())

    c.lists = [[[0, 3, 4], [0, 3, 4]]]                          # five pages in all
    o, lse, code = run([0, 3, 4], 3)
    assert code == 0
    c.check(o, lse)
    o, lse, code = run([0, 3, 4, 5], 4)
    assert code == 0
    c.check(o, lse)
    c.lists = [[list(range(5)), list(range(5))]]
    o, lse, code = run([0, 1, 2, 3, 4, 5], 6)                   # one entry more than the sequence has pages
    assert code == 0
    c.check(o, lse)
    for bad in (-1, -(1 << 31)):
        c.lists = [[[0, 3], [0, 3]]]
        o, lse, code = run([bad, 0, 3], 3)
        assert code == 1
        c.check(o, lse)
    o, lse, code = run([0, 3], -2)                              # a negative count is an empty list
    assert code == 0
    c.lists = [[[], []]]
    c.check(o, lse)
