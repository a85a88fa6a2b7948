"""bsa_cache_write and bsa_cache_read on the GPU: codes, scales and values equal the reference's bit for
bit (the row scales are powers of two and every rounding is of an exactly representable quotient or tie)."""
import numpy as np
import pytest
import torch

import synth
from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu
FMTS = [C.BF16, C.E4M3, C.E2M1]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_kv_gb300 import build
    build.build()


def rows(seed, *shape):
    """bf16 rows of mixed size: normal values times a power of ten for each (token, head)."""
    g = np.random.default_rng(seed)
    x = g.normal(size=shape) * 10.0 ** g.integers(-3, 3, size=shape[:-1] + (1,))
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def reference_write(cs, cache, name, x, slots):
    """The cache's bytes after the write, on the CPU."""
    codes, sc = cache[name].clone(), None if cache[name + "_scale"] is None else cache[name + "_scale"].clone()
    c, e, g = C.quantise(x.double().numpy(), cs.format)
    for t, s in enumerate(slots):
        if 0 <= s < cs.pages * cs.page:
            p, r = divmod(s, cs.page)
            codes[p, :, r] = torch.from_numpy(np.ascontiguousarray(c[t]))
            if e is not None:
                sc[p, :, r] = torch.from_numpy(e[t])
            if g is not None:
                per = cs.head_dim // 16
                sc[p, :, cs.page + r * per:cs.page + (r + 1) * per] = torch.from_numpy(g[t])
    return codes, sc


def garbage_cache(bsa, cs):
    cache = bsa.alloc_cache(cs)
    for t in cache.values():
        if t is not None:
            t.fill_(0xA7)
    return cache


def to_cpu(cache):
    return {n: None if t is None else t.cpu() for n, t in cache.items()}


def check_write(fmt, tokens, hkv, d, page, pages, slots, seed=0, fused=False, x=None):
    import block_sparse_long_kv_gb300 as bsa
    cs = bsa.make_cache_shape(pages, page, hkv, d, fmt)
    cache = garbage_cache(bsa, cs)
    before = to_cpu(cache)
    if x is None:
        x = rows(seed, tokens, hkv, d), rows(seed + 1, tokens, hkv, d)
    if fused:
        both = torch.cat([x[0].flatten(1), x[1].flatten(1)], 1).cuda()
        k, v = both[:, :hkv * d].view(tokens, hkv, d), both[:, hkv * d:].view(tokens, hkv, d)
    else:
        k, v = x[0].cuda(), x[1].cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.cache_write(cs, k, v, torch.tensor(slots, dtype=torch.int32, device="cuda"), cache, st)
    torch.cuda.synchronize()
    after = to_cpu(cache)
    for name, y in (("k", x[0]), ("v", x[1])):
        codes, sc = reference_write(cs, before, name, y, slots)
        np.testing.assert_array_equal(after[name].numpy(), codes.numpy())
        if sc is not None:
            np.testing.assert_array_equal(after[name + "_scale"].numpy(), sc.numpy())
    return int(st.item())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens, hkv, page, pages, fused", [(1, 4, 128, 2, False), (19, 3, 64, 3, True), (130, 1, 256, 1, False),
                                                              (2433, 2, 64, 40, True)])
def test_write_bytes(fmt, d, tokens, hkv, page, pages, fused):
    slots = np.random.default_rng(tokens).permutation(pages * page)[:tokens].tolist()
    assert check_write(fmt, tokens, hkv, d, page, pages, slots, fused=fused) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_left_out_and_bad_slots(fmt):
    slots = [5, -1, 64, -7, 127, 0]
    assert check_write(fmt, 6, 2, 64, 64, 2, slots) == 0
    slots[2] = 128                                             # one past the cache
    assert check_write(fmt, 6, 2, 64, 64, 2, slots) == 1
    slots[2] = (1 << 31) - 1
    assert check_write(fmt, 6, 2, 64, 64, 2, slots) == 1


@pytest.mark.parametrize("fmt", [C.E4M3, C.E2M1])
@pytest.mark.parametrize("d", [64, 128])
def test_every_kind_of_value(fmt, d):
    """Zero rows, one-hot rows, rows at and next to the scale's borders, ties of the codes, signed zeros, the
    smallest and largest bf16 values."""
    n = 600
    g = np.random.default_rng(11)
    x = np.zeros((n, 1, d))
    for i in range(n):
        kind = i % 6
        if kind == 0:
            x[i, 0, g.integers(d)] = g.choice([-1, 1]) * 2.0 ** int(g.integers(-126, 127))
        elif kind == 1:                                        # ties of e2m1 and e4m3 under a power of two
            x[i, 0] = g.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 0, -0.0, 17, 19, 21], size=d) * 2.0 ** int(g.integers(-20, 20))
        elif kind == 2:                                        # the maximum at a border
            x[i, 0] = g.normal(size=d) * 0.1
            x[i, 0, 0] = g.choice([448, 446, 450, 2688, 2672, 2704, 1.75, 1.3125]) * 2.0 ** int(g.integers(-6, 6))
        elif kind == 3:
            x[i, 0] = g.normal(size=d) * 2.0 ** g.integers(-30, 10, size=d)
        elif kind == 4:
            x[i, 0] = g.normal(size=d) * g.choice([1e-38, 1e-36, 1e38])
    x = np.clip(x, -3.3e38, 3.3e38)
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    assert check_write(fmt, n, 1, d, 64, 10, list(range(n)), x=(t, -t)) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d, hkv, page, lengths", [(64, 2, 64, [1, 64, 65, 0, 200]), (128, 4, 128, [300, 0, 0, 1]),
                                                   (128, 1, 256, [1000]), (64, 3, 64, [5, 0])])
def test_read_gathers_every_token(fmt, d, hkv, page, lengths):
    import block_sparse_long_kv_gb300 as bsa
    need = [-(-n // page) for n in lengths]
    pages, stride = sum(need) + 2, max(max(need), 1) + 1
    cs = bsa.make_cache_shape(pages, page, hkv, d, fmt)
    cache = garbage_cache(bsa, cs)
    order = np.random.default_rng(1).permutation(pages)
    table = torch.full((len(lengths), stride), -9, dtype=torch.int32)
    x, slots, at = [], [], 0
    for b, n in enumerate(lengths):
        table[b, :need[b]] = torch.from_numpy(order[at:at + need[b]].astype(np.int32))
        at += need[b]
        slots += [int(table[b, i // page]) * page + i % page for i in range(n)]
    total = sum(lengths)
    k, v = rows(3, total, hkv, d), rows(4, total, hkv, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.cache_write(cs, k.cuda(), v.cuda(), torch.tensor(slots, dtype=torch.int32, device="cuda"), cache, st)
    cu = torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32, device="cuda")
    ko = torch.full((total + 3, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 7.0)
    bsa.cache_read(cs, cu, table.cuda(), max(lengths), cache, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for got, y in ((ko, k), (vo, v)):
        np.testing.assert_array_equal(got[:total].double().cpu().numpy(), C.held(y.double().numpy(), fmt))
        assert (got[total:] == 7).all()                        # rows behind the last sequence


@pytest.mark.parametrize("fmt", FMTS)
def test_read_bad_table_and_lengths(fmt):
    import block_sparse_long_kv_gb300 as bsa
    cs = bsa.make_cache_shape(4, 64, 2, 64, fmt)
    cache = garbage_cache(bsa, cs)
    k, v = rows(5, 256, 2, 64), rows(6, 256, 2, 64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.cache_write(cs, k.cuda(), v.cuda(), torch.arange(256, dtype=torch.int32, device="cuda"), cache, st)

    def read(cu, table, most=200):
        ko = torch.full((200, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        vo = torch.full_like(ko, 7.0)
        st.zero_()
        bsa.cache_read(cs, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                       torch.tensor(table, dtype=torch.int32, device="cuda"), most, cache, ko, vo, st)
        torch.cuda.synchronize()
        return ko.double().cpu().numpy(), vo.double().cpu().numpy(), int(st.item())

    hk = C.held(k.double().numpy(), fmt)
    for bad in (-1, 4, 1 << 30):
        ko, vo, code = read([0, 150], [[3, bad, 0, 0]])
        assert code == 1
        np.testing.assert_array_equal(ko[:64], hk[192:256])
        assert (ko[64:128] == 7).all() and (vo[64:128] == 7).all() and (ko[150:] == 7).all()
        np.testing.assert_array_equal(ko[128:150], hk[:22])
    # inconsistent entries read as empty sequences: too long, decreasing, past the end, negative
    for cu in ([0, 201], [0, 120, 60], [0, 50, 400], [-5, 30]):
        assert read(cu, [[0, 1, 2, 3]] * (len(cu) - 1))[2] == 1, cu
    assert read([0, 100, 150], [[0, 1, 2, 3]] * 2, most=99)[2] == 1
    ko, _, code = read([0, 0, 0], [[-1] * 4] * 2)
    assert code == 0 and (ko == 7).all()


def test_cache_past_32_bit_offsets():
    """Pages whose byte offsets pass 2^32: written, read back and attended to in place."""
    import block_sparse_long_kv_gb300 as bsa
    pages, page, hkv, d = 40000, 64, 16, 128                   # 5.2 GB of e4m3 codes for K and as much for V
    cs = bsa.make_cache_shape(pages, page, hkv, d, C.E4M3)
    cache = bsa.alloc_cache(cs)
    assert bsa.cache_code_bytes(cs) > 1 << 32
    table = torch.tensor([[39999, 39998, 5]], dtype=torch.int32, device="cuda")
    k, v = rows(8, 150, hkv, d), rows(9, 150, hkv, d)
    i = torch.arange(150, device="cuda")
    slots = (table[0, i // page] * page + i % page).int()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.cache_write(cs, k.cuda(), v.cuda(), slots, cache, st)
    ko, vo = torch.empty(150, hkv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(150, hkv, d, dtype=torch.bfloat16, device="cuda")
    bsa.cache_read(cs, torch.tensor([0, 150], dtype=torch.int32, device="cuda"), table, 150, cache, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    np.testing.assert_array_equal(ko.double().cpu().numpy(), C.held(k.double().numpy(), C.E4M3))
    np.testing.assert_array_equal(vo.double().cpu().numpy(), C.held(v.double().numpy(), C.E4M3))


def test_python_refusals():
    import block_sparse_long_kv_gb300 as bsa
    cs = bsa.make_cache_shape(2, 64, 2, 64, C.E4M3)
    cache = bsa.alloc_cache(cs)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        bsa.cache_write(cs, k.half(), k, slots, cache)
    with pytest.raises(TypeError):
        bsa.cache_write(cs, k, k, slots.long(), cache)
    with pytest.raises(ValueError):
        bsa.cache_write(cs, k, k, slots[:2], cache)
    with pytest.raises(TypeError):
        bsa.cache_write(cs, k, k, slots, dict(cache, k_scale=None))
    with pytest.raises(ValueError):
        bsa.cache_write(cs, k, k, slots, dict(cache, v=cache["v"].flatten()[:100]))
    with pytest.raises(RuntimeError):
        bsa.alloc_cache(bsa.make_cache_shape(2, 60, 2, 64, C.E4M3))
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        bsa.cache_read(cs, cu, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), 3, cache, k, k)
    with pytest.raises(RuntimeError):                          # 100 tokens need two pages of the table
        bsa.cache_read(cs, cu, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 100,
                       cache, torch.zeros(100, 2, 64, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(100, 2, 64, dtype=torch.bfloat16, device="cuda"))
