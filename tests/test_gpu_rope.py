"""bsa_qk_norm_rope on the GPU against the float64 reference.

Tolerance, before the first run: the fast sine and cosine of an angle in [-pi, pi] are within 2^-21
of it, and the fp32 angle within 2^-21; products, sums and the norm's reciprocal root add a few 2^-23.
So an element is within 2^-18 of its pair's |a| + |b|, and the bf16 rounding adds 2^-8 of the value.
"""
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


def bf(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def check(got, x, w, pos, freq, eps, rotary, pairs, norm):
    want, size = C.norm_rope(f64(x), None if w is None else f64(w), pos, freq, eps, rotary, pairs, norm)
    err = np.abs(f64(got) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 1e-38).all(), float((err / (np.abs(want) + size + 1e-30)).max())


def run(tokens, hq, hkv, d, rotary, flags=0, eps=1e-6, weights=True, fused=False, inplace=False, first=0, seed=0):
    import block_sparse_long_kv_gb300 as bsa
    g = torch.Generator().manual_seed(seed)
    if fused:
        row = bf(g, tokens, (hq + 2 * hkv) * d).cuda()
        q, k = row[:, :hq * d].view(tokens, hq, d), row[:, hq * d:(hq + hkv) * d].view(tokens, hkv, d)
    else:
        row = None
        q, k = bf(g, tokens, hq, d).cuda(), bf(g, tokens, hkv, d).cuda()
    wq = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() if weights else None
    wk = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() if weights else None
    pos = (first + torch.arange(tokens)).int()
    freq = (1e4 ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary // 2))).float()
    q0, k0, row0 = q.clone(), k.clone(), None if row is None else row.clone()
    qo = q if inplace else torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    ko = k if inplace else torch.empty(tokens, hkv, d, dtype=torch.bfloat16, device="cuda")
    s = bsa.make_rope_shape(tokens, hq, hkv, d, rotary, eps, flags)
    bsa.qk_norm_rope(s, q, k, wq, wk, pos.cuda(), freq.cuda() if rotary else None, qo, ko)
    torch.cuda.synchronize()
    pairs, norm = bool(flags & bsa.ROPE_PAIRS), not flags & bsa.ROPE_NO_NORM
    check(qo, q0, wq, pos.numpy(), freq.numpy(), eps, rotary, pairs, norm)
    check(ko, k0, wk, pos.numpy(), freq.numpy(), eps, rotary, pairs, norm)
    if row is not None:
        v = slice((hq + hkv) * d, None)
        assert torch.equal(row[:, v], row0[:, v])           # the values' columns are not touched
    return qo, ko


@pytest.mark.parametrize("flags", [0, 1, 2, 3])
@pytest.mark.parametrize("d, rotary", [(128, 128), (128, 96), (128, 16), (64, 64), (64, 48), (64, 32)])
def test_styles(d, rotary, flags):
    run(37, 4, 2, d, rotary, flags)


@pytest.mark.parametrize("tokens, hq, hkv, d", [(1, 32, 4, 128), (1, 1, 1, 64), (3, 5, 3, 64), (2, 7, 1, 128),
                                                (1215, 4, 2, 128), (1216, 4, 2, 128), (1300, 3, 1, 64), (2500, 16, 1, 128)])
def test_token_and_head_counts(tokens, hq, hkv, d):
    run(tokens, hq, hkv, d, d, fused=True)


@pytest.mark.parametrize("first", [0, 131072 - 20, 1 << 20, (1 << 31) - 41])
def test_far_positions(first):
    run(40, 4, 2, 128, 128, first=first)


@pytest.mark.parametrize("fused", [False, True])
def test_in_place_gives_the_same_bits(fused):
    a = run(300, 8, 2, 128, 128, fused=fused)
    b = run(300, 8, 2, 128, 128, fused=fused, inplace=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_weights_no_rotation_and_zero_rows():
    run(9, 4, 2, 64, 0)
    run(9, 4, 2, 64, 0, weights=False, eps=1e-3)
    import block_sparse_long_kv_gb300 as bsa
    z = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    zk = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    qo, ko = torch.ones_like(z), torch.ones_like(zk)
    s = bsa.make_rope_shape(5, 4, 2, 64, 64)
    freq = torch.ones(32, device="cuda")
    bsa.qk_norm_rope(s, z, zk, None, None, torch.arange(5, dtype=torch.int32, device="cuda"), freq, qo, ko)
    assert (qo == 0).all() and (ko == 0).all()


def test_negative_positions_leave_rows_alone():
    import block_sparse_long_kv_gb300 as bsa
    q = torch.randn(6, 4, 128, device="cuda").to(torch.bfloat16)
    k = torch.randn(6, 2, 128, device="cuda").to(torch.bfloat16)
    pos = torch.tensor([3, -1, 7, -5, -1, 0], dtype=torch.int32, device="cuda")
    freq = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    qo, ko = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    s = bsa.make_rope_shape(6, 4, 2, 128, 128)
    bsa.qk_norm_rope(s, q, k, None, None, pos, freq, qo, ko)
    live = (pos >= 0).cpu()
    assert (qo[~live] == 5).all() and (ko[~live] == 5).all()
    check(qo[live], q[live], None, pos[live].cpu().numpy(), freq.cpu().numpy(), 1e-6, 128, False, True)
    check(ko[live], k[live], None, pos[live].cpu().numpy(), freq.cpu().numpy(), 1e-6, 128, False, True)


def test_python_refusals():
    import block_sparse_long_kv_gb300 as bsa
    q = torch.zeros(4, 4, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pos, freq = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(64, device="cuda")
    s = bsa.make_rope_shape(4, 4, 2, 128, 128)
    with pytest.raises(TypeError):
        bsa.qk_norm_rope(s, q.float(), k, None, None, pos, freq, q, k)
    with pytest.raises(TypeError):
        bsa.qk_norm_rope(s, q, k, None, None, pos.long(), freq, q, k)
    with pytest.raises(TypeError):
        bsa.qk_norm_rope(s, q.cpu(), k, None, None, pos, freq, q, k)
    with pytest.raises(ValueError):
        bsa.qk_norm_rope(s, q[:3], k, None, None, pos, freq, q, k)
    with pytest.raises(ValueError):
        bsa.qk_norm_rope(s, q.transpose(0, 1), k, None, None, pos, freq, q, k)
    with pytest.raises(ValueError):
        bsa.qk_norm_rope(s, q, k, None, None, pos[:2], freq, q, k)
    with pytest.raises(ValueError):
        bsa.qk_norm_rope(s, q, k, None, None, pos, freq[:32], q, k)
    with pytest.raises(RuntimeError):                         # an output inside the other input
        bsa.qk_norm_rope(s, q, k, None, None, pos, freq, q, q.view(-1)[:1024].view(4, 2, 128))
