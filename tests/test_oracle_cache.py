"""Pins for the reference of the norm / rotation, the cache formats and the drafted-token attention."""
import numpy as np
import pytest
import torch

from oracle import bsa_oracle as O
from oracle import cache_oracle as C
import synth


def test_rotation_keeps_norms_and_relative_angles():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 64))
    f = 10000.0 ** (-np.arange(16) / 16)
    for pairs in (False, True):
        y, _ = C.norm_rope(x, None, [0, 5, 131071], f, 0.0, 32, pairs, False)
        np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-12)
        np.testing.assert_array_equal(y[0], x[0])                # position 0 turns nothing
        np.testing.assert_array_equal(y[..., 32:], x[..., 32:])  # past the rotary dimensions
        a, _ = C.norm_rope(x[:1], None, [7], f, 0.0, 32, pairs, False)
        b, _ = C.norm_rope(x[1:2], None, [9], f, 0.0, 32, pairs, False)
        a2, _ = C.norm_rope(x[:1], None, [107], f, 0.0, 32, pairs, False)
        b2, _ = C.norm_rope(x[1:2], None, [109], f, 0.0, 32, pairs, False)
        np.testing.assert_allclose((a * b).sum(-1), (a2 * b2).sum(-1), rtol=1e-9)


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(1).normal(size=(4, 3, 128)) * 7
    y, _ = C.norm_rope(x, None, np.zeros(4), None, 0.0, 0, False, True)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)


def test_e4m3_table_is_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(C.E4M3_VALUES, t)
    assert C.E4M3_VALUES[-1] == 448.0
    np.testing.assert_array_equal(C.E2M1_VALUES, [0, 0.5, 1, 1.5, 2, 3, 4, 6])


def test_e4m3_rounding_is_torchs():
    x = np.random.default_rng(2).normal(size=5000).astype(np.float32) * np.float32(3.0) ** np.random.default_rng(3).integers(-6, 4, 5000)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = C._nearest(np.abs(x.astype(np.float64)), C.E4M3_VALUES) + 128 * np.signbit(x)
    np.testing.assert_array_equal(got, want)


def test_e2m1_ties_go_to_the_even_code():
    a = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0])
    np.testing.assert_array_equal(C.E2M1_VALUES[C._nearest(a, C.E2M1_VALUES)], [0, 1, 1, 2, 2, 4, 4, 6])


@pytest.mark.parametrize("fmt, most", [(C.E4M3, 448.0), (C.E2M1, 2688.0)])
def test_row_exponent_is_the_least(fmt, most):
    for amax in (1e-30, 0.1, 1.0, most, most * 1.0001, 447.9, 3.0e38):
        k = int(C._least_exponent(np.array([amax]), most)[0])
        assert amax <= most * 2.0 ** k and (k == -126 or amax > most * 2.0 ** (k - 1))
    assert C._least_exponent(np.array([0.0]), most)[0] == -126


@pytest.mark.parametrize("fmt", [C.E4M3, C.E2M1])
def test_held_values_are_close_and_bf16(fmt):
    x = synth.bf16_to_f64(synth.bf16_bits(np.random.default_rng(4).normal(size=(64, 128)).astype(np.float32)))
    h = C.held(x, fmt)
    np.testing.assert_array_equal(h, synth.bf16_to_f64(synth.bf16_bits(h.astype(np.float32))))
    # E4M3: half a step of the value, or of the smallest step of the row; E2M1: a code is within one unit
    # of its group scale (steps of 2 up to 6), and the saturation adds at most 6 * 2^-4 units
    if fmt == C.E4M3:
        bound = np.maximum(np.abs(x) * 2.0 ** -4, np.abs(x).max(-1, keepdims=True) / 448 * 2.0 ** -9)
    else:
        g = np.abs(x).reshape(64, 8, 16).max(-1).repeat(16, -1)
        bound = g / 6 * (1 + 2.0 ** -4) * (1 + 6 * 2.0 ** -4)
    assert (np.abs(h - x) <= bound).all()
    assert (C.held(np.zeros((2, 64)), fmt) == 0).all()


def test_a_chain_of_drafts_is_causal_attention():
    rng = np.random.default_rng(5)
    n, t, d = 40, 6, 16
    k, v = rng.normal(size=(1, n + t, 1, d)), rng.normal(size=(1, n + t, 1, d))
    q = rng.normal(size=(1, n + t, 2, d))
    od, ld = O.dense_attention(q, k, v)
    o, lse, _, _ = C.tree_attention(q[0, n:], k[0, n:, 0], v[0, n:, 0], k[0, :n, 0], v[0, :n, 0],
                                    np.arange(t) - 1, 1 / np.sqrt(d))
    np.testing.assert_allclose(o, od[0, n:], atol=1e-12)
    np.testing.assert_allclose(lse, ld[0, :, n:].T, atol=1e-12)


def test_siblings_do_not_see_each_other():
    rng = np.random.default_rng(6)
    q, kn, vn = rng.normal(size=(3, 1, 8)), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    k, v = rng.normal(size=(5, 8)), rng.normal(size=(5, 8))
    o, _, _, _ = C.tree_attention(q, kn, vn, k, v, [-1, 0, 0], 1.0)
    kn2, vn2 = kn.copy(), vn.copy()
    kn2[1], vn2[1] = 9.0, -9.0
    o2, _, _, _ = C.tree_attention(q, kn2, vn2, k, v, [-1, 0, 0], 1.0)
    np.testing.assert_array_equal(o[[0, 2]], o2[[0, 2]])
    assert not np.array_equal(o[1], o2[1])


@pytest.mark.parametrize("fmt", [C.E4M3, C.E2M1])
def test_inf_and_nan_are_held_as_nan(fmt):
    """The element's (E2M1: its group's) values are NaN, the others those of a row with zeros in their place."""
    x = synth.bf16_to_f64(synth.bf16_bits(np.random.default_rng(7).normal(size=(40, 64)).astype(np.float32)))
    bad = np.zeros(x.shape, bool)
    for t in range(40):
        bad[t, np.random.default_rng(t).permutation(64)[:t % 4]] = True
    lost = bad if fmt == C.E4M3 else bad.reshape(40, 4, 16).any(-1, keepdims=True).repeat(16, -1).reshape(40, 64)
    want = C.held(np.where(lost, 0.0, x), fmt)
    x[bad] = np.random.default_rng(8).choice([np.nan, np.inf, -np.inf], size=bad.sum())
    got = C.held(x, fmt)
    assert np.isnan(got[lost]).all()
    np.testing.assert_array_equal(got[~lost], want[~lost])
