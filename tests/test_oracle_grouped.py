"""Pins of the grouped-query attention oracle: closed forms, differences,
torch's own codes, what an append in pieces must give."""
import numpy as np
import pytest
import torch

from oracle import grouped as og
from oracle.latent import visible


def test_codes_are_torchs():
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(5000) * 50, og.E4M3[:127], -og.E4M3[:127],
                        (og.E4M3[:126] + og.E4M3[1:127]) / 2, g.uniform(-2.0 ** -8, 2.0 ** -8, 500)])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(og.e4m3(x.astype(np.float64)), want)
    vals = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(og.E4M3, vals, equal_nan=True)


def test_exponent_is_the_smallest():
    for a in (448.0, 448.01, 447.9, 1.75, 1.7500001, 1e-30, 2.0 ** -140, 3e38, 1.0):
        e = og.exponent(a)
        assert a <= 448 * 2.0 ** e and (e == -127 or a > 448 * 2.0 ** (e - 1))
    assert og.exponent(0.0) == -127


@pytest.mark.parametrize("cuts", [[40], [1] * 40, [7, 20, 13], [16, 16, 8]])
def test_pieces_give_the_same_cache(cuts):
    """Whole numbers of a few digits never lose one under a larger scale, so
    the pieces' second rounding changes nothing."""
    g = np.random.default_rng(1)
    x = g.integers(-8, 9, (40, 2, 64)) * 2.0 ** g.integers(0, 3, (40, 1, 1))
    c = og.Cache(4, 16, 2, 64)
    table, at = [2, 0, 3], 0
    for n in cuts:
        at += n
        c.append("k", x[at - n:at], table, at)
    assert np.array_equal(c.rows("k", table, 40), x)
    whole = og.Cache(4, 16, 2, 64)
    whole.append("k", x, table, 40)
    assert np.array_equal(whole.e["k"], c.e["k"])


def test_turn_is_a_complex_product_and_backward_its_transpose():
    g = np.random.default_rng(2)
    x, angle = g.standard_normal((3, 2, 64)), g.uniform(-9, 9, (3, 16))
    z = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) * np.exp(1j * angle)[:, None]
    y = og.turn(x, angle[:, None], 32, True)
    assert np.allclose(y[..., 0:32:2], z.real) and np.allclose(y[..., 1:32:2], z.imag)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    perm = np.r_[0:32:2, 1:32:2, 32:64]
    assert np.allclose(og.turn(x[..., perm], angle[:, None], 32, False), y[..., perm])


@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_gradients_are_differences(interleaved):
    g = np.random.default_rng(3)
    x, w, dy = g.standard_normal((2, 3, 64)), g.standard_normal(64), g.standard_normal((2, 3, 64))
    angle = g.uniform(-3, 3, (2, 16))
    f = lambda x, w: (og.norm_turn(x, w, 1e-3, angle, 32, interleaved)[0] * dy).sum()
    dx, _, dw, _ = og.norm_turn_backward(dy, x, w, 1e-3, angle, 32, interleaved)
    for _ in range(5):
        d, e = g.standard_normal(x.shape), g.standard_normal(64)
        assert np.isclose((f(x + 1e-6 * d, w) - f(x - 1e-6 * d, w)) / 2e-6, (dx * d).sum(), rtol=1e-6)
        assert np.isclose((f(x, w + 1e-6 * e) - f(x, w - 1e-6 * e)) / 2e-6, (dw * e).sum(), rtol=1e-6)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_gradients_are_differences(causal):
    g = np.random.default_rng(4)
    q, k, v, do = (g.standard_normal(s) for s in ((4, 6, 64), (7, 2, 64), (7, 2, 64), (4, 6, 64)))
    see = visible(4, 7, causal)
    f = lambda q, k, v: (og.attention(q, k, v, see, 0.2)["out"] * do).sum()
    r = og.attention_backward(do, q, k, v, causal, 0.2)
    for _ in range(3):
        a, b, c = (g.standard_normal(x.shape) for x in (q, k, v))
        for up, want in ((((a, 0, 0)), (r["dq"] * a).sum()), ((0, b, 0), (r["dk"] * b).sum()),
                         ((0, 0, c), (r["dv"] * c).sum())):
            h = 1e-6
            hi = f(q + h * up[0], k + h * up[1], v + h * up[2])
            lo = f(q - h * up[0], k - h * up[1], v - h * up[2])
            assert np.isclose((hi - lo) / (2 * h), want, rtol=1e-5, atol=1e-8)


def test_attention_of_a_lone_key_and_of_none():
    g = np.random.default_rng(5)
    q, k, v = g.standard_normal((3, 4, 64)), g.standard_normal((1, 2, 64)), g.standard_normal((1, 2, 64))
    r = og.attention(q, k, v, visible(3, 1, True), 0.125)
    assert not r["out"][:2].any() and np.isneginf(r["lse"][:2]).all()
    assert np.allclose(r["out"][2], v[0].repeat(2, 0)) and np.allclose(r["lse"][2], 0.125 * (q[2] * k[0].repeat(2, 0)).sum(-1))
    r = og.attention_backward(np.ones((3, 4, 64)), q, k, v, True, 0.125)
    assert np.allclose(r["dq"], 0) and np.allclose(r["dk"], 0) and np.allclose(r["dv"], 2)


def test_bytes_and_rows_agree():
    """The library's order of bytes, element by element."""
    g = np.random.default_rng(6)
    k = g.integers(0, 120, (2, 3, 2, 4, 16, 16)).astype(np.uint8)
    v = g.integers(0, 120, (2, 3, 2, 32, 2, 2, 2, 4)).astype(np.uint8)
    s = g.integers(120, 130, (2, 2, 3, 2)).astype(np.uint8)
    c = og.Cache.of_bytes(k, v, s[0], s[1])
    for page, h, t, d in ((0, 0, 0, 0), (1, 2, 29, 63), (1, 0, 22, 33), (0, 1, 13, 6)):
        b, i = divmod(t, 16)
        assert c.codes["k"][page, h, t, d] == k[page, h, b, d // 16, i, d % 16]
        assert c.codes["v"][page, h, t, d] == v[page, h, b, d // 2, (i // 4) % 2, d % 2, i // 8, i % 4]
    rows = c.rows("v", [1, 0], 40)
    assert rows[33, 2, 5] == og.E4M3[v[0, 2, 0, 2, 0, 1, 0, 1]] * 2.0 ** (int(s[1][0, 2, 0]) - 127)
