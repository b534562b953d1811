"""Pins of the latent-attention oracle: brute-force sums, closed forms,
finite differences, the absorbed form against the expanded one."""
import math

import numpy as np
import pytest

from oracle import latent as ol

SCALE = 192 ** -0.5


def _draw(seed, n_q, n_k, h):
    g = np.random.default_rng(seed)
    return g.standard_normal((n_q, h, 192)), g.standard_normal((n_k, h, 256)), g.standard_normal((n_k, 64))


@pytest.mark.parametrize("n_q,n_k,causal", [(1, 1, True), (3, 5, True), (4, 2, True), (3, 4, False), (2, 0, True)])
def test_attention_is_the_sum_over_visible_keys(n_q, n_k, causal):
    q, kv, kr = _draw(n_q * 10 + n_k, n_q, n_k, 2)
    got = ol.attention(q, kv, kr, causal, SCALE)
    for h in range(2):
        for i in range(n_q):
            keys = [j for j in range(n_k) if not causal or j <= i + n_k - n_q]
            e = [math.exp(SCALE * (sum(q[i, h, :128] * kv[j, h, :128]) + sum(q[i, h, 128:] * kr[j]))) for j in keys]
            if not keys:
                assert np.all(got["out"][i, h] == 0) and got["lse"][i, h] == -np.inf
                continue
            want = sum(w * kv[j, h, 128:] for w, j in zip(e, keys)) / sum(e)
            assert np.allclose(got["out"][i, h], want, rtol=1e-12, atol=1e-14)
            assert abs(got["lse"][i, h] - math.log(sum(e))) < 1e-12


def test_equal_keys_average_the_values():
    q, kv, kr = _draw(1, 4, 7, 1)
    kv[:, :, :128] = kv[0, :, :128]
    kr[:] = kr[0]
    out = ol.attention(q, kv, kr, False, SCALE)["out"]
    assert np.allclose(out[:, 0], kv[:, 0, 128:].mean(0), atol=1e-13)


@pytest.mark.parametrize("causal,n_q,n_k", [(True, 4, 6), (True, 6, 4), (False, 3, 5)])
def test_gradients_against_differences(causal, n_q, n_k):
    q, kv, kr = _draw(7, n_q, n_k, 2)
    g = np.random.default_rng(8)
    dout = g.standard_normal((n_q, 2, 128))
    grads = ol.attention_backward(dout, q, kv, kr, causal, SCALE)
    f = lambda: float((ol.attention(q, kv, kr, causal, SCALE)["out"] * dout).sum())
    step = 1e-5
    for name, x in (("dq", q), ("dkv", kv), ("dk_rope", kr)):
        for _ in range(12):
            at = tuple(g.integers(0, s) for s in x.shape)
            old = x[at]
            x[at] = old + step
            up = f()
            x[at] = old - step
            down = f()
            x[at] = old
            assert abs((up - down) / (2 * step) - grads[name][at]) < 1e-7, (name, at)


def test_absorbed_equals_expanded():
    g = np.random.default_rng(3)
    n, n_q, h = 11, 3, 2
    rows, w = g.standard_normal((n, 576)), g.standard_normal((h, 256, 512)) / 512 ** 0.5
    q = g.standard_normal((n_q, h, 192))
    kv = np.einsum("nr,hdr->nhd", rows[:, :512], w)
    a = ol.attention(q, kv, rows[:, 512:], True, SCALE)
    b = ol.cached(q, w, rows, SCALE)
    assert np.allclose(a["out"], b["out"], atol=1e-12) and np.allclose(a["lse"], b["lse"], atol=1e-12)
    # the chain 0 <- 1 <- 2 as a tree is the causal mask; a branch hides its sibling
    c = ol.cached(q, w, rows, SCALE, tree=[0b001, 0b011, 0b111])
    assert np.allclose(a["out"], c["out"], atol=1e-12)
    keep = [j for j in range(n) if j != n - 2]
    d = ol.cached(q, w, rows, SCALE, tree=[0b001, 0b011, 0b101])
    e = ol.attention(q[2:], kv[keep], rows[keep, 512:], True, SCALE)
    assert np.allclose(d["out"][2], e["out"][0], atol=1e-12)
    none = ol.cached(q[:1], w, rows[:1], SCALE, tree=[0])
    assert np.all(none["out"] == 0) and np.all(none["lse"] == -np.inf)


def test_rotation_keeps_lengths_and_depends_on_differences():
    g = np.random.default_rng(5)
    x, y = g.standard_normal((2, 64))
    freq = 10000.0 ** (-np.arange(32) / 32)
    for il in (True, False):
        r = lambda v, p: ol.rotate(v, p * freq, il)
        assert abs((r(x, 37) ** 2).sum() - (x ** 2).sum()) < 1e-12
        assert abs(r(x, 40) @ r(y, 33) - r(x, 7) @ r(y, 0)) < 1e-12
    row = ol.cache_row(g.standard_normal((3, 576)), 1.0, 0.0)
    assert np.allclose((row ** 2).mean(1), 1.0)
