"""Pins of the latent attention oracle's root mean squares: they follow
simulated roundings, and the comparison that uses them refuses a decode that
leaves out tokens, at every size that the GPU tests run."""
import numpy as np
import pytest
import torch

from oracle import latent as ol
from tests.latent_util import decode_excess, row_excess
from tests.test_gpu_latent import DECODE

SCALE = 192 ** -0.5


def _bf(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).bfloat16().double().numpy()


def _draw(seed, n, n_q, h, q_std=1.0):
    g = np.random.default_rng(seed)
    return (q_std * g.standard_normal((n_q, h, 192)), g.standard_normal((h, 256, 512)) / 512 ** 0.5,
            g.standard_normal((n, 576)))


def test_spread_is_the_definition():
    q, w, rows = _draw(0, 70, 3, 2)
    for tree in (None, [0b001, 0b011, 0b000]):
        a, b = ol.cached(q, w, rows, SCALE, tree), ol.cached_spread(q, w, rows, SCALE, tree)
        assert np.allclose(a["out"], b["out"], atol=1e-12) and np.allclose(a["lse"], b["lse"], atol=1e-12)
    none = ol.cached_spread(q[:1], w, rows[:1], SCALE, [0])
    assert np.all(none["out"] == 0) and np.all(none["lse"] == -np.inf) and np.all(none["out_rms"] == 0)


@pytest.mark.parametrize("n", [1, 9, 66, 700])
def test_spread_follows_simulated_roundings(n):
    """q_lat, the weights and out rounded to bf16 in a simulation: rows stay
    inside, and the root mean square of all is not far below what is said."""
    q, w, rows = _draw(n, n, 1, 24)
    rows, w, q = _bf(rows), _bf(w), _bf(q)
    ref = ol.cached_spread(q, w, rows, SCALE)
    ql = _bf(np.einsum("hd,hdr->hr", q[0, :, :128], w[:, :128]))
    s = SCALE * (ql @ rows[:, :512].T + q[0, :, 128:] @ rows[:, 512:].T)
    e = np.exp(s - s.max(1, keepdims=True) + 0.3)
    o = _bf(np.einsum("hr,hdr->hd", (_bf(e) @ rows[:, :512]) / e.sum(1, keepdims=True), w[:, 128:]))[None]
    lse = (s.max(1) - 0.3 + np.log(e.sum(1)))[None]
    assert decode_excess(o, lse, ref) <= 0
    real, said = np.linalg.norm(o - ref["out"]), np.sqrt((ref["out_rms"] ** 2).sum())
    assert 0.4 < real / said < 1.2, real / said


SIZES = sorted({(n, n_q) for _, _, lens, nq in DECODE for n, n_q in zip(lens, nq) if n and n_q}
               | {(n, 1) for n in (1, 2, 3, 17, 40, 89, 4097, 9000)}          # many requests, the long ones
               | {(5888, 2), (5889, 2), (6337, 2)}                            # runs of one and of two tiles
               | {(100, 7), (48, 48), (75, 48), (61, 5), (130, 64)}           # trees
               | {(1500, 1), (300, 1), (700, 4), (700, 16), (200, 17), (70, 15), (130, 70), (66, 66), (150, 3)})


@pytest.mark.parametrize("n,n_q", SIZES)
def test_comparison_refuses_what_is_wrong(n, n_q):
    q, w, rows = _draw(n + n_q, n, n_q, 3)
    ref = ol.cached_spread(q, w, rows, SCALE)
    sees = np.isfinite(ref["lse"])
    assert decode_excess(ref["out"], ref["lse"], ref) <= 0
    excess = lambda out: (np.linalg.norm(out - ref["out"], axis=-1) / (6 * ref["out_rms"] + ref["out_floor"] + 1e-30))[sees]
    assert excess(np.zeros_like(ref["out"])).min() > 1, "zeros"
    assert excess(np.roll(ref["out"], 32, -1)).min() > 1, "another wave's columns"
    old = n - n_q
    for gone in {min(64, old), min(n // 2, old)} - {0}:                # a tile, half the cache
        less = ol.cached_spread(q, w, rows[gone:], SCALE)
        assert excess(less["out"]).max() > 1, f"{gone} tokens left out"
        assert decode_excess(ref["out"], less["lse"], ref) > 0, f"lse with {gone} tokens left out"
        twice = ol.cached_spread(q, w, np.concatenate([rows[:gone], rows]), SCALE)
        assert decode_excess(twice["out"], twice["lse"], ref) > 0, f"{gone} tokens counted twice"


@pytest.mark.parametrize("scale,q_std", [(1e-3, 20.0), (SCALE, 20.0)])
@pytest.mark.parametrize("n", [300, 1000])
def test_comparison_refuses_half_a_cache_at_other_scores(n, scale, q_std):
    q, w, rows = _draw(n, n, 1, 3, q_std)
    ref = ol.cached_spread(q, w, rows, scale)
    halves = [ol.cached_spread(q, w, part, scale) for part in (rows[n // 2:], rows[:n // 2])]
    # (far apart scores: one key may have nearly all the weight, in either half)
    assert max(decode_excess(x["out"], ref["lse"], ref) for x in halves) > 0
    assert decode_excess(np.zeros_like(ref["out"]), ref["lse"], ref) > 0
    assert row_excess(ref["out"] * 1.01, ref["out"], ref["out_rms"], ref["out_floor"]) < 0 < row_excess(
        ref["out"] * 1.06, ref["out"], ref["out_rms"], ref["out_floor"])


def _gradients(q, kv, kr, do, causal):
    a = ol.attention_backward(do, q, kv, kr, causal, SCALE)
    return a["dq"], a["dkv"], a["dk_rope"]


@pytest.mark.parametrize("n_q,n_k,causal", [(5, 5, True), (9, 4, True), (130, 130, True), (40, 90, False)])
def test_gradient_spread(n_q, n_k, causal):
    """The definition's gradients; simulated roundings stay inside; a key
    whose gradients are missing, a tile of keys that dq leaves out, a delta of
    0 do not."""
    h = 3
    q, kv, kr, do = (_bf(t) for t in (lambda g: (g.standard_normal((n_q, h, 192)), g.standard_normal((n_k, h, 256)),
                                                 g.standard_normal((n_k, 64)), g.standard_normal((n_q, h, 128))))(
        np.random.default_rng(n_q)))
    r = ol.attention_spread(do, q, kv, kr, causal, SCALE)
    dq, dkv, dkr = _gradients(q, kv, kr, do, causal)
    assert np.allclose(r["dq"], dq) and np.allclose(r["dkv"], dkv) and np.allclose(r["dk_rope"], dkr)
    see = ol.visible(n_q, n_k, causal)
    sim = {"out": np.zeros((n_q, h, 128)), "dq": np.zeros(q.shape), "dkv": np.zeros(kv.shape)}
    rope = np.zeros(kr.shape)
    for x in range(h):
        k = np.concatenate([kv[:, x, :128], kr], 1)
        s = np.where(see, SCALE * (q[:, x] @ k.T), -np.inf)
        m = np.max(s, 1, keepdims=True)
        e = np.exp(s - np.where(np.isfinite(m), m, 0) + 0.3)
        z = e.sum(1, keepdims=True)
        z[z == 0] = 1
        o = _bf(_bf(e) @ kv[:, x, 128:] / z)
        p = e / z
        ds = _bf(p * (do[:, x] @ kv[:, x, 128:].T - (do[:, x] * o).sum(1, keepdims=True)))
        dk = SCALE * ds.T @ q[:, x]
        sim["out"][:, x], sim["dq"][:, x] = o, _bf(SCALE * ds @ k)
        sim["dkv"][:, x] = _bf(np.concatenate([dk[:, :128], _bf(p).T @ do[:, x]], 1))
        rope += dk[:, 128:]
    parts = lambda dq, dkv, dkr: {"dq": dq, "dk": dkv[..., :128], "dv": dkv[..., 128:], "dk_rope": dkr}
    want = parts(r["dq"], r["dkv"], r["dk_rope"])
    ex = lambda name, got: row_excess(got, want[name], r[name + "_rms"], 2.0 ** -16 * (1 + np.linalg.norm(want[name], axis=-1)))
    assert row_excess(sim["out"], r["out"], r["out_rms"], 1e-9) <= 0
    for name, got in parts(sim["dq"], sim["dkv"], _bf(rope)).items():
        assert ex(name, got) <= 0, name
        assert ex(name, np.zeros_like(got)) > 0, name
    last = n_k - 1                                       # (with the causal order only the last query sees it)
    for name in ("dk", "dv"):
        less = want[name].copy()
        less[last] = 0
        assert ex(name, less) > 0, f"{name} of one key missing"
    part = n_k // 2
    assert ex("dq", _gradients(q, kv[part:], kr[part:], do, False)[0]) > 0, "keys left out"
