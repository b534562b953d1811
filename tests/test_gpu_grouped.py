"""GPU parity of grouped-query attention (norms with rotation, packed sequences
with gradients, the 8-bit cache, decode) against the fp64 oracle: every element
within the bound that the oracle derives from the bf16 roundings of a kernel's
matrix operands, every row within the root mean square they give; codes and
scales bit for bit."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_amd as moe
from mixture_experts_layer_sigmoid_amd import _lib as L
from oracle import grouped as og
from oracle.latent import visible
from tests.gpu_util import log
from tests.latent_util import row_excess

pytestmark = pytest.mark.gpu


def _bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _i32(v):
    return torch.tensor(np.asarray(v).tolist(), dtype=torch.int32, device="cuda")


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int)


def _inside(got, want, tol, what):
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), what
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok], want[~ok]), what
    far = np.abs(got[ok] - want[ok]) - tol[ok]
    assert far.size == 0 or far.max() <= 0, f"{what}: {far.max():.3e} over its bound"


def _rows_hold(got, ref, name, what):
    # fp32 sums: 2^-18 of a row's own size beside the roundings
    floor = 2.0 ** -18 * (np.linalg.norm(ref[name], axis=-1) + 1e-3)
    assert row_excess(got, ref[name], ref[name + "_rms"], floor) <= 0, f"{what}: rows of {name}"


def _check_lse(lse, want, what):
    # scores are exact products summed in fp32
    _inside(_np(lse), want, 1e-5 * (1 + np.abs(np.nan_to_num(want, neginf=0))), what + " lse")


# ---- norms and rotation ---------------------------------------------------------
NORM = [
    # T, heads, kv, D, rotary, interleaved, which weights
    (1, 1, 1, 64, 64, False, "qk"),
    (5, 12, 3, 128, 128, True, "qk"),
    (67, 64, 8, 128, 64, False, "qk"),
    (130, 5, 5, 64, 16, True, "q"),
    (9, 20, 4, 128, 96, False, "k"),
    (33, 3, 1, 64, 48, False, ""),
    (40, 16, 2, 128, 0, False, "qk"),               # no rotation
]


def _norm_case(T, h, kv, d, rotary, weights, seed=0):
    g = np.random.default_rng(seed + T)
    wide = _bf(g.standard_normal((T, (h + 2 * kv) * d + 16)) * g.uniform(0.01, 4, (T, 1)))
    q = wide[:, 8:8 + h * d].unflatten(1, (h, d))
    k = wide[:, 8 + h * d:8 + (h + kv) * d].unflatten(1, (kv, d))
    w = {n: _bf(1 + 0.2 * g.standard_normal(d)) if n in weights else None for n in "qk"}
    rot = {}
    if rotary:
        angle = g.uniform(-4, 4, (50, rotary // 2))
        cos, sin = (torch.from_numpy(f(angle).astype(np.float32)).cuda() for f in (np.cos, np.sin))
        pos = g.integers(0, 50, T)
        pos[0] = 70 if T > 2 else -3                 # past the table: its nearest row
        rot = dict(cos=cos, sin=sin, positions=_i32(pos))
        angle = angle[np.clip(pos, 0, 49)]
    return q, k, w, rot, angle if rotary else None, g


@pytest.mark.parametrize("T,h,kv,d,rotary,il,weights", NORM)
def test_norm_parity(gpu_lib, T, h, kv, d, rotary, il, weights):
    log(f"qk norm T={T} h={h}/{kv} D={d} rotary={rotary} interleaved={il} weights={weights}")
    q, k, w, rot, angle, g = _norm_case(T, h, kv, d, rotary, weights)
    eps = 1e-5
    plan = moe.QKNormRope(T=T + 3, n_heads=h, n_kv_heads=kv, head_dim=d, rotary=rotary or None, interleaved=il, eps=eps,
                          backward=True)
    bufs = (plan.q, plan.k, plan.dq, plan.dk)
    for t in bufs:
        t.fill_(7.0)
    plan.ws.fill_(255)
    got = plan(q, k, w["q"], w["k"], **rot)
    dy = _bf(g.standard_normal((T, h, d))), _bf(g.standard_normal((T, kv, d)))
    grads = plan.backward(*dy, q, k, w["q"], w["k"], **rot)
    torch.cuda.synchronize()
    for i, (n, x) in enumerate((("q", q), ("k", k))):
        wn = None if w[n] is None else _np(w[n])
        want, tol = og.norm_turn(_np(x), wn, eps, angle, rotary, il)
        _inside(_np(got[i]), want, tol + 1e-30, n)
        dx, dtol, dw, wtol = og.norm_turn_backward(_np(dy[i]), _np(x), wn, eps, angle, rotary, il)
        _inside(_np(grads[i]), dx, dtol + 1e-30, "d" + n)
        if wn is None:
            assert grads[2 + i] is None
        else:
            _inside(_np(grads[2 + i]), dw, wtol, "dw_" + n)
    assert all((t[T:] == 7).all() for t in bufs), "rows behind the call's"
    first = [t.clone() for t in (*got, *grads) if t is not None]
    plan(q, k, w["q"], w["k"], **rot)
    again = plan.backward(*dy, q, k, w["q"], w["k"], **rot)
    torch.cuda.synchronize()
    for x, y in zip(first, [t for t in (*got, *again) if t is not None]):
        assert torch.equal(x, y), "two runs differ"


def test_norm_in_place_and_many_tokens(gpu_lib):
    """In place in the projection's rows; more tokens than the backward has
    workgroups; zero and huge rows."""
    log("qk norm in place")
    T, h, kv, d = 4500, 3, 1, 64
    q, k, w, rot, angle, g = _norm_case(T, h, kv, d, 32, "qk")
    q[3], q[4] = 0, 1e18
    plan = moe.QKNormRope(T=T, n_heads=h, n_kv_heads=kv, head_dim=d, rotary=32, backward=True)
    want = [t.clone() for t in plan(q, k, w["q"], w["k"], **rot)]
    dy = _bf(g.standard_normal((T, h, d))), _bf(g.standard_normal((T, kv, d)))
    q[4] = 1                                          # its square is too large for fp32's sum of gradients
    grads = plan.backward(*dy, q, k, w["q"], w["k"], **rot)
    for i, (n, x) in enumerate((("q", q), ("k", k))):
        _, _, dw, tol = og.norm_turn_backward(_np(dy[i]), _np(x), _np(w[n]), 1e-6, angle, 32, False)
        _inside(_np(grads[2 + i]), dw, tol, "dw_" + n)
    q[4] = 1e18
    L.moe_qk_norm_rope(q, q.stride(0), k, k.stride(0), 1, w["q"], w["k"], 1e-6, rot["cos"], rot["sin"], 50,
                       rot["positions"], 32, 0, T, h, kv, d, q, q.stride(0), k, k.stride(0))
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.isfinite(want[0].float()).all() and not want[0][3].any()


def test_norm_of_no_tokens(gpu_lib):
    plan = moe.QKNormRope(T=4, n_heads=2, n_kv_heads=1, head_dim=64, backward=True)
    q, k = (torch.empty((0, n, 64), dtype=torch.bfloat16, device="cuda") for n in (2, 1))
    w = _bf(np.ones(64))
    got = plan(q, k, w, w)
    plan.dw_q.fill_(3), plan.dw_k.fill_(3)
    dq, dk, dw_q, dw_k = plan.backward(q, k, q, k, w, w)
    torch.cuda.synchronize()
    assert got[0].shape == dq.shape == (0, 2, 64) and not dw_q.any() and not dw_k.any()


# ---- packed sequences -------------------------------------------------------------
def _draw(seed, lens_q, lens_k, h, kv, d, std=1.0):
    g = np.random.default_rng(seed)
    tq, tk = sum(lens_q), sum(lens_k)
    mk = lambda *s: _bf(g.standard_normal(s))
    return _bf(g.standard_normal((tq, h, d)) * std), mk(tk, kv, d), mk(tk, kv, d), mk(tq, h, d)


def _reference(ins, lens_q, lens_k, causal, scale):
    q, k, v, do = (_np(t) for t in ins)
    parts = []
    for a, b, c, e in zip(_cu(lens_q), _cu(lens_q)[1:], _cu(lens_k), _cu(lens_k)[1:]):
        r = og.attention(q[a:b], k[c:e], v[c:e], visible(b - a, e - c, causal), scale)
        parts.append(r | og.attention_backward(do[a:b], q[a:b], k[c:e], v[c:e], causal, scale))
    return {n: np.concatenate([p[n] for p in parts]) for n in parts[0]}


PACKED = [
    # heads, kv, D, lens_q, lens_k, causal
    (1, 1, 128, [1], [1], True),
    (6, 2, 64, [1, 37, 130, 64, 65], [1, 37, 130, 64, 65], True),
    (8, 1, 128, [5, 0, 33], [70, 4, 0], False),       # a sequence without queries, one without keys
    (4, 4, 64, [100, 3], [30, 3], True),              # the first 70 queries see nothing
    (10, 2, 128, [31, 1, 9], [129, 200, 63], True),   # later pieces of longer prompts; groups of 5
    (14, 2, 64, [200], [201], False),
    (24, 2, 128, [129, 20], [129, 84], True),         # groups of 12
    (3, 1, 128, [320], [320], True),                  # the backward's rows in parts
    (8, 2, 64, [3, 20], [1500, 700], True),           # the forward's keys in parts
    (2, 1, 128, [1, 5, 2], [2100, 0, 3], False),      # parts without keys
    (12, 4, 128, [40, 7], [900, 600], False),
    # more sequences than a wave has lanes, some empty on either side
    (4, 2, 64, [5 * i % 11 for i in range(150)], [5 * i % 11 + i % 3 for i in range(150)], True),
    (6, 1, 128, [i % 3 for i in range(200)], [7 * i % 90 for i in range(200)], False),
    # many rows of long sequences: the backward's larger workgroups
    (512, 16, 128, [129], [600], True),
    (256, 8, 64, [200, 0, 57], [1500, 9, 300], False),
    (110, 22, 64, [597, 3], [1197, 3], True),
    (704, 22, 128, [129], [1201], True),
    (512, 8, 64, [130, 0, 57], [2500, 1109, 0], False),
    (360, 72, 128, [251], [1250], True),
]


@pytest.mark.parametrize("h,kv,d,lens_q,lens_k,causal", PACKED)
def test_attention_parity(gpu_lib, h, kv, d, lens_q, lens_k, causal):
    log(f"grouped attention {h}/{kv} D={d} {lens_q} {lens_k} causal={causal}")
    ins = _draw(h + len(lens_q), lens_q, lens_k, h, kv, d)
    ref = _reference(ins, lens_q, lens_k, causal, d ** -0.5)
    a = moe.GroupedAttention(Tq=sum(lens_q) + 5, Tk=sum(lens_k) + 9, n_heads=h, n_kv_heads=kv, head_dim=d,
                             n_seqs=len(lens_q) + 1, causal=causal, backward=True)
    bufs = (a.out, a.lse, a.dq, a.dk, a.dv)
    for t in bufs:
        t.fill_(7.0)
    a.ws.fill_(255)                                     # NaN wherever it is read before it is written
    cu = _i32(_cu(lens_q)), _i32(_cu(lens_k))
    out, lse = a.forward(*ins[:3], *cu)
    grads = a.backward(ins[3], *ins[:3], *cu)
    torch.cuda.synchronize()
    _inside(_np(out), ref["out"], ref["out_tol"], "out")
    _check_lse(lse, ref["lse"], "forward")
    for name, t in zip(("dq", "dk", "dv"), grads):
        _inside(_np(t), ref[name], ref[name + "_tol"], name)
    for name, t in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        _rows_hold(_np(t), ref, name, "attention")
    for t, x in zip(bufs, (out, lse, *grads)):
        assert (t[x.shape[0]:] == 7).all(), "rows behind the call's"
    first = [t.clone() for t in (out, lse, *grads)]
    a.forward(*ins[:3], *cu)
    a.backward(ins[3], *ins[:3], *cu)
    torch.cuda.synchronize()
    for x, y in zip(first, (out, lse, *grads)):
        assert torch.equal(x, y), "two runs differ"


@pytest.mark.parametrize("scale,std", [(128 ** -0.5, 40.0), (1e-3, 1.0), (2.0, 1.0)])
def test_attention_score_ranges(gpu_lib, scale, std):
    """Scores from nearly equal to hundreds apart."""
    log(f"grouped attention scale={scale} std={std}")
    lens = [90, 141]
    ins = _draw(5, lens, lens, 4, 2, 128, std)
    ref = _reference(ins, lens, lens, True, scale)
    a = moe.GroupedAttention(Tq=231, Tk=231, n_heads=4, n_kv_heads=2, n_seqs=2, scale=scale)
    out, lse = a(*ins[:3], _i32(_cu(lens)), _i32(_cu(lens)))
    torch.cuda.synchronize()
    # fp32 scores of this size: their rounding moves weights by up to 2^-22 |s|
    _inside(_np(out), ref["out"], ref["out_tol"] + 2.0 ** -19 * np.abs(ref["lse"]).max(), "out")
    _check_lse(lse, ref["lse"], f"scale {scale}")


def test_attention_strides_outside_rows_and_hidden_nan(gpu_lib):
    """Slices of one projection's rows, rows outside every sequence (NaN in,
    untouched out), NaN in a hidden key and in neighbouring sequences."""
    log("grouped attention strides")
    h, kv, d, pad = 6, 2, 128, 9
    lens = [40, 70]
    q, k, v, do = _draw(11, lens, lens, h, kv, d)
    ref = _reference((q, k, v, do), lens, lens, True, d ** -0.5)
    nan = float("nan")
    qkv = torch.full((110 + 2 * pad, (h + 2 * kv) * d + 8), nan, dtype=torch.bfloat16, device="cuda")
    cut = lambda t, at, n: t[:, at:at + n * d].unflatten(1, (n, d))
    wq, wk, wv = cut(qkv, 0, h), cut(qkv, h * d, kv), cut(qkv, (h + kv) * d, kv)
    wdo = torch.full((110 + 2 * pad, h * d + 24), nan, dtype=torch.bfloat16, device="cuda")
    held = slice(pad, pad + 110)
    for w, x in ((wq, q), (wk, k), (wv, v), (cut(wdo, 0, h), do)):
        w[held] = x
    cu = _i32(_cu(lens) + pad)
    T = qkv.shape[0]
    mk = lambda n: torch.full((T, n + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out, dqkv = mk(h * d), mk((h + 2 * kv) * d)
    lse = torch.full((T, h), 7.0, device="cuda")
    ws = torch.empty(L.moe_gqa_attn_bwd_workspace(T, T, h, kv, d), dtype=torch.uint8, device="cuda")
    ld = lambda t: t.stride(0)
    heads = (1, cu, cu, 2, T, T, h, kv, d, 1, d ** -0.5)
    fws = torch.empty(L.moe_gqa_attn_fwd_workspace(T, h, d), dtype=torch.uint8, device="cuda")
    L.moe_gqa_attn_fwd(wq, ld(wq), wk, ld(wk), wv, ld(wv), *heads, out, ld(out), lse, fws)
    dq, dk, dv = cut(dqkv, 0, h), cut(dqkv, h * d, kv), cut(dqkv, (h + kv) * d, kv)
    L.moe_gqa_attn_bwd(wdo, ld(wdo), wq, ld(wq), wk, ld(wk), wv, ld(wv), 1, out, ld(out), lse, *heads[1:], dq, ld(dq),
                       dk, ld(dk), dv, ld(dv), ws)
    torch.cuda.synchronize()
    _inside(_np(out[held, :h * d].unflatten(1, (h, d))), ref["out"], ref["out_tol"], "out")
    _check_lse(lse[held], ref["lse"], "strided")
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _inside(_np(t[held]), ref[name], ref[name + "_tol"], name)
    for t, n in ((out, h * d), (lse, h), (dqkv, (h + 2 * kv) * d)):
        assert (t[:pad] == 7).all() and (t[pad + 110:] == 7).all() and (t[:, n:] == 7).all()
    # the first sequence's last key is hidden from every query but the last
    k2 = k.clone()
    k2[39] = nan
    a = moe.GroupedAttention(Tq=110, Tk=110, n_heads=h, n_kv_heads=kv, n_seqs=2)
    o2, _ = a(q, k2, v, _i32(_cu(lens)), _i32(_cu(lens)))
    torch.cuda.synchronize()
    rest = np.r_[0:39, 40:110]
    assert np.isnan(_np(o2)[39]).all()
    _inside(_np(o2)[rest], ref["out"][rest], ref["out_tol"][rest], "beside NaN keys")


def test_attention_rows_past_4gb(gpu_lib):
    """Row offsets beyond 2^32 bytes."""
    log("grouped attention wide rows")
    n, ld = 9000, 1 << 18
    buf = torch.empty((n, ld), dtype=torch.bfloat16, device="cuda")        # 4.7 GB
    g = np.random.default_rng(2)
    q, k, v = _bf(g.standard_normal((3, 2, 64))), _bf(g.standard_normal((n, 1, 64))), _bf(g.standard_normal((n, 1, 64)))
    wk, wv = buf[:, :64].unflatten(1, (1, 64)), buf[:, 64:128].unflatten(1, (1, 64))
    wk.copy_(k), wv.copy_(v)
    a = moe.GroupedAttention(Tq=3, Tk=n, n_heads=2, n_kv_heads=1, head_dim=64, n_seqs=1)
    out, lse = a(q, wk, wv, _i32([0, 3]), _i32([0, n]))
    torch.cuda.synchronize()
    ref = og.attention(_np(q), _np(k), _np(v), visible(3, n, True), 0.125)
    _inside(_np(out), ref["out"], ref["out_tol"], "wide rows")
    _check_lse(lse, ref["lse"], "wide rows")


def test_attention_gradient_is_the_difference(gpu_lib):
    """dk and dv of shared heads against differences of the forward itself,
    along the directions of the gradients."""
    log("grouped attention differences")
    h, kv, d, n = 8, 2, 64, 96
    q, k, v, do = _draw(21, [n], [n], h, kv, d)
    cu = _i32([0, n])
    a = moe.GroupedAttention(Tq=n, Tk=n, n_heads=h, n_kv_heads=kv, head_dim=d, n_seqs=1, backward=True)
    a.forward(q, k, v, cu, cu)
    grads = [t.double() for t in a.backward(do, q, k, v, cu, cu)]
    ins = [q, k, v]
    for i, gr in enumerate(grads):
        step = (gr / gr.abs().max() * 0.25).bfloat16()
        hi, lo = ((x.float() + s * step.float()).bfloat16() for x, s in ((ins[i], 1), (ins[i], -1)))
        f = []
        for x in (hi, lo):
            o, _ = a.forward(*(x if j == i else y for j, y in enumerate(ins)), cu, cu)
            f.append((o.double() * do.double()).sum().item())
        want = (gr * (hi.double() - lo.double())).sum().item()
        # the outputs' roundings (2^-8 / sqrt(3) of each of n h d terms, two
        # sides, 6 root mean squares) and the third order of a step this size
        noise = 6 * 2 ** 0.5 * (a.out.double() * do.double()).norm().item() * 2.0 ** -8
        assert abs(f[0] - f[1] - want) <= noise + 0.05 * abs(want), (i, f[0] - f[1], want)


# ---- the cache ----------------------------------------------------------------------
class Paged:
    """Requests' tokens scattered over the pages of a cache that is all NaN
    codes and scale 255 elsewhere."""

    def __init__(self, seed, lens, page, kv, d, spare=2, fill=0x7F):
        self.g = np.random.default_rng(seed)
        self.lens, self.page, self.kv, self.d = list(lens), page, kv, d
        need = [-(-n // page) for n in lens]
        ids = self.g.permutation(sum(need) + spare)
        self.cache = moe.GroupedCache.empty(sum(need) + spare, page, kv, d)
        for t in (self.cache.k, self.cache.v):
            t.fill_(fill)
        for t in (self.cache.k_scales, self.cache.v_scales):
            t.fill_(255)
        self.table = np.full((len(lens), max(1, max(need, default=1))), 2 ** 30, np.int64)   # unused: no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n

    def bytes(self):
        c = self.cache
        return [t.cpu().numpy().copy() for t in (c.k, c.v, c.k_scales, c.v_scales)]

    def oracle(self):
        return og.Cache.of_bytes(*self.bytes())

    def draw(self, n):
        """n tokens' keys and values, of uneven size."""
        s = 2.0 ** self.g.integers(-3, 4, (n, 1, 1))
        return [_bf(self.g.standard_normal((n, self.kv, self.d)) * s) for _ in range(2)]

    def append(self, lens, new, k, v, stream=None):
        moe.grouped_cache_append(k, v, self.cache, _i32(self.table), _i32(lens), _i32(_cu(new)), stream=stream)

    def fill(self):
        """All requests' tokens at once."""
        k, v = self.draw(sum(self.lens))
        self.append(self.lens, self.lens, k, v)


APPENDS = [
    # lens at the end, page, kv, D, new tokens a call (each request's, in turn)
    ([1], 16, 1, 128, [[1]]),
    ([40, 17, 33], 16, 2, 64, [[1, 17, 30], [39, 0, 3]]),
    ([100, 5, 64], 48, 3, 128, [[60, 5, 16], [1, 0, 16], [1, 0, 31], [38, 0, 1]]),
    ([37], 32, 1, 64, [[1]] * 37),
    ([200, 200], 128, 1, 128, [[100, 3], [100, 197]]),
    # more requests than a wave has lanes
    ([i % 23 + i % 2 for i in range(150)], 16, 2, 64, [[i % 23 for i in range(150)], [i % 2 for i in range(150)]]),
]


@pytest.mark.parametrize("lens,page,kv,d,calls", APPENDS)
def test_append_parity(gpu_lib, lens, page, kv, d, calls):
    """Codes, scales and everything around them, bit for bit, after each call."""
    log(f"grouped append {lens} page={page} kv={kv} D={d}")
    pg = Paged(len(lens) + page, lens, page, kv, d)
    at = [0] * len(lens)
    for new in calls:
        at = [a + n for a, n in zip(at, new)]
        k, v = pg.draw(sum(new))
        want = pg.oracle()
        pg.append(at, new, k, v)
        torch.cuda.synchronize()
        cu = _cu(new)
        for name, x in (("k", _np(k)), ("v", _np(v))):
            for b, n in enumerate(new):
                if n:
                    want.append(name, x[cu[b]:cu[b + 1]], pg.table[b], at[b])
        got = pg.oracle()
        for name in "kv":
            assert np.array_equal(got.codes[name], want.codes[name]), name
            assert np.array_equal(got.e[name], want.e[name]), name
    assert at == lens


def test_append_values_of_every_size(gpu_lib):
    """Zeros, the smallest and largest magnitudes, signs of zeros, ties."""
    log("grouped append sizes")
    pg = Paged(3, [64], 16, 1, 64)
    k, v = (torch.zeros((64, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[0, 0, 0], k[0, 0, 1] = 448.0, -0.0
    k[1, 0, :] = torch.arange(64, device="cuda") * 0.0078125           # ties under scale 1
    k[16, 0, 3], k[17, 0, 5] = 2.0 ** 126, -1.0
    k[32, 0, 7], k[33, 0, 1] = 2.0 ** -133, -(2.0 ** -130)
    v[0, 0, 9], v[20, 0, 1], v[33, 0, 63] = 449.0, 450.0, 1.75
    want = pg.oracle()
    pg.append([64], [64], k, v)
    torch.cuda.synchronize()
    for name, x in (("k", k), ("v", v)):
        want.append(name, _np(x), pg.table[0], 64)
        got = pg.oracle()
        assert np.array_equal(got.codes[name], want.codes[name]) and np.array_equal(got.e[name], want.e[name])
    # NaN and infinities leave NaN codes, and only the block's own tokens coarser
    before = pg.bytes()
    k, v = pg.draw(16)
    k[3, 0, 2], v[5, 0, 6], v[5, 0, 7] = float("nan"), float("inf"), float("-inf")
    moe.grouped_cache_append(k, v, pg.cache, _i32(pg.table[:, 1:2]), _i32([16]), _i32([0, 16]))
    torch.cuda.synchronize()
    c = pg.oracle()
    page = pg.table[0, 1]
    assert np.isnan(og.E4M3[c.codes["k"][page, 0, 3, 2]]) and np.isnan(og.E4M3[c.codes["v"][page, 0, 5, 6:8]]).all()
    assert np.isfinite(og.E4M3[c.codes["k"][page, 0]]).sum() == 16 * 64 - 1
    rest = np.setdiff1d(np.arange(pg.cache.n_pages), page)
    for x, y in zip(before, pg.bytes()):
        assert np.array_equal(x[rest], y[rest])


def test_append_strides_and_tokens_without_place(gpu_lib):
    """Slices of a projection's rows; more rows than the request has tokens;
    rows outside every request; lengths beyond the table."""
    log("grouped append strides")
    kv, d = 2, 128
    g = np.random.default_rng(8)
    qkv = _bf(g.standard_normal((30, 6 * d)))
    k, v = qkv[:, 2 * d:4 * d].unflatten(1, (kv, d)), qkv[:, 4 * d:].unflatten(1, (kv, d))
    pg = Paged(8, [20, 32], 16, kv, d)
    want = pg.oracle()
    # request 0: 12 rows, its 5 tokens are the last 5; request 1: clamped to its 32 places
    moe.grouped_cache_append(k, v, pg.cache, _i32(pg.table), _i32([5, 900]), _i32([2, 14, 24]))
    torch.cuda.synchronize()
    for name, x in (("k", _np(k)), ("v", _np(v))):
        want.append(name, x[9:14], pg.table[0], 5)
        want.append(name, x[14:24], pg.table[1], 32)
        got = pg.oracle()
        # the second request's block held earlier tokens of scale 255, which stays
        assert np.array_equal(got.e[name], want.e[name])
        assert np.array_equal(got.codes[name], want.codes[name])


# ---- decode -------------------------------------------------------------------------
def _decode(pg, q, nq, scale=None, tree=None, lens=None, plan=None, stream=None):
    h = q.shape[1]
    plan = plan or moe.GroupedDecode(n_heads=h, n_kv_heads=pg.kv, head_dim=pg.d, max_tokens=q.shape[0],
                                     max_seqs=len(nq), scale=scale)
    lse = torch.full((q.shape[0], h), 7.0, device="cuda")
    out = plan(q, pg.cache, _i32(pg.table), _i32(pg.lens if lens is None else lens), _i32(_cu(nq)), tree, lse, stream)
    return out, lse


def _check_decode(pg, q, nq, out, lse, scale=None, tree=None, lens=None, what="decode", fp32=0.0):
    c, lens = pg.oracle(), pg.lens if lens is None else lens
    cu, qn = _cu(nq), _np(q)
    scale = pg.d ** -0.5 if scale is None else scale
    for b, n in enumerate(lens):
        if not nq[b]:
            continue
        rows = slice(cu[b], cu[b + 1])
        words = None if tree is None else [int(w) & (2 ** 64 - 1) for w in tree[rows].tolist()]
        see = og.new_tokens_see(nq[b], n, words)
        ref = og.attention(qn[rows], c.rows("k", pg.table[b], n), c.rows("v", pg.table[b], n), see, scale)
        _inside(_np(out[rows]), ref["out"], ref["out_tol"] + fp32, f"{what}, request {b}")
        if lse is not None:
            _check_lse(lse[rows], ref["lse"], f"{what}, request {b}")
        if not fp32:
            _rows_hold(_np(out[rows]), ref, "out", f"{what}, request {b}")


DECODES = [
    # lens, page, heads, kv, D, new tokens a request, tree
    ([1], 16, 1, 1, 128, [1], False),
    ([33, 1, 700, 64], 16, 8, 2, 64, [1, 1, 1, 1], False),
    ([531], 64, 64, 8, 128, [1], False),
    ([90, 5, 300], 48, 10, 2, 128, [4, 5, 1], False),          # a chain; a request all new; groups of 5
    ([40, 200], 32, 16, 1, 64, [7, 3], False),                 # 112 packed rows
    ([130, 9, 64], 16, 8, 2, 128, [9, 9, 4], True),
    ([500], 128, 4, 4, 64, [64], True),
    ([3, 0, 2], 16, 4, 2, 128, [3, 0, 5], False),              # nothing cached, no rows, more rows than tokens
    # more segments than run at once, some cut, short ones last
    ([1, 33, 5000, 700, 2, 64, 31, 0, 340], 64, 32, 32, 64, [1, 1, 1, 2, 1, 1, 1, 1, 1], False),
    ([7 * i % 90 for i in range(66)] + [6000, 4100, 30, 2900], 32, 8, 4, 128, [1] * 70, False),
    ([20 + i for i in range(200)], 16, 8, 4, 64, [1] * 200, False),
]


@pytest.mark.parametrize("lens,page,h,kv,d,nq,tree", DECODES)
def test_decode_parity(gpu_lib, lens, page, h, kv, d, nq, tree):
    log(f"grouped decode {lens} page={page} {h}/{kv} D={d} nq={nq} tree={tree}")
    pg = Paged(sum(lens) + h, lens, page, kv, d)
    pg.fill()
    q = _bf(pg.g.standard_normal((sum(nq), h, d)))
    words = None
    if tree:
        w = [int(pg.g.integers(0, 2 ** 62)) & ((1 << i) - 1) | (1 << i) for n in nq for i in range(n)]
        w[0] = 0                                                # sees the earlier tokens only
        words = torch.tensor([x - (1 << 64) if x >> 63 else x for x in w], dtype=torch.int64, device="cuda")
    out, lse = _decode(pg, q, nq, tree=words)
    torch.cuda.synchronize()
    _check_decode(pg, q, nq, out, lse, tree=words)
    first = out.clone()
    again, _ = _decode(pg, q, nq, tree=words)
    torch.cuda.synchronize()
    assert torch.equal(first, again), "two runs differ"


def test_decode_in_pieces(gpu_lib):
    """Long and short requests of one call: caches cut into many pieces, more
    tiles a wave than one look into the page table serves."""
    log("grouped decode pieces")
    lens = [140000, 2, 700, 33, 9000]
    pg = Paged(5, lens, 16, 1, 64)
    pg.fill()
    q = _bf(pg.g.standard_normal((5, 2, 64)) * 2)
    out, lse = _decode(pg, q, [1] * 5)
    torch.cuda.synchronize()
    # fp32 sums of 140000 weights: 2^-24 sqrt(n) of their size and less
    _check_decode(pg, q, [1] * 5, out, lse, fp32=1e-6, what="pieces")
    # 40 tiles of rows over one cache: a piece has 371 tiles, a wave 93
    pg = Paged(6, [70000], 64, 1, 64, spare=1)
    pg.fill()
    q = _bf(pg.g.standard_normal((40, 32, 64)))
    out, lse = _decode(pg, q, [40])
    torch.cuda.synchronize()
    _check_decode(pg, q, [40], out, lse, fp32=1e-6, what="70000 tokens")


def test_decode_score_ranges(gpu_lib):
    log("grouped decode score ranges")
    pg = Paged(6, [300, 1000], 64, 2, 128)
    pg.fill()
    q = _bf(pg.g.standard_normal((2, 6, 128)) * 20)
    for scale in (1e-3, 0.05):
        out, lse = _decode(pg, q, [1, 1], scale=scale)
        torch.cuda.synchronize()
        # fp32 scores up to several hundred: weights move by 2^-22 of them
        _check_decode(pg, q, [1, 1], out, lse, scale=scale, fp32=2.0 ** -12 * scale / 0.05, what=f"scale {scale}")


def test_decode_hidden_nan(gpu_lib):
    """NaN codes in new tokens reach only the new tokens that see them; what
    lies behind a request's length reaches nobody (every other byte is NaN)."""
    log("grouped decode hidden NaN")
    h, kv, d = 4, 2, 128
    pg = Paged(9, [70], 16, kv, d)
    pg.fill()
    q = _bf(pg.g.standard_normal((4, h, d)))
    clean = _np(_decode(pg, q, [4])[0])
    page, at = int(pg.table[0, 68 // 16]), 68 % 16
    for name in "kv":
        save = [t.clone() for t in (pg.cache.k, pg.cache.v)]
        if name == "k":
            pg.cache.k[page, 1, 0, 2, at, 5] = 0xFF
        else:
            pg.cache.v[page, 1, 0, 33 // 2, (at // 4) % 2, 1, at // 8, at % 4] = 0x7F
        got = _np(_decode(pg, q, [4])[0])                       # token 68 is new token 2
        assert np.array_equal(got[:2], clean[:2]) and np.array_equal(got[:, :2], clean[:, :2]), name
        bad = got[2:, 2:]
        if name == "k":
            assert np.isnan(bad).all()
        else:
            assert np.isnan(bad[..., 33]).all() and np.isfinite(np.delete(bad, 33, -1)).all()
            rest = np.delete(bad, 33, -1)
            assert np.array_equal(rest, np.delete(clean[2:, 2:], 33, -1))
        tree = torch.tensor([1, 2, 4, 8], dtype=torch.int64, device="cuda")
        got = _np(_decode(pg, q, [4], tree=tree)[0])
        assert np.isfinite(got[[0, 1, 3]]).all() and np.isnan(got[2, 2:]).any(), name
        pg.cache.k.copy_(save[0]), pg.cache.v.copy_(save[1])


def test_decode_strides_and_rows_left_alone(gpu_lib):
    log("grouped decode strides")
    h, kv, d = 6, 2, 64
    pg = Paged(12, [50, 90], 32, kv, d)
    pg.fill()
    wide = _bf(pg.g.standard_normal((9, h * d + 40)))
    q = wide[:, 16:16 + h * d].unflatten(1, (h, d))
    out = torch.full((9, h * d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, h), 7.0, device="cuda")
    ws = torch.zeros(L.moe_gqa_decode_workspace(d), dtype=torch.uint8, device="cuda")
    table, cu = _i32(pg.table), _i32([2, 3, 6])                 # rows 0, 1 and 6 .. 8 are nobody's
    L.moe_gqa_decode(q, q.stride(0), 1, *pg.cache._tensors(), table, table.shape[1], _i32(pg.lens), cu, None, 2, 9, h,
                     kv, d, d ** -0.5, out, out.stride(0), lse, ws)
    torch.cuda.synchronize()
    _check_decode(pg, q[2:6], [1, 3], out[2:6, :h * d].unflatten(1, (h, d)), lse[2:6])
    rest = [0, 1, 6, 7, 8]
    assert (out[rest] == 7).all() and (lse[rest] == 7).all() and (out[:, h * d:] == 7).all()


def test_decode_cache_past_4gb(gpu_lib):
    """Blocks beyond 2^32 bytes."""
    log("grouped decode big cache")
    pg = Paged(3, [200], 64, 8, 128)
    pg.fill()
    n_pages = 70000                                             # 4.6 GB of keys, as much of values
    big = moe.GroupedCache.empty(n_pages, 64, 8, 128)
    table = pg.table.copy()
    for j, p in enumerate(pg.table[0]):
        to = n_pages - 1 - 7 * j
        for x, y in zip(big._tensors()[:4], pg.cache._tensors()[:4]):
            x[to] = y[int(p)]
        table[0, j] = to
    q = _bf(pg.g.standard_normal((1, 16, 128)))
    want, _ = _decode(pg, q, [1])
    want = want.clone()
    pg.cache, pg.table = big, table
    got, _ = _decode(pg, q, [1])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    k, v = pg.draw(1)
    moe.grouped_cache_append(k, v, big, _i32(table), _i32([201]), _i32([0, 1]))
    torch.cuda.synchronize()
    page = n_pages - 1 - 7 * 3
    got = og.E4M3[big.k[page, :, 0, :, 8].cpu().numpy()].reshape(8, 128)
    e = big.k_scales[page, :, 0].cpu().numpy().astype(float) - 127
    assert np.allclose(got * 2.0 ** e[:, None], _np(k)[0], rtol=2.0 ** -4, atol=2.0 ** -3)


# ---- together -----------------------------------------------------------------------
def test_streams_and_graph_replays(gpu_lib):
    """On a stream of the caller's, and captured: each replay gives what the
    eager calls give on the inputs of that moment."""
    log("grouped streams and graphs")
    h, kv, d = 16, 2, 128
    pg = Paged(8, [400, 130], 32, kv, d)
    pg.fill()
    T = 2
    q0, k0, w, rot, _, g = _norm_case(T, h, kv, d, 64, "qk", seed=3)
    v0 = _bf(g.standard_normal((T, kv, d)))
    plan = moe.GroupedDecode(n_heads=h, n_kv_heads=kv, max_tokens=T, max_seqs=2)
    norm = moe.QKNormRope(T=T, n_heads=h, n_kv_heads=kv, rotary=64, backward=True)
    table, lens, cu = _i32(pg.table), _i32(pg.lens), _i32([0, 1, 2])
    ins = _draw(9, [80], [80], 4, 2, 64)
    att = moe.GroupedAttention(Tq=80, Tk=80, n_heads=4, n_kv_heads=2, head_dim=64, n_seqs=1, backward=True)
    acu = _i32([0, 80])
    dy = _bf(g.standard_normal((T, h, d))), _bf(g.standard_normal((T, kv, d)))

    def step(stream=None):
        q, k = norm(q0, k0, w["q"], w["k"], **rot, stream=stream)
        moe.grouped_cache_append(k, v0, pg.cache, table, lens, cu, stream=stream)
        o = plan(q, pg.cache, table, lens, cu, stream=stream)
        a, _ = att.forward(*ins[:3], acu, acu, stream=stream)
        return (o, a, *att.backward(ins[3], *ins[:3], acu, acu, stream=stream),
                *norm.backward(*dy, q0, k0, w["q"], w["k"], **rot, stream=stream), pg.cache.k, pg.cache.v_scales)

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        q0.copy_(_bf(g.standard_normal((T, h, d))))
        lens.copy_(_i32([400 - 31 * i, 130 - 7 * i]))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in outs[:-2]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, outs):
            assert torch.equal(x, y), f"replay {i}"


def test_decode_pieces_replayed_and_side_by_side(gpu_lib):
    """Cut caches in a captured call whose lengths change between replays, and
    two objects' calls on two streams at once."""
    log("grouped decode pieces in graphs and on two streams")
    h, kv, d = 16, 2, 64
    pg = Paged(12, [9000, 60, 3000], 16, kv, d)
    pg.fill()
    q = _bf(pg.g.standard_normal((3, h, d)))
    table, lens, cu = _i32(pg.table), _i32(pg.lens), _i32([0, 1, 2, 3])
    mk = lambda: moe.GroupedDecode(n_heads=h, n_kv_heads=kv, head_dim=d, max_tokens=3, max_seqs=3)
    plan, other = mk(), mk()
    call = lambda p, **k: p(q, pg.cache, table, lens, cu, **k)
    call(plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(plan)
    for n in ([9000, 60, 3000], [40, 1, 900], [8999, 33, 2], [0, 60, 3000], [9000, 60, 3000]):
        lens.copy_(_i32(n))
        out.zero_()
        for _ in range(2):
            graph.replay()
        want = call(other)
        torch.cuda.synchronize()
        assert torch.equal(out, want), n
    pg.lens = [9000, 60, 3000]
    _check_decode(pg, q, [1] * 3, out, None, fp32=1e-6, what="replayed")
    want = out.clone()
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip((plan, other), side):
            call(p, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(plan.out, want) and torch.equal(other.out, want)


def test_tokens_one_by_one_are_the_prompt(gpu_lib):
    """Norm, append and decode token by token over the 8-bit cache against the
    attention of the whole prompt over the cache's own values."""
    log("grouped decode steps against the prompt")
    n, h, kv, d = 70, 8, 2, 128
    g = np.random.default_rng(31)
    qkv = _bf(g.standard_normal((n, (h + 2 * kv) * d)))
    q = qkv[:, :h * d].unflatten(1, (h, d))
    k = qkv[:, h * d:(h + kv) * d].unflatten(1, (kv, d))
    v = qkv[:, (h + kv) * d:].unflatten(1, (kv, d))
    w = _bf(1 + 0.1 * g.standard_normal(d))
    angle = np.arange(n)[:, None] * 100.0 ** (-np.arange(64) / 64)
    rot = dict(cos=torch.from_numpy(np.cos(angle).astype(np.float32)).cuda(),
               sin=torch.from_numpy(np.sin(angle).astype(np.float32)).cuda())
    pg = Paged(1, [n], 16, kv, d)
    norm = moe.QKNormRope(T=n, n_heads=h, n_kv_heads=kv)
    step = moe.QKNormRope(T=1, n_heads=h, n_kv_heads=kv)
    plan = moe.GroupedDecode(n_heads=h, n_kv_heads=kv, max_tokens=1, max_seqs=1)
    table, cu = _i32(pg.table), _i32([0, 1])
    outs = []
    for t in range(n):
        q1, k1 = step(q[t:t + 1], k[t:t + 1], w, w, **rot, positions=_i32([t]))
        moe.grouped_cache_append(k1, v[t:t + 1], pg.cache, table, _i32([t + 1]), cu)
        outs.append(plan(q1, pg.cache, table, _i32([t + 1]), cu).clone())
    out = torch.cat(outs)
    qn, kn = norm(q, k, w, w, **rot, positions=torch.arange(n, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    c = pg.oracle()
    ck, cv = c.rows("k", pg.table[0], n), c.rows("v", pg.table[0], n)
    # a code is off by at most half a step, a second rounding under a larger
    # scale by another where it falls below the codes' normal range
    assert (np.abs(ck - _np(kn)) <= 2.0 ** -4 * np.abs(_np(kn)) + 2.0 ** -8 * np.abs(_np(kn)).max() / 224).all()
    a = moe.GroupedAttention(Tq=n, Tk=n, n_heads=h, n_kv_heads=kv, n_seqs=1)
    whole, _ = a(qn, _bf(ck), _bf(cv), _i32([0, n]), _i32([0, n]))
    torch.cuda.synchronize()
    ref = og.attention(_np(qn), ck, cv, visible(n, n, True), d ** -0.5)
    _inside(_np(whole), ref["out"], ref["out_tol"], "whole prompt")
    # the last step saw the very same codes (an earlier one may have seen its
    # own block under a smaller scale)
    _inside(_np(out[n - 1:]), ref["out"][n - 1:], ref["out_tol"][n - 1:], "last step")


def test_class_refusals(gpu_lib):
    q, k, v, do = _draw(1, [4], [4], 4, 2, 64)
    cu = _i32([0, 4])
    a = moe.GroupedAttention(Tq=4, Tk=4, n_heads=4, n_kv_heads=2, head_dim=64, n_seqs=1)
    for bad in ((q.float(), k, v, cu, cu), (q[:, :2], k, v, cu, cu), (q, k[:3], v, cu, cu), (q, k, v[:, :1], cu, cu),
                (q, k, v, cu.long(), cu), (q, k, v, _i32([0, 2, 4]), cu), (q.transpose(0, 1), k, v, cu, cu),
                (q, k, v.cpu(), cu, cu), (q, k.transpose(0, 1).contiguous().transpose(0, 1), v, cu, cu)):
        with pytest.raises(ValueError):
            a.forward(*bad)
    with pytest.raises(ValueError):
        a.backward(do, q, k, v, cu, cu)              # built without backward
    pg = Paged(1, [4], 16, 2, 64)
    plan = moe.GroupedDecode(n_heads=4, n_kv_heads=2, head_dim=64, max_tokens=2, max_seqs=1)
    other = moe.GroupedCache.empty(2, 16, 2, 128)
    good = [q[:1], pg.cache, _i32(pg.table), _i32([4]), _i32([0, 1])]
    for i, bad in ((0, q[:3]), (1, other), (2, _i32(pg.table).long()), (3, _i32([4, 4])), (4, _i32([0, 1, 1]))):
        with pytest.raises(ValueError):
            plan(*[bad if j == i else x for j, x in enumerate(good)])
    with pytest.raises(ValueError):
        plan(*good, tree_mask=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        moe.grouped_cache_append(k, v[:3], pg.cache, *good[2:])
    c = pg.cache
    for bad in ((c.k.view(-1), c.v, c.k_scales, c.v_scales), (c.k, c.v[:1], c.k_scales, c.v_scales),
                (c.k, c.v, c.k_scales.int(), c.v_scales), (c.k, c.v, c.k_scales, c.v_scales[..., :0])):
        with pytest.raises(ValueError):
            moe.GroupedCache(*bad)
    n = moe.QKNormRope(T=4, n_heads=4, n_kv_heads=2, head_dim=64, rotary=32)
    w, cs, pos = _bf(np.ones(64)), torch.ones((9, 16), device="cuda"), _i32([0, 1, 2, 3])
    for kw in (dict(w_q=w[:32]), dict(w_q=w.float()), dict(cos=cs), dict(cos=cs, sin=cs),
               dict(cos=cs, sin=cs[:, :8], positions=pos), dict(cos=cs, sin=cs, positions=pos[:3]),
               dict(cos=cs, sin=cs, positions=pos.long())):
        with pytest.raises(ValueError):
            n(q, k, **kw)
    with pytest.raises(ValueError):
        n(q, k[:3])


def test_no_decode_object_during_a_capture(gpu_lib):
    """Its workspace is cleared once, which a capture would only record."""
    g = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(g):
        x.add_(1)
        with pytest.raises(ValueError):
            moe.GroupedDecode(n_heads=4, n_kv_heads=2, head_dim=64, max_tokens=2, max_seqs=1)
    g.replay()
    torch.cuda.synchronize()
    assert (x == 1).all()


def test_layer_example(gpu_lib):
    """The example layer: prompt, decode steps, a drafted tree, gradients."""
    log("grouped layer example")
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "grouped_moe_layer.py")
    spec = importlib.util.spec_from_file_location("grouped_moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, tree, grads, y = mod.main(heads=16, kv_heads=2, hidden=512, prompt=130, steps=3)
    torch.cuda.synchronize()
    # a code is off by at most 2^-4 of its value, evenly spread (1 / sqrt(3) of
    # that in the mean square). Values carry it to the output as it is; keys to
    # scores of variance 1 and so to the weights, relatively. The two together
    # 0.051 of the output's norm, twice that for one short draw.
    assert worst < 2 * 2 ** 0.5 * 2.0 ** -4 / 3 ** 0.5
    # the same codes in other places: weights and result rounded on each side
    assert tree < 4 * 2.0 ** -8
    assert all(torch.isfinite(t.float()).all() for t in grads) and torch.isfinite(y.float()).all()
