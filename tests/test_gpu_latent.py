"""GPU parity of latent attention (expanded forward and backward, absorbed
decode over a paged cache, cache append) against the fp64 oracle. Every
element is compared, within the bound that the oracle derives for it from
the bf16 roundings of a kernel's matrix operands."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_amd as moe
from mixture_experts_layer_sigmoid_amd import _lib as L
from oracle import latent as ol
from tests.gpu_util import log

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int)


def _inside(got, want, tol, what):
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), what
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok], want[~ok]), what
    far = np.abs(got[ok] - want[ok]) - tol[ok]
    assert far.size == 0 or far.max() <= 0, f"{what}: {far.max():.3e} over its bound"


def _draw(seed, lens_q, lens_k, h, q_std=1.0):
    g = np.random.default_rng(seed)
    mk = lambda *s, std=1.0: _bf(g.standard_normal(s) * std)
    tq, tk = sum(lens_q), sum(lens_k)
    return (mk(tq, h, 192, std=q_std), mk(tk, h, 256), mk(tk, 64), mk(tq, h, 128))


def _reference(ins, lens_q, lens_k, causal, scale, backward):
    q, kv, kr, do = (_np(t) for t in ins)
    parts = []
    for a, b, c, d in zip(_cu(lens_q), _cu(lens_q)[1:], _cu(lens_k), _cu(lens_k)[1:]):
        r = ol.attention(q[a:b], kv[c:d], kr[c:d], causal, scale)
        if backward:
            r |= ol.attention_backward(do[a:b], q[a:b], kv[c:d], kr[c:d], causal, scale)
        parts.append(r)
    return {k: np.concatenate([p[k] for p in parts]) for k in parts[0]}


def _check_forward(out, lse, ref, what):
    _inside(_np(out), ref["out"], ref["out_tol"], what + " out")
    # scores are exact products summed in fp32
    _inside(_np(lse), ref["lse"], 1e-5 * (1 + np.abs(np.nan_to_num(ref["lse"], neginf=0))), what + " lse")


EXPANDED = [
    # heads, lens_q, lens_k, causal
    (1, [1], [1], True),
    (3, [1, 37, 130, 64, 65], [1, 37, 130, 64, 65], True),
    (2, [5, 0, 33], [70, 4, 0], False),         # a sequence without queries, one without keys
    (2, [100, 3], [30, 3], True),               # the first 70 queries see nothing
    (2, [31, 1], [129, 200], True),             # later pieces of longer prompts
    (1, [520, 513], [520, 640], True),          # the eight-wave tiles, cut at every edge
    (2, [700], [701], False),
]


@pytest.mark.parametrize("h,lens_q,lens_k,causal", EXPANDED)
def test_expanded_parity(gpu_lib, h, lens_q, lens_k, causal):
    log(f"latent expanded h={h} {lens_q} {lens_k} causal={causal}")
    ins = _draw(h + len(lens_q), lens_q, lens_k, h)
    ref = _reference(ins, lens_q, lens_k, causal, SCALE, True)
    a = moe.LatentAttention(Tq=sum(lens_q), Tk=sum(lens_k), n_heads=h, n_seqs=len(lens_q), causal=causal,
                            backward=True)
    cu = _i32(_cu(lens_q)), _i32(_cu(lens_k))
    out, lse = a.forward(*ins[:3], *cu)
    grads = a.backward(ins[3], *ins[:3], *cu)
    torch.cuda.synchronize()
    _check_forward(out, lse, ref, "forward")
    for name, t in zip(("dq", "dkv", "dk_rope"), grads):
        _inside(_np(t), ref[name], ref[name + "_tol"], name)
    first = [t.clone() for t in (out, lse, *grads)]
    a.forward(*ins[:3], *cu)
    a.backward(ins[3], *ins[:3], *cu)
    torch.cuda.synchronize()
    for x, y in zip(first, (a.out, a.lse, a.dq, a.dkv, a.dk_rope)):
        assert torch.equal(x, y), "two runs differ"


@pytest.mark.parametrize("scale,q_std", [(SCALE, 40.0), (1e-3, 1.0), (3.0, 1.0)])
def test_expanded_score_ranges(gpu_lib, scale, q_std):
    """Scores from nearly equal to hundreds apart."""
    log(f"latent expanded scale={scale} q_std={q_std}")
    lens = [90, 141]
    ins = _draw(5, lens, lens, 2, q_std)
    ref = _reference(ins, lens, lens, True, scale, False)
    a = moe.LatentAttention(Tq=231, Tk=231, n_heads=2, n_seqs=2, scale=scale)
    out, lse = a(*ins[:3], _i32(_cu(lens)), _i32(_cu(lens)))
    torch.cuda.synchronize()
    # fp32 scores of this size: their rounding moves weights by up to 2^-22 |s|
    big = np.abs(ref["lse"]).max()
    ref["out_tol"] += 2.0 ** -21 * big * 4
    _check_forward(out, lse, ref, f"scale {scale}")


def test_expanded_strides_outside_rows_and_hidden_nan(gpu_lib):
    """Slices of wider rows, rows outside every sequence (NaN in, untouched
    out), NaN in keys that the mask hides and in neighbouring sequences."""
    log("latent expanded strides")
    h, pad = 2, 9
    lens_q, lens_k = [40, 70], [50, 70]
    q, kv, kr, do = _draw(11, lens_q, lens_k, h)
    ref = _reference((q, kv, kr, do), lens_q, lens_k, True, SCALE, True)
    nan = float("nan")

    def wide(t, extra):
        rows, n = t.shape[0], t[0].numel()
        w = torch.full((rows + 2 * pad, n + extra), nan, dtype=torch.bfloat16, device="cuda")
        v = w[:, 8:8 + n].view(rows + 2 * pad, *t.shape[1:]) if extra == 0 else w[:, 8:8 + n].unflatten(1, t.shape[1:])
        v[pad:pad + rows] = t
        return v

    wq, wkv, wkr, wdo = wide(q, 64), wide(kv, 16), wide(kr, 512), wide(do, 8)
    cu_q, cu_k = _i32(_cu(lens_q) + pad), _i32(_cu(lens_k) + pad)
    tq, tk = wq.shape[0], wkv.shape[0]
    out = torch.full((tq, h * 128 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq, h), 7.0, device="cuda")
    dq = torch.full((tq, h * 192 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    dkv = torch.full((tk, h * 256 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    dkr = torch.full((tk, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.moe_mla_attn_bwd_workspace(tq, tk, h), dtype=torch.uint8, device="cuda")
    ld = lambda t: t.stride(0)
    L.moe_mla_attn_fwd(wq, ld(wq), wkv, ld(wkv), wkr, ld(wkr), 1, cu_q, cu_k, 2, tq, tk, h, 1, SCALE, out, ld(out),
                       lse)
    L.moe_mla_attn_bwd(wdo, ld(wdo), wq, ld(wq), wkv, ld(wkv), wkr, ld(wkr), 1, out, ld(out), lse, cu_q, cu_k, 2, tq,
                       tk, h, 1, SCALE, dq, ld(dq), dkv, ld(dkv), dkr, ld(dkr), ws)
    torch.cuda.synchronize()
    held_q, held_k = slice(pad, pad + 110), slice(pad, pad + 120)
    _check_forward(out[held_q, :h * 128].unflatten(1, (h, 128)), lse[held_q], ref, "strided")
    _inside(_np(dq[held_q, :h * 192].unflatten(1, (h, 192))), ref["dq"], ref["dq_tol"], "dq")
    _inside(_np(dkv[held_k, :h * 256].unflatten(1, (h, 256))), ref["dkv"], ref["dkv_tol"], "dkv")
    _inside(_np(dkr[held_k, :64]), ref["dk_rope"], ref["dk_rope_tol"], "dk_rope")
    for t, n in ((out, h * 128), (lse, h), (dq, h * 192)):
        assert (t[:pad] == 7).all() and (t[pad + 110:] == 7).all() and (t[:, n:] == 7).all()
    for t, n in ((dkv, h * 256), (dkr, 64)):
        assert (t[:pad] == 7).all() and (t[pad + 120:] == 7).all() and (t[:, n:] == 7).all()
    # the last key's key part is hidden from every query but the last
    kv2 = kv.clone()
    kv2[49, :, :128] = nan
    a = moe.LatentAttention(Tq=110, Tk=120, n_heads=h, n_seqs=2)
    o2, _ = a(q, kv2, kr, _i32(_cu(lens_q)), _i32(_cu(lens_k)))
    torch.cuda.synchronize()
    rest = np.r_[0:39, 40:110]
    assert np.isnan(_np(o2)[39]).all()
    _inside(_np(o2)[rest], ref["out"][rest], ref["out_tol"][rest], "beside NaN keys")


def test_expanded_rows_past_4gb(gpu_lib):
    """Row offsets beyond 2^32 bytes."""
    log("latent expanded wide rows")
    n, ld = 9000, 1 << 18
    buf = torch.empty((n, ld), dtype=torch.bfloat16, device="cuda")        # 4.7 GB
    g = np.random.default_rng(2)
    q, kv, kr = _bf(g.standard_normal((3, 1, 192))), _bf(g.standard_normal((n, 1, 256))), _bf(g.standard_normal((n, 64)))
    wide = buf[:, :256].unflatten(1, (1, 256))
    wide.copy_(kv)
    a = moe.LatentAttention(Tq=3, Tk=n, n_heads=1, n_seqs=1)
    out, lse = a(q, wide, kr, _i32([0, 3]), _i32([0, n]))
    torch.cuda.synchronize()
    ref = ol.attention(_np(q), _np(kv), _np(kr), True, SCALE)
    _check_forward(out, lse, ref, "wide rows")


class Paged:
    """Requests' cache rows scattered over pages; everything else is NaN."""

    def __init__(self, seed, lens, page, h, spare=2):
        g = np.random.default_rng(seed)
        self.lens, self.page = lens, page
        need = [-(-n // page) for n in lens]
        ids = g.permutation(sum(need) + spare)
        cache = np.full((sum(need) + spare, page, 576), np.nan, np.float32)
        self.table = np.full((len(lens), max(1, max(need))), 2 ** 30, np.int64)     # unused entries: no page
        self.rows, at = [], 0
        for b, n in enumerate(lens):
            rows = np.asarray(torch.from_numpy(g.standard_normal((n, 576)).astype(np.float32)).bfloat16().float())
            self.rows.append(rows.astype(np.float64))
            for j in range(need[b]):
                self.table[b, j] = ids[at]
                part = rows[j * page:(j + 1) * page]
                cache[ids[at], :len(part)] = part
                at += 1
        self.cache = _bf(cache)
        self.w = _bf(g.standard_normal((h, 256, 512)) / 512 ** 0.5)

    def put(self, b, j, values):
        self.rows[b][j] = values
        self.cache[self.table[b, j // self.page], j % self.page] = _bf(np.asarray(values)[None])[0]


def _decode(pg, q, nq, tree=None, scale=SCALE, stream=None, plan=None):
    """nq: new tokens per request."""
    h = q.shape[1]
    plan = plan or moe.LatentDecode(pg.w, max_tokens=q.shape[0], max_seqs=len(nq), scale=scale)
    lse = torch.full((q.shape[0], h), 7.0, device="cuda")
    out = plan(q, pg.cache, _i32(pg.table), _i32(pg.lens), _i32(_cu(nq)),
               None if tree is None else torch.tensor(tree, dtype=torch.int64, device="cuda"), lse=lse, stream=stream)
    return out, lse


def _check_decode(pg, q, nq, out, lse, tree=None, scale=SCALE, what=""):
    qn, w, at = _np(q), _np(pg.w), _cu(nq)
    for b in range(len(nq)):
        s = slice(at[b], at[b + 1])
        if s.start == s.stop:
            continue
        words = None if tree is None else [t & (2 ** 64 - 1) for t in tree[s]]
        ref = ol.cached(qn[s], w, pg.rows[b], scale, words)
        _inside(_np(out[s]), ref["out"], ref["out_tol"], f"{what} out of request {b}")
        _inside(_np(lse[s]), ref["lse"], ref["lse_tol"], f"{what} lse of request {b}")


DECODE = [
    # heads, page, lens, new tokens
    (1, 16, [1], [1]),
    (16, 64, [531, 64, 65, 1, 63], [1, 1, 1, 1, 1]),
    (5, 1, [3, 130], [1, 2]),
    (16, 7, [200, 9, 70], [3, 0, 4]),               # pages end inside a tile, a request without new tokens
    (40, 100, [128, 300], [1, 1]),                  # 64-row tiles
    (128, 32, [190, 66], [1, 2]),                   # two row tiles a request: taken in step
    (24, 64, [3, 2], [5, 2]),                       # more new tokens than the cache holds: the first see nothing
    (3, 16, [700], [90]),                           # a later piece of a prompt
    (16, 64, [0, 12, 0], [1, 1, 2]),                # empty requests
]


@pytest.mark.parametrize("h,page,lens,nq", DECODE)
def test_decode_parity(gpu_lib, h, page, lens, nq):
    log(f"latent decode h={h} page={page} lens={lens} nq={nq}")
    pg = Paged(h + page, lens, page, h)
    q = _draw(h, [sum(nq)], [1], h)[0]
    out, lse = _decode(pg, q, nq)
    torch.cuda.synchronize()
    # requests with fewer rows than new tokens: the oracle sees what is there
    _check_decode(pg, q, nq, out, lse, what="decode")
    one, _ = out.clone(), None
    out2, _ = _decode(pg, q, nq)
    torch.cuda.synchronize()
    assert torch.equal(one, out2), "two runs differ"


def test_decode_many_requests_and_long_ones(gpu_lib):
    """More requests than a wave's lanes; caches cut into pieces."""
    log("latent decode many")
    g = np.random.default_rng(0)
    lens = [int(v) for v in g.integers(0, 90, 130)]
    lens[7], lens[100] = 9000, 4097
    pg = Paged(1, lens, 16, 2)
    q = _draw(3, [130], [1], 2)[0]
    out, lse = _decode(pg, q, [1] * 130)
    torch.cuda.synchronize()
    _check_decode(pg, q, [1] * 130, out, lse, what="many")


@pytest.mark.parametrize("lens", [[5888], [5889], [6337, 1]])
def test_decode_runs_of_one_and_of_two_tiles(gpu_lib, lens):
    """Where the cut changes: 92 token tiles (runs of one), 93 and 100 (runs of two, the last of one)."""
    log(f"latent decode runs {lens}")
    nq = [2] + [1] * (len(lens) - 1)
    pg = Paged(5, lens, 32, 3)
    q = _draw(5, [sum(nq)], [1], 3)[0]
    out, lse = _decode(pg, q, nq)
    torch.cuda.synchronize()
    _check_decode(pg, q, nq, out, lse, what="runs")


@pytest.mark.parametrize("h,nq,lens", [(16, 7, [100, 7, 64]), (4, 48, [48, 75]), (128, 5, [61])])
def test_decode_trees(gpu_lib, h, nq, lens):
    log(f"latent tree h={h} nq={nq}")
    g = np.random.default_rng(nq)
    pg = Paged(nq, lens, 16, h)
    n = len(lens)
    q = _draw(h, [nq * n], [1], h)[0]
    tree = []
    for _ in range(n):
        m = []
        for i in range(nq):
            p = int(g.integers(-1, i)) if i else -1
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        tree += m
    tree[nq // 2] = 0                               # a token that sees no new token, itself included
    out, lse = _decode(pg, q, [nq] * n, tree)
    torch.cuda.synchronize()
    _check_decode(pg, q, [nq] * n, out, lse, tree, what="tree")


def test_decode_tree_of_64_and_words_with_the_top_bit(gpu_lib):
    log("latent tree 64")
    pg = Paged(4, [64, 130], 64, 1)
    q = _draw(4, [128], [1], 1)[0]
    tree = [(1 << i) | (1 << 63) if i % 3 else 0 for i in range(64)] * 2
    signed = [t - 2 ** 64 if t >> 63 else t for t in tree]
    out, lse = _decode(pg, q, [64, 64], signed)
    torch.cuda.synchronize()
    _check_decode(pg, q, [64, 64], out, lse, tree, what="tree 64")


def test_decode_hidden_rows_may_hold_anything(gpu_lib):
    """Infinities and NaN in drafted rows that a token does not see."""
    log("latent hidden rows")
    pg = Paged(9, [70], 16, 4)
    q = _draw(9, [4], [1], 4)[0]
    tree = [0b0001, 0b0011, 0b0101, 0b1001]          # 1, 2 and 3 are siblings
    bad = np.full(576, np.nan)
    bad[::3], bad[1::3] = np.inf, -np.inf
    clean = _np(_decode(pg, q, [4], tree)[0])
    pg.put(0, 68, bad)                               # drafted token 2
    out, lse = _decode(pg, q, [4], tree)
    torch.cuda.synchronize()
    got = _np(out)
    for i in (0, 1, 3):
        assert np.array_equal(got[i], clean[i]), i
    assert np.isnan(got[2]).all()
    # the causal order hides later tokens alike
    pg2 = Paged(9, [70], 16, 4)
    clean = _np(_decode(pg2, q, [4])[0])
    pg2.put(0, 69, bad)
    got = _np(_decode(pg2, q, [4])[0])
    assert np.array_equal(got[:3], clean[:3]) and np.isnan(got[3]).all()


def test_decode_score_ranges(gpu_lib):
    log("latent decode score ranges")
    pg = Paged(6, [300, 1000], 64, 3)
    q = (_draw(6, [2], [1], 3)[0].float() * 20).bfloat16()
    for scale in (1e-3, SCALE):
        out, lse = _decode(pg, q, [1, 1], scale=scale)
        torch.cuda.synchronize()
        _check_decode(pg, q, [1, 1], out, lse, scale=scale, what=f"scale {scale}")


def test_decode_rows_past_4gb(gpu_lib):
    """Cache rows beyond 2^32 bytes."""
    log("latent decode big cache")
    page, n_pages = 64, 60000                        # 4.4 GB
    pg = Paged(3, [200], page, 16)
    big = torch.empty((n_pages, page, 576), dtype=torch.bfloat16, device="cuda")
    used = [int(x) for x in pg.table[0]]
    for j, p in enumerate(used):
        big[n_pages - 1 - 7 * j] = pg.cache[p]
        pg.table[0, j] = n_pages - 1 - 7 * j
    pg.cache = big
    q = _draw(3, [1], [1], 16)[0]
    out, lse = _decode(pg, q, [1])
    torch.cuda.synchronize()
    _check_decode(pg, q, [1], out, lse, what="big cache")


def test_streams_and_graph_replays(gpu_lib):
    """On a stream of the caller's, and captured: each replay gives what the
    eager call gives on the inputs of that moment."""
    log("latent streams and graphs")
    pg = Paged(8, [400, 130], 32, 16)
    q = _draw(8, [2], [1], 16)[0]
    plan = moe.LatentDecode(pg.w, max_tokens=2, max_seqs=2)
    table, lens, cu = _i32(pg.table), _i32(pg.lens), _i32([0, 1, 2])
    att_in = _draw(9, [80], [80], 2)
    att = moe.LatentAttention(Tq=80, Tk=80, n_heads=2, n_seqs=1, backward=True)
    acu = _i32([0, 80])
    side = torch.cuda.Stream()

    def step(stream=None):
        o = plan(q, pg.cache, table, lens, cu, stream=stream)
        a, _ = att.forward(*att_in[:3], acu, acu, stream=stream)
        return (o, a, *att.backward(att_in[3], *att_in[:3], acu, acu, stream=stream))

    side.wait_stream(torch.cuda.current_stream())
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    got = step(side)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        q.copy_(_draw(20 + i, [2], [1], 16)[0])
        lens.copy_(_i32([400 - 31 * i, 130 - 7 * i]))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, outs):
            assert torch.equal(x, y), f"replay {i}"


@pytest.mark.parametrize("T,h,interleaved", [(1, 1, True), (67, 16, True), (130, 5, False)])
def test_append_parity(gpu_lib, T, h, interleaved):
    log(f"latent append T={T} h={h} interleaved={interleaved}")
    g = np.random.default_rng(T)
    wide = _bf(g.standard_normal((T, 640)) * 3)
    kv_a = wide[:, 32:608]
    w = _bf(1 + 0.1 * g.standard_normal(512))
    q = _bf(g.standard_normal((T, h, 192)))
    angle = g.uniform(-3, 3, (50, 32))
    cos, sin = (torch.from_numpy(f(angle).astype(np.float32)).cuda() for f in (np.cos, np.sin))
    pos = g.integers(0, 50, T)
    pos[0] = 70                                      # past the table: its last row
    slots = g.permutation(T + 9)[:T]
    slots[T // 2] = -1 if T > 1 else slots[0]
    cache = torch.full((1, T + 9, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty_like(q)
    moe.latent_cache_append(kv_a, cache, torch.tensor(slots, device="cuda"), norm_weight=w, eps=1e-5, cos=cos, sin=sin,
                            positions=_i32(pos), q=q, q_out=q_out, interleaved=interleaved)
    torch.cuda.synchronize()
    ang = angle[np.minimum(pos, 49)]
    x = _np(kv_a)
    rows = np.concatenate([ol.cache_row(x, _np(w), 1e-5), ol.rotate(x[:, 512:], ang, interleaved)], 1)
    got = _np(cache)[0]
    held = slots >= 0
    # one rounding; cos and sin are fp32
    tol = ol.SLACK * ol.U * np.abs(rows) + 1e-5
    _inside(got[slots[held]], rows[held], tol[held], "cache rows")
    untouched = np.setdiff1d(np.arange(T + 9), slots)
    assert (got[untouched] == 5).all()
    qn = _np(q)
    want = np.concatenate([qn[..., :128], ol.rotate(qn[..., 128:], ang[:, None], interleaved)], 2)
    _inside(_np(q_out), want, ol.SLACK * ol.U * np.abs(want) + 1e-5, "q")
    assert torch.equal(q_out[..., :128], q[..., :128])
    inplace = q.clone()
    moe.latent_cache_append(kv_a, cache, torch.tensor(slots, device="cuda"), norm_weight=w, eps=1e-5, cos=cos, sin=sin,
                            positions=_i32(pos), q=inplace, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(inplace, q_out)
    # without norm weight, rotation and queries: the rows themselves
    moe.latent_cache_append(kv_a, cache, torch.tensor(slots, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(cache[0][torch.tensor(slots[held], device="cuda")], kv_a[torch.tensor(held, device="cuda")])


def test_class_refusals(gpu_lib):
    q, kv, kr, do = _draw(1, [4], [4], 2)
    cu = _i32([0, 4])
    a = moe.LatentAttention(Tq=4, Tk=4, n_heads=2, n_seqs=1)
    for bad in ((q.float(), kv, kr, cu, cu), (q[:, :1], kv, kr, cu, cu), (q, kv[:3], kr, cu, cu),
                (q, kv, kr, cu.long(), cu), (q, kv, kr, _i32([0, 2, 4]), cu), (q.transpose(0, 1), kv, kr, cu, cu),
                (q, kv, kr.cpu(), cu, cu)):
        with pytest.raises(ValueError):
            a.forward(*bad)
    with pytest.raises(ValueError):
        a.backward(do, q, kv, kr, cu, cu)            # built without backward
    pg = Paged(1, [4], 16, 2)
    plan = moe.LatentDecode(pg.w, max_tokens=2, max_seqs=1)
    good = [q[:1], pg.cache, _i32(pg.table), _i32([4]), _i32([0, 1])]
    for i, bad in ((0, q[:3]), (1, pg.cache[..., :512]), (2, _i32(pg.table).long()), (3, _i32([4, 4])),
                   (4, _i32([0, 1, 1]))):
        with pytest.raises(ValueError):
            plan(*[bad if j == i else x for j, x in enumerate(good)])
    with pytest.raises(ValueError):
        moe.LatentDecode(pg.w[:, :128], max_tokens=1, max_seqs=1)
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    rows = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(kv_a=rows[:, :512]), dict(slots=slots.int()), dict(cos=torch.zeros(2, 32, device="cuda")),
               dict(norm_weight=rows[0, :500])):
        args = {"kv_a": rows, "cache": pg.cache, "slots": slots} | kw
        with pytest.raises(ValueError):
            moe.latent_cache_append(args.pop("kv_a"), args.pop("cache"), args.pop("slots"), **args)


def test_expand_is_the_projection(gpu_lib):
    log("latent expand")
    g = np.random.default_rng(4)
    c, w = _bf(g.standard_normal((77, 512))), _bf(g.standard_normal((3, 256, 512)) / 512 ** 0.5)
    kv = moe.LatentExpand(w, max_tokens=77)(c)
    torch.cuda.synchronize()
    want = np.einsum("tr,hdr->thd", _np(c), _np(w))
    # exact products summed in fp32, one rounding
    tol = ol.U * np.abs(want) + 2.0 ** -18 * np.einsum("tr,hdr->thd", np.abs(_np(c)), np.abs(_np(w)))
    _inside(_np(kv), want, tol, "expand")


def test_layer_example(gpu_lib):
    """The example layer: prompt, decode steps, a drafted tree, gradients."""
    log("latent layer example")
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_moe_layer.py")
    spec = importlib.util.spec_from_file_location("latent_moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, tree, grads, y = mod.main(heads=16, hidden=512, prompt=130, steps=3)
    torch.cuda.synchronize()
    # expanded: kv and the weights rounded; absorbed: q_lat and the weights
    # rounded; both outputs rounded. Relative to the output's norm each counts
    # at most u = 2^-8 in the root mean square (a rounding's is below u / 1.7).
    assert worst < 6 * 2.0 ** -8
    # the same rows under other tiles: weights and result rounded on each side
    assert tree < 4 * 2.0 ** -8
    assert all(torch.isfinite(t.float()).all() for t in grads) and torch.isfinite(y.float()).all()
