"""Grouped-query attention at the ends of what its calls take."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_amd as moe
from mixture_experts_layer_sigmoid_amd import _lib as L
from oracle import grouped as og
from tests.gpu_util import log
from tests.test_gpu_grouped import Paged, _bf, _check_decode, _cu, _i32, _inside, _norm_case, _np

pytestmark = pytest.mark.gpu


# ---- norms and rotation ---------------------------------------------------------
@pytest.mark.parametrize("T,h,kv,d,rotary,il,weights", [
    (4500, 21, 3, 128, 128, False, "qk"),   # several rounds of a token's one wave, key heads from its middle on
    (4200, 36, 6, 64, 32, True, "qk"),
    (4097, 10, 5, 128, 64, True, "k"),       # one token more than the backward's waves
    (1100, 40, 8, 128, 96, False, "q"),     # two waves a token, three rounds
])
def test_norm_of_many_tokens(gpu_lib, T, h, kv, d, rotary, il, weights):
    """Every row of both directions, also ones of large and small values (a
    head's sum of squares stays below fp32's largest number)."""
    log(f"qk norm T={T} h={h}/{kv} D={d} rotary={rotary} interleaved={il} weights={weights}")
    q, k, w, rot, angle, g = _norm_case(T, h, kv, d, rotary, weights)
    q[4], k[4], q[5], k[T - 1] = 1e18, -1e18, 1e-30, 0
    eps = 1e-6
    plan = moe.QKNormRope(T=T, n_heads=h, n_kv_heads=kv, head_dim=d, rotary=rotary, interleaved=il, eps=eps,
                          backward=True)
    for t in (plan.q, plan.k, plan.dq, plan.dk):
        t.fill_(float("nan"))
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


# ---- packed sequences -------------------------------------------------------------
@pytest.mark.parametrize("h,kv,d,lens_q", [(64, 8, 128, [96]), (16, 1, 64, [60, 0, 41]), (4, 4, 128, [7]),
                                           (96, 4, 64, [1500, 2])])
def test_attention_without_any_key(gpu_lib, h, kv, d, lens_q):
    """Sequences that all lack keys: out and dq 0, lse -inf, whichever number of
    rows there is (none of them could be split over keys)."""
    log(f"grouped attention without keys {h}/{kv} D={d} {lens_q}")
    tq = sum(lens_q)
    g = np.random.default_rng(tq)
    q, do = _bf(g.standard_normal((tq, h, d))), _bf(g.standard_normal((tq, h, d)))
    k = torch.empty((0, kv, d), dtype=torch.bfloat16, device="cuda")
    cu_q, cu_k = _i32(_cu(lens_q)), _i32([0] * (len(lens_q) + 1))
    for tk in (0, 5000):                                # buffers of no keys, and of some that the call leaves
        a = moe.GroupedAttention(Tq=tq, Tk=tk, n_heads=h, n_kv_heads=kv, head_dim=d, n_seqs=len(lens_q), backward=True)
        for t in (a.out, a.lse, a.dq, a.dk, a.dv):
            t.fill_(7.0)
        a.ws.fill_(255)
        out, lse = a.forward(q, k, k, cu_q, cu_k)
        dq, dk, dv = a.backward(do, q, k, k, cu_q, cu_k)
        torch.cuda.synchronize()
        assert not out.any() and not dq.any() and torch.isneginf(lse).all()
        assert dk.shape == dv.shape == (0, kv, d)
        assert (a.dk == 7).all() and (a.dv == 7).all()


# ---- the cache ----------------------------------------------------------------------
@pytest.mark.parametrize("d,page", [(128, 32), (64, 16)])
def test_append_after_going_back(gpu_lib, d, page):
    """Drafted tokens are written, rejected and written over, bit for bit: back
    into a block it keeps the scale that they had raised, back to its first
    position it gets one of its own."""
    log(f"grouped append after going back D={d}")
    pg = Paged(d, [60, 60], page, 2, d)
    want = pg.oracle()
    sizes = {"prompt": 1.0, "draft": 2.0 ** 9, "next": 2.0 ** -3}
    #        what, lens after it, new tokens
    steps = [("prompt", [21, 32], [21, 32]), ("draft", [29, 40], [8, 8]),      # 5 and 0 tokens before them
             ("next", [24, 33], [3, 1]), ("draft", [40, 41], [16, 8]), ("next", [32, 34], [8, 1]),
             ("next", [33, 48], [1, 14]), ("next", [17, 20], [4, 4])]
    scales = []
    for what, lens, new in steps:
        k, v = (x * sizes[what] for x in pg.draw(sum(new)))
        pg.append(lens, new, k, v)
        torch.cuda.synchronize()
        cu = _cu(new)
        for name, x in (("k", k), ("v", v)):
            for b in range(2):
                want.append(name, x[cu[b]:cu[b + 1]].double().cpu().numpy(), pg.table[b], lens[b])
        got = pg.oracle()
        for name in "kv":
            assert np.array_equal(got.codes[name], want.codes[name]), (what, name)
            assert np.array_equal(got.e[name], want.e[name]), (what, name)
        at = lambda b, blk: got.e["k"][pg.table[b][blk * 16 // page], :, blk * 16 % page // 16]
        scales.append((at(0, 1), at(1, 2)))
    prompt, draft, after = scales[:3]
    assert (draft[0] > prompt[0]).all()
    assert np.array_equal(after[0], draft[0]), "5 earlier tokens: kept"
    assert (after[1] < draft[1]).all(), "no earlier token: its own"


# ---- decode -------------------------------------------------------------------------
@pytest.mark.parametrize("lens,h,kv,d", [
    # 160 segments, two a unit at once: 4 requests in 8 to 20 pieces
    ([12000, 3000, 6000, 4500] + [5 * i + 1 for i in range(16)], 16, 8, 64),
    # 256 segments, room for more: half of them in 2 and 3 pieces
    ([1, 3000, 33, 5000] * 16, 16, 4, 128),
    # 800 segments: 5 requests in 7 to 24 pieces, the short ones last
    ([8000, 20000, 9, 70] + [3 * i % 90 for i in range(92)] + [8000, 6001, 7333, 31], 8, 8, 64),
    # 800 segments, 480 of them in 2 pieces: 960 of the workspace's 1024 places
    ([1040] * 60 + [1] * 40, 8, 8, 64),
])
def test_decode_cut_caches_of_many_requests(gpu_lib, lens, h, kv, d):
    """Every rule for the number of pieces with caches that are cut; nothing is
    written behind the workspace, and its counters are zero again."""
    B = len(lens)
    log(f"grouped decode {B} requests, {sum(lens)} tokens, {h}/{kv} D={d}")
    pg = Paged(B, lens, 32, kv, d)
    pg.fill()
    q = _bf(pg.g.standard_normal((B, h, d)))
    need = L.moe_gqa_decode_workspace(d)
    buf = torch.full((need + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[:need]
    ws.zero_()
    out = torch.full((B, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, h), 7.0, device="cuda")
    table, lens_d, cu = _i32(pg.table), _i32(lens), _i32(range(B + 1))
    call = lambda: L.moe_gqa_decode(q, h * d, 1, *pg.cache._tensors(), table, table.shape[1], lens_d, cu, None, B, B, h,
                                    kv, d, d ** -0.5, out, h * d, lse, ws)
    call()
    torch.cuda.synchronize()
    assert (buf[need:] == 0xA5).all(), "behind the workspace"
    assert not ws[:2 * 1024 * 4].any(), "the counters, at its start"
    # fp32 sums of up to 20000 weights: 2^-24 sqrt(n) of their size and less
    _check_decode(pg, q, [1] * B, out, lse, fp32=1e-6, what="cut caches")
    first = out.clone()
    for _ in range(3):
        out.fill_(7.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, first), "two runs differ"


def test_decode_more_drafts_than_a_mask_has_bits(gpu_lib):
    """New tokens from the 65th on are hidden from all, and see what their mask
    says of the first 64."""
    log("grouped decode 70 drafts")
    nq, h, kv, d = [70, 66], 4, 2, 64
    pg = Paged(4, [100, 66], 16, kv, d)
    pg.fill()
    q = _bf(pg.g.standard_normal((sum(nq), h, d)))
    words = torch.from_numpy(pg.g.integers(-2 ** 63, 2 ** 63, sum(nq))).cuda()
    plan = moe.GroupedDecode(n_heads=h, n_kv_heads=kv, head_dim=d, max_tokens=sum(nq), max_seqs=2)
    lse = torch.empty((sum(nq), h), device="cuda")
    out = plan(q, pg.cache, _i32(pg.table), _i32(pg.lens), _i32(_cu(nq)), words, lse)
    torch.cuda.synchronize()
    _check_decode(pg, q, nq, out, lse, tree=words)


def test_decode_lengths_beyond_the_table(gpu_lib):
    """A length is cut to what the request's pages hold."""
    log("grouped decode lengths beyond the table")
    h, kv, d = 8, 2, 128
    pg = Paged(6, [64, 64], 16, kv, d)
    pg.fill()
    q = _bf(pg.g.standard_normal((4, h, d)))
    plan = moe.GroupedDecode(n_heads=h, n_kv_heads=kv, head_dim=d, max_tokens=4, max_seqs=2)
    out = plan(q, pg.cache, _i32(pg.table), _i32([2 ** 31 - 1, 65]), _i32([0, 3, 4]))
    torch.cuda.synchronize()
    _check_decode(pg, q, [3, 1], out, None)
