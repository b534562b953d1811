"""Host-side argument checks of the grouped-query attention entry points and
classes (no call here reaches the device)."""
import pytest
import torch

from mixture_experts_layer_sigmoid_amd import _lib as L
from mixture_experts_layer_sigmoid_amd import gqa

OK, INVALID, UNSUPPORTED, ALIGN, WS = 0, -1, -2, -3, -4
A = 0x10000  # aligned fake device address (never dereferenced)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _norm(lib, **k):
    a = dict(q=A, q_ld=256, k=A, k_ld=128, fmt=1, wq=A, wk=A, eps=1e-6, cos=A, sin=A, max_pos=4, pos=A, rot=128, il=0,
             T=4, h=2, kv=1, d=128, qo=A, qo_ld=256, ko=A, ko_ld=128) | k
    return lib.moe_qk_norm_rope(*a.values(), None)


def _norm_bwd(lib, **k):
    a = dict(dqo=A, dqo_ld=256, dko=A, dko_ld=128, q=A, q_ld=256, k=A, k_ld=128, fmt=1, wq=A, wk=A, eps=1e-6, cos=A,
             sin=A, max_pos=4, pos=A, rot=128, il=0, T=4, h=2, kv=1, d=128, dq=A, dq_ld=256, dk=A, dk_ld=128, dwq=A,
             dwk=A, ws=A, wsb=BIG) | k
    return lib.moe_qk_norm_rope_bwd(*a.values(), None)


def _fwd(lib, **k):
    a = dict(q=A, q_ld=256, k=A, k_ld=128, v=A, v_ld=128, fmt=1, cq=A, ck=A, B=1, Tq=4, Tk=4, h=2, kv=1, d=128,
             causal=1, scale=1.0, out=A, out_ld=256, lse=None, ws=A, wsb=BIG) | k
    return lib.moe_gqa_attn_fwd(*a.values(), None)


def _bwd(lib, **k):
    a = dict(do=A, do_ld=256, q=A, q_ld=256, k=A, k_ld=128, v=A, v_ld=128, fmt=1, out=A, out_ld=256, lse=A, cq=A, ck=A,
             B=1, Tq=4, Tk=4, h=2, kv=1, d=128, causal=1, scale=1.0, dq=A, dq_ld=256, dk=A, dk_ld=128, dv=A, dv_ld=128,
             ws=A, wsb=BIG) | k
    return lib.moe_gqa_attn_bwd(*a.values(), None)


def _app(lib, **k):
    a = dict(k=A, k_ld=128, v=A, v_ld=128, fmt=1, kc=A, vc=A, ks=A, vs=A, page=16, pages=8, table=A, max_pages=4, lens=A,
             cu=A, B=1, T=4, kv=1, d=128) | k
    return lib.moe_gqa_append(*a.values(), None)


def _dec(lib, **k):
    a = dict(q=A, q_ld=256, fmt=1, kc=A, vc=A, ks=A, vs=A, page=16, pages=8, table=A, max_pages=4, lens=A, cu=A,
             tree=None, B=1, T=4, h=2, kv=1, d=128, scale=1.0, out=A, out_ld=256, lse=None, ws=A, wsb=BIG) | k
    return lib.moe_gqa_decode(*a.values(), None)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_norm_refusals(lib, call):
    for bad in (dict(T=-1), dict(T=(1 << 23) + 1), dict(h=0), dict(h=1025), dict(kv=0), dict(eps=-1.0), dict(eps=2.0),
                dict(eps=float("nan")), dict(cos=None), dict(sin=None), dict(pos=None), dict(max_pos=0), dict(rot=0),
                dict(rot=8), dict(rot=24), dict(rot=144), dict(il=2), dict(q_ld=248), dict(k_ld=120),
                dict(q_ld=(1 << 23) + 8), dict(q=None), dict(k=None)):
        assert call(lib, **bad) == INVALID, bad
    for bad in (dict(fmt=0), dict(d=96), dict(d=256)):
        assert call(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q_ld=260), dict(k_ld=132), dict(q=A + 8), dict(k=A + 2), dict(wq=A + 8), dict(cos=A + 4)):
        assert call(lib, **bad) == ALIGN, bad
    assert b"moe_qk_norm_rope" in lib.moe_last_error()


def test_norm_forward_refusals(lib):
    assert _norm(lib, qo_ld=512) == INVALID, "in place with another stride"
    assert _norm(lib, qo=None) == INVALID and _norm(lib, ko=None) == INVALID
    assert _norm(lib, T=0, q=None, k=None, qo=None, ko=None, pos=None) == OK


def test_norm_backward_refusals(lib):
    need = lib.moe_qk_norm_rope_bwd_workspace(128)
    assert need > 0 and lib.moe_qk_norm_rope_bwd_workspace(96) == 0
    assert _norm_bwd(lib, wsb=need - 1) == WS and _norm_bwd(lib, ws=None) == WS
    for bad in (dict(dqo=None), dict(dko=None), dict(dq=None), dict(dk=None), dict(dwq=None), dict(dwk=None),
                dict(dq_ld=248), dict(dko_ld=120)):
        assert _norm_bwd(lib, **bad) == INVALID, bad
    assert _norm_bwd(lib, ws=A + 8) == ALIGN
    assert _norm_bwd(lib, T=0, wq=None, wk=None, ws=None, q=None, k=None, dqo=None, dko=None, dq=None, dk=None) == OK


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_attention_refusals(lib, call):
    for bad in (dict(B=-1), dict(Tq=-1), dict(h=0), dict(h=1025), dict(kv=0), dict(kv=3), dict(h=3, kv=2),
                dict(causal=2), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0),
                dict(scale=3e38), dict(q_ld=248), dict(k_ld=120), dict(v_ld=120), dict(out_ld=248),
                dict(q_ld=(1 << 23) + 8), dict(Tq=1 << 28), dict(Tq=1 << 27, h=2), dict(B=1 << 22, h=2), dict(q=None),
                dict(k=None), dict(v=None), dict(cq=None), dict(ck=None), dict(out=None)):
        assert call(lib, **bad) == INVALID, bad
    for bad in (dict(fmt=0), dict(fmt=2), dict(d=96), dict(d=192)):
        assert call(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q_ld=260), dict(k_ld=132), dict(v_ld=132), dict(out_ld=260), dict(q=A + 8), dict(k=A + 2),
                dict(v=A + 8), dict(out=A + 8)):
        assert call(lib, **bad) == ALIGN, bad
    assert b"moe_gqa_attn" in lib.moe_last_error()
    assert call(lib, B=0) == OK
    assert call(lib, Tq=0, Tk=0, q=None, k=None, v=None, out=None) == OK


def test_attention_forward_workspace(lib):
    need = lib.moe_gqa_attn_fwd_workspace(4, 2, 128)
    assert _fwd(lib, wsb=need - 1) == WS and _fwd(lib, ws=None) == WS and _fwd(lib, ws=A + 8) == ALIGN
    for bad in ((-1, 2, 128), (4, 0, 128), (4, 2, 96), (0, 2, 64)):
        assert lib.moe_gqa_attn_fwd_workspace(*bad) == 0
    sizes = [lib.moe_gqa_attn_fwd_workspace(t, 6, 64) for t in (0, 1, 2, 90, 200, 5000, 1 << 20)]
    assert sizes == sorted(sizes)


def test_attention_backward_refusals(lib):
    need = lib.moe_gqa_attn_bwd_workspace(4, 4, 2, 1, 128)
    assert _bwd(lib, wsb=need - 1) == WS and _bwd(lib, ws=None) == WS
    for bad in (dict(do=None), dict(lse=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(do_ld=248),
                dict(dq_ld=248), dict(dk_ld=120), dict(dv_ld=120)):
        assert _bwd(lib, **bad) == INVALID, bad
    assert _bwd(lib, dk_ld=132) == ALIGN and _bwd(lib, ws=A + 8) == ALIGN
    for bad in ((-1, 4, 2, 1, 128), (4, 4, 0, 1, 128), (4, 4, 3, 2, 128), (4, 4, 2, 1, 96)):
        assert lib.moe_gqa_attn_bwd_workspace(*bad) == 0
    for h, kv, d in ((8, 1, 128), (64, 8, 128), (6, 3, 64)):
        grid = [[lib.moe_gqa_attn_bwd_workspace(q, k, h, kv, d) for k in (0, 1, 100, 128, 129, 900, 5000, 30000)]
                for q in (0, 1, 64, 500, 5000)]
        assert all(row == sorted(row) for row in grid) and all(list(c) == sorted(c) for c in zip(*grid))


@pytest.mark.parametrize("call", [_app, _dec])
def test_cache_refusals(lib, call):
    for bad in (dict(B=-1), dict(B=65537), dict(T=-1), dict(kv=0), dict(T=(1 << 24) + 1), dict(page=0), dict(page=8),
                dict(page=24), dict(pages=0), dict(max_pages=0), dict(page=1 << 20, max_pages=1 << 11),
                dict(page=1 << 20, pages=1 << 15), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None),
                dict(table=None), dict(lens=None), dict(cu=None)):
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, fmt=0) == UNSUPPORTED and call(lib, d=96) == UNSUPPORTED
    for bad in (dict(kc=A + 8), dict(vc=A + 8)):
        assert call(lib, **bad) == ALIGN, bad
    assert call(lib, B=0) == OK and call(lib, T=0) == OK


def test_append_refusals(lib):
    for bad in (dict(k=None), dict(v=None), dict(k_ld=120), dict(v_ld=120), dict(kv=1025, k_ld=1025 * 128),
                dict(B=65536, kv=9, k_ld=1152, v_ld=1152)):
        assert _app(lib, **bad) == INVALID, bad
    for bad in (dict(k=A + 8), dict(v=A + 4), dict(k_ld=132)):
        assert _app(lib, **bad) == ALIGN, bad


def test_decode_refusals(lib):
    for bad in (dict(q=None), dict(out=None), dict(q_ld=248), dict(out_ld=248), dict(h=0), dict(h=1025), dict(h=3, kv=2),
                dict(scale=0.0), dict(scale=float("nan")), dict(scale=3e38), dict(T=(1 << 23) + 1)):
        assert _dec(lib, **bad) == INVALID, bad
    for bad in (dict(q=A + 8), dict(out=A + 8), dict(ws=A + 8), dict(q_ld=260)):
        assert _dec(lib, **bad) == ALIGN, bad
    need = lib.moe_gqa_decode_workspace(128)
    assert _dec(lib, wsb=need - 1) == WS and _dec(lib, ws=None) == WS
    assert lib.moe_gqa_decode_workspace(96) == 0 and 0 < lib.moe_gqa_decode_workspace(64) < need


# ---- the classes, with tensors in host memory: none may reach a kernel ----------
BF = torch.bfloat16


@pytest.fixture
def no_calls(monkeypatch):
    def reached(*a, **k):
        raise AssertionError("reached the library")
    for name in ("moe_qk_norm_rope", "moe_qk_norm_rope_bwd", "moe_gqa_attn_fwd", "moe_gqa_attn_bwd", "moe_gqa_append",
                 "moe_gqa_decode"):
        monkeypatch.setattr(gqa.L, name, reached)


def test_classes_refuse_host_tensors(no_calls):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    q, k = torch.zeros((3, 4, 64), dtype=BF), torch.zeros((3, 2, 64), dtype=BF)
    n = gqa.QKNormRope(T=3, n_heads=4, n_kv_heads=2, head_dim=64, backward=True, device="cpu")
    a = gqa.GroupedAttention(Tq=3, Tk=3, n_heads=4, n_kv_heads=2, head_dim=64, n_seqs=1, backward=True, device="cpu")
    d = gqa.GroupedDecode(n_heads=4, n_kv_heads=2, head_dim=64, max_tokens=3, max_seqs=1, device="cpu")
    with pytest.raises(ValueError, match="current GPU"):
        n.forward(q, k)
    with pytest.raises(ValueError, match="current GPU"):
        n.backward(q, k, q, k)
    with pytest.raises(ValueError, match="current GPU"):
        a.forward(q, k, k, i32(0, 3), i32(0, 3))
    with pytest.raises(ValueError, match="current GPU"):
        a.backward(q, q, k, k, i32(0, 3), i32(0, 3))
    with pytest.raises(ValueError, match="current GPU"):
        gqa.GroupedCache.empty(2, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="current GPU"):
        d(q, None, i32(0)[None], i32(3), i32(0, 3))


def test_classes_refuse_sizes():
    for kw in (dict(n_heads=3, n_kv_heads=2), dict(n_heads=4, n_kv_heads=0), dict(n_heads=2048, n_kv_heads=2),
               dict(n_heads=4, n_kv_heads=2, head_dim=96)):
        with pytest.raises(ValueError):
            gqa.GroupedAttention(Tq=1, Tk=1, n_seqs=1, device="cpu", **kw)
        with pytest.raises(ValueError):
            gqa.GroupedDecode(max_tokens=1, max_seqs=1, device="cpu", **kw)
        with pytest.raises(ValueError):
            gqa.QKNormRope(T=1, device="cpu", **kw)
    with pytest.raises(ValueError):
        gqa.GroupedDecode(n_heads=4, n_kv_heads=2, max_tokens=1 << 24, max_seqs=1, device="cpu")
    for page, d in ((8, 64), (40, 64), (16, 96)):
        with pytest.raises(ValueError):
            gqa.GroupedCache.empty(2, page, 2, d, device="cpu")


def test_rows_of_no_tokens_and_of_one():
    """Strides that are never used may be anything; a token's values may not."""
    class T:
        dtype, device, shape, st = BF, "cuda:0", torch.Size((0, 3, 64)), (0, 0, 0)

        def stride(self):
            return self.st

        def get_device(self):
            return 0

    t = T()
    assert gqa._rows(t, "q", 3, 64, 0) == 192
    t.shape, t.st = torch.Size((1, 3, 64)), (7, 64, 1)
    assert gqa._rows(t, "q", 3, 64, 0) == 192
    t.st = (7, 128, 1)
    with pytest.raises(ValueError, match="consecutive"):
        gqa._rows(t, "q", 3, 64, 0)
    with pytest.raises(ValueError, match="current GPU"):
        gqa._rows(t, "q", 3, 64, 1)
    with pytest.raises(ValueError, match="current GPU"):
        gqa._here(torch.zeros(1), "q")
