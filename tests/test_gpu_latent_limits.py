"""Latent attention at sizes near its documented limits, where a launch has
more work items or workgroups than one launch may have."""
import pytest
import torch

import mixture_experts_layer_sigmoid_amd as moe
from mixture_experts_layer_sigmoid_amd import _lib as L
from tests.gpu_util import log
from tests.test_gpu_latent import SCALE, Paged, _draw, _i32
from tests.test_gpu_latent_gradients import check
from tests.test_gpu_latent_rows import _check

pytestmark = pytest.mark.gpu


def test_backward_of_more_than_2_to_26_keys(gpu_lib):
    """64 work items a key for the rotary key's gradient. A sequence of 2^26
    keys without queries, whose gradients are 0, and one of 100 behind it
    (104 GB, hardly any of it touched)."""
    log("latent backward of 2^26 + 100 keys")
    many, n = 1 << 26, 100
    Tk = many + n
    ins = _draw(3, [n], [n], 1)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kv, kr = torch.empty((Tk, 1, 256), **bf), torch.empty((Tk, 64), **bf)
    kv[many:], kr[many:] = ins[1], ins[2]
    out, lse = torch.empty((n, 1, 128), **bf), torch.empty((n, 1), device="cuda")
    dq, dkv, dkr = torch.empty((n, 1, 192), **bf), torch.empty((Tk, 1, 256), **bf), torch.full((Tk, 64), 7.0, **bf)
    ws = torch.empty(L.moe_mla_attn_bwd_workspace(n, Tk, 1), dtype=torch.uint8, device="cuda")
    cu = _i32([0, 0, n]), _i32([0, many, Tk])
    L.moe_mla_attn_fwd(ins[0], 192, kv, 256, kr, 64, 1, *cu, 2, n, Tk, 1, 1, SCALE, out, 128, lse)
    L.moe_mla_attn_bwd(ins[3], 128, ins[0], 192, kv, 256, kr, 64, 1, out, 128, lse, *cu, 2, n, Tk, 1, 1, SCALE, dq, 192,
                       dkv, 256, dkr, 64, ws)
    torch.cuda.synchronize()
    check(ins, (out, dq, dkv[many:], dkr[many:]), [n], [n], True)
    assert not dkr[:many].any()
    for a in range(0, many, 1 << 24):
        assert not dkv[a:a + (1 << 24)].any()
    del kv, dkv, dkr, kr, ws
    torch.cuda.empty_cache()


def test_decode_of_2_to_24_tokens(gpu_lib):
    """The most that a call takes with one head: 131072 blocks of 128 tokens,
    524288 of 32; all but three of the tokens are in no request (70 GB)."""
    log("latent decode of 2^24 tokens")
    T, n = 1 << 24, 3
    at = T - n - 2
    pg = Paged(2, [90], 16, 1)
    q = torch.empty((T, 1, 192), dtype=torch.bfloat16, device="cuda")
    q[at:at + n] = _draw(7, [n], [1], 1)[0]
    plan = moe.LatentDecode(pg.w, max_tokens=T, max_seqs=1)
    plan.out.fill_(7.0)
    lse = torch.full((T, 1), 7.0, device="cuda")
    out = plan(q, pg.cache, _i32(pg.table), _i32(pg.lens), _i32([at, at + n]), lse=lse)
    torch.cuda.synchronize()
    _check(pg, q[at:at + n], [n], out[at:at + n], lse[at:at + n])
    for t in (out, lse):
        assert (t[:at] == 7).all() and (t[at + n:] == 7).all()
    del plan, q, out, lse
    torch.cuda.empty_cache()
