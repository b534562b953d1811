"""The latent-attention classes with fewer rows than they are built for."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_amd as moe
from tests.gpu_util import log
from tests.test_gpu_latent import _bf, _cu, _draw, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens_q,lens_k", [([40, 70], [50, 70]), ([1], [1]), ([3], [140]), ([], []), ([0], [9])])
def test_attention_of_fewer_rows(gpu_lib, lens_q, lens_k):
    """What a plan of the exact size gives, bit for bit."""
    log(f"latent attention of fewer rows {lens_q} {lens_k}")
    h, tq, tk = 3, sum(lens_q), sum(lens_k)
    ins = _draw(1, lens_q, lens_k, h)
    cu = _i32(_cu(lens_q)), _i32(_cu(lens_k))

    def run(plan):
        out, lse = plan.forward(*ins[:3], *cu)
        res = (out, lse, *plan.backward(ins[3], *ins[:3], *cu))
        torch.cuda.synchronize()
        return res

    wide = moe.LatentAttention(Tq=200, Tk=210, n_heads=h, n_seqs=4, backward=True)
    for t in (wide.out, wide.lse, wide.dq, wide.dkv, wide.dk_rope):
        t.fill_(7.0)
    got = run(wide)
    want = run(moe.LatentAttention(Tq=tq, Tk=tk, n_heads=h, n_seqs=len(lens_q), backward=True))
    for name, x, y, buf in zip(("out", "lse", "dq", "dkv", "dk_rope"), got, want,
                               (wide.out, wide.lse, wide.dq, wide.dkv, wide.dk_rope)):
        assert x.shape == y.shape and torch.equal(x, y), name
        assert (buf[x.shape[0]:] == 7).all(), f"{name}: rows behind the call's"


def test_attention_refuses_more_rows_and_uneven_ones(gpu_lib):
    h = 2
    a = moe.LatentAttention(Tq=4, Tk=6, n_heads=h, n_seqs=1, backward=True)
    q, kv, kr, do = _draw(2, [5], [7], h)
    cu = _i32([0, 3])
    for bad in ((q, kv[:6], kr[:6]), (q[:4], kv, kr), (q[:4], kv[:6], kr[:5]), (q[:4], kv[:5], kr[:6])):
        with pytest.raises(ValueError):
            a.forward(*bad, cu, cu)
    with pytest.raises(ValueError):
        a.backward(do[:4], q[:3], kv[:6], kr[:6], cu, cu)


def test_expand_of_fewer_rows(gpu_lib):
    """Every size up to the object's, bit for bit what an object of that size gives."""
    log("latent expand of fewer rows")
    g = np.random.default_rng(6)
    c, w = _bf(g.standard_normal((140, 512))), _bf(g.standard_normal((2, 256, 512)) / 512 ** 0.5)
    wide = moe.LatentExpand(w, max_tokens=140)
    for n in (0, 1, 32, 77, 128, 129, 140):
        wide.out.fill_(7.0)
        got = wide(c[:n])
        want = moe.LatentExpand(w, max_tokens=n)(c[:n])
        torch.cuda.synchronize()
        assert got.shape == (n, 2, 256) and torch.equal(got, want), n
        assert (wide.out[n:] == 7).all(), n
    with pytest.raises(ValueError):
        moe.LatentExpand(w, max_tokens=139)(c)
