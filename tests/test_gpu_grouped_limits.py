"""Grouped-query attention at the ends of what its calls take."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_amd as moe
from tests.gpu_util import log
from tests.test_gpu_grouped import _bf, _cu, _i32

pytestmark = pytest.mark.gpu


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
