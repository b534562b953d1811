"""Latent decode on the GPU: joins of several tokens a workgroup, teams of
workgroups, rows that no request holds, more than 64 requests or drafted
tokens, each (token, head) row by row against the oracle."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_amd as moe
from tests.gpu_util import log
from tests.test_gpu_latent import Paged, _cu, _draw, _i32
from tests.test_gpu_latent_rows import _check, _signed, _tree

pytestmark = pytest.mark.gpu


def _run(h, page, lens, nq, tree=None, before=0, behind=0, seed=0):
    """A call with `before` and `behind` rows of q that no request holds."""
    pg = Paged(seed + h, lens, page, h)
    n = sum(nq)
    T = before + n + behind
    q = _draw(seed, [T], [1], h)[0]
    q[:before], q[before + n:] = float("nan"), float("nan")
    plan = moe.LatentDecode(pg.w, max_tokens=T, max_seqs=len(nq))
    plan.out.fill_(7.0)
    lse = torch.full((T, h), 7.0, device="cuda")
    words = None
    if tree is not None:
        words = torch.tensor([0] * before + _signed(tree) + [0] * behind, dtype=torch.int64, device="cuda")
    args = (q, pg.cache, _i32(pg.table), _i32(pg.lens), _i32(before + _cu(nq)), words)
    out = plan(*args, lse=lse)
    torch.cuda.synchronize()
    held = slice(before, before + n)
    for t in (out, lse):
        assert (t[:before] == 7).all() and (t[before + n:] == 7).all(), "rows that no request holds"
    _check(pg, q[held], nq, out[held], lse[held], tree)
    first = out[held].clone()
    plan(*args, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(first, out[held]), "two runs differ"


# heads, new tokens in all (three of them in no request): with two workgroups a
# compute unit to fill, a workgroup joins 1, 2, 4, 8, 16 and 32 tokens of a head
@pytest.mark.parametrize("h,T", [(128, 6), (128, 9), (128, 19), (16, 201), (128, 27), (128, 53), (128, 101), (512, 5)])
def test_joins_of_many_tokens(gpu_lib, h, T):
    """One long cache, which is cut into pieces, among short ones, some whole."""
    log(f"latent join h={h} T={T}")
    g = np.random.default_rng(T)
    n = T - 3
    lens = [int(v) for v in g.integers(1, 130, n)]
    lens[n // 2] = 1500 if h < 512 else 300
    _run(h, 32, lens, [1] * n, before=1, behind=2, seed=T)


# rows of the average request in tiles of 64: 8, 16 and 32, taken by as many
# workgroups; the others' last groups have fewer
@pytest.mark.parametrize("nq", [[4, 5, 3], [8, 9, 7], [16, 17, 15]])
@pytest.mark.parametrize("drafted", [False, True])
def test_teams_of_workgroups(gpu_lib, nq, drafted):
    log(f"latent teams nq={nq} drafted={drafted}")
    tree = _tree(np.random.default_rng(nq[0]), nq) if drafted else None
    _run(128, 16, [700, 200, 70], nq, tree, seed=nq[0])


@pytest.mark.parametrize("h,lens,nq", [(16, [130], [70]), (3, [66, 200], [66, 65])])
def test_trees_of_more_than_64(gpu_lib, h, lens, nq):
    """Drafted tokens from the 65th on are hidden from all."""
    log(f"latent tree h={h} nq={nq}")
    _run(h, 16, lens, nq, _tree(np.random.default_rng(h), nq), seed=h)


@pytest.mark.parametrize("h", [1, 8])
def test_trees_of_many_requests(gpu_lib, h):
    log(f"latent tree of 70 requests h={h}")
    g = np.random.default_rng(h)
    nq = [int(v) for v in g.integers(0, 4, 70)]
    lens = [n + int(v) for n, v in zip(nq, g.integers(0, 200, 70))]
    _run(h, 16, lens, nq, _tree(g, nq), before=2, seed=h)
