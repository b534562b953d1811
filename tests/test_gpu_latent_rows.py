"""Latent attention on the GPU, row by row: the norm of every (token, head)
row's error within 6 times the root mean square that its roundings give
(oracle.latent's spread; tests/test_oracle_latent_spread.py shows that
missing or doubled tokens are refused at these sizes)."""
import numpy as np
import pytest
import torch

from oracle import latent as ol
from tests.gpu_util import log
from tests.latent_util import decode_excess
from tests.test_gpu_latent import DECODE, SCALE, Paged, _cu, _decode, _draw, _i32, _np

pytestmark = pytest.mark.gpu


def _check(pg, q, nq, out, lse, tree=None, scale=SCALE):
    qn, w, at, o, l = _np(q), _np(pg.w), _cu(nq), _np(out), _np(lse)
    for b in range(len(nq)):
        s = slice(at[b], at[b + 1])
        if s.start == s.stop:
            continue
        words = None if tree is None else [t & (2 ** 64 - 1) for t in tree[s]]
        over = decode_excess(o[s], l[s], ol.cached_spread(qn[s], w, pg.rows[b], scale, words))
        assert over <= 0, f"request {b}: {over:.2f} of its bound beyond it"


def _tree(g, nq, far=4):
    """Words of random trees; a token's parent is one of the `far` before it."""
    words = []
    for n in nq:
        m = []
        for i in range(n):
            p = int(g.integers(max(-1, i - far), i)) if i else -1
            m.append((m[p] if p >= 0 else 0) | (1 << i if i < 64 else 0))
        words += m
    return words


def _signed(words):
    return None if words is None else [w - 2 ** 64 if w >> 63 else w for w in words]


@pytest.mark.parametrize("h,page,lens,nq", DECODE)
def test_decode_rows(gpu_lib, h, page, lens, nq):
    log(f"latent decode rows h={h} page={page} lens={lens} nq={nq}")
    pg = Paged(h + page, lens, page, h)
    q = _draw(h, [sum(nq)], [1], h)[0]
    out, lse = _decode(pg, q, nq)
    torch.cuda.synchronize()
    _check(pg, q, nq, out, lse)


@pytest.mark.parametrize("h,page,lens,nq", [
    (2, 16, [9000, 4097] + [int(v) for v in np.random.default_rng(0).integers(0, 90, 128)], [1] * 130),
    (3, 32, [5888], [2]), (3, 32, [5889], [2]), (3, 32, [6337, 1], [2, 1]),
    (16, 64, [9000], [1]),
])
def test_decode_rows_of_long_caches(gpu_lib, h, page, lens, nq):
    log(f"latent decode long rows h={h} page={page} lens={lens[:3]}")
    pg = Paged(5, lens, page, h)
    q = _draw(5, [sum(nq)], [1], h)[0]
    out, lse = _decode(pg, q, nq)
    torch.cuda.synchronize()
    _check(pg, q, nq, out, lse)


@pytest.mark.parametrize("h,lens,nq", [(16, [100, 7, 64], [7, 7, 7]), (4, [48, 75], [48, 48]), (128, [61], [5]),
                                       (1, [64, 130], [64, 64])])
def test_decode_rows_of_trees(gpu_lib, h, lens, nq):
    log(f"latent tree rows h={h} nq={nq}")
    pg = Paged(nq[0], lens, 16, h)
    q = _draw(h, [sum(nq)], [1], h)[0]
    tree = _tree(np.random.default_rng(h), nq)
    tree[nq[0] // 2] = 0                             # sees no new token, itself included
    out, lse = _decode(pg, q, nq, _signed(tree))
    torch.cuda.synchronize()
    _check(pg, q, nq, out, lse, tree)


@pytest.mark.parametrize("scale", [1e-3, SCALE])
def test_decode_rows_at_other_scores(gpu_lib, scale):
    log(f"latent decode rows scale={scale}")
    pg = Paged(6, [300, 1000], 64, 3)
    q = (_draw(6, [2], [1], 3)[0].float() * 20).bfloat16()
    out, lse = _decode(pg, q, [1, 1], scale=scale)
    torch.cuda.synchronize()
    _check(pg, q, [1, 1], out, lse, scale=scale)
