"""Grouped-query attention in fp64: norms of queries and keys with the
rotation by position, attention over packed sequences and its gradients, the
8-bit paged cache and attention over it. One sequence at a time, from the
definitions.

Functions also return how far a kernel that rounds its matrix operands to bf16
may be off, element by element (*_tol), and the root mean square of a row's
error (*_rms): see oracle.latent for U, RMS and SLACK.
"""
from __future__ import annotations

import numpy as np

from .latent import RMS, SLACK, U, _norm, softmax, visible

BLOCK = 16


# ---- norms and rotation ---------------------------------------------------------
def turn(x, angle, rotary, interleaved):
    """The first `rotary` values of the last axis, in pairs, by angle [...,
    rotary / 2]."""
    y = x.copy()
    half = rotary // 2
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
    y[..., a] = x[..., a] * np.cos(angle) - x[..., b] * np.sin(angle)
    y[..., b] = x[..., a] * np.sin(angle) + x[..., b] * np.cos(angle)
    return y


def norm_turn(x, w, eps, angle, rotary, interleaved):
    """x [T, heads, D], w [D] or None, angle [T, rotary / 2] or None -> result
    and its bound (one rounding; fp32 before it: 2^-20 of each pair's terms)."""
    u = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    mass = np.abs(u)
    if angle is None:
        return u, SLACK * U * np.abs(u) + 2.0 ** -20 * mass
    y = turn(u, angle[:, None], rotary, interleaved)
    half = rotary // 2
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
    pair = mass[..., a] + mass[..., b]
    mass[..., a] = pair
    mass[..., b] = pair
    return y, SLACK * U * np.abs(y) + 2.0 ** -20 * mass


def norm_turn_backward(dy, x, w, eps, angle, rotary, interleaved):
    """dx, dw (None without w) and their bounds."""
    g = dy if angle is None else turn(dy, -angle[:, None], rotary, interleaved)
    big = np.abs(dy).max(-1, keepdims=True) * 2          # of a turned pair
    if w is None:
        return g, SLACK * U * np.abs(g) + 2.0 ** -20 * big, None, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    gw = g * w
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdims=True))
    # fp32 products and sums of D terms: 2^-18 of the terms' absolute values
    mass = r * (big * np.abs(w) + np.abs(xh) * (big * np.abs(w * xh)).mean(-1, keepdims=True))
    dw = (g * xh).sum((0, 1))
    return dx, SLACK * U * np.abs(dx) + 2.0 ** -18 * mass, dw, 2.0 ** -18 * (big * np.abs(xh)).sum((0, 1)) + 1e-30


# ---- attention ------------------------------------------------------------------
def attention(q, k, v, see, scale):
    """q [n_q, h, D], k and v [n_k, h / G, D], see [n_q, n_k] -> out, lse, out's
    bound and root mean square."""
    n_q, h, d = q.shape
    g = h // k.shape[1]
    r = {"out": np.zeros(q.shape), "lse": np.zeros((n_q, h)), "out_tol": np.zeros(q.shape), "out_rms": np.zeros((n_q, h))}
    for x in range(h):
        kx, vx = k[:, x // g], v[:, x // g]
        p, r["lse"][:, x] = softmax(scale * (q[:, x] @ kx.T), see)
        out = p @ vx
        r["out"][:, x] = out
        # the weights' rounding, the result's rounding
        r["out_tol"][:, x] = SLACK * U * (p @ np.abs(vx) + np.abs(out)) + 1e-7
        r["out_rms"][:, x] = _norm(RMS ** 2 * ((p * p) @ (vx * vx) + out * out))
    return r


def attention_backward(dout, q, k, v, causal, scale):
    """Gradients, bounds and root mean squares; dk and dv summed over the
    group's heads."""
    n_q, h, d = q.shape
    n_k, kv = k.shape[:2]
    g = h // kv
    see = visible(n_q, n_k, causal)
    r = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    tol = {n + "_tol": np.zeros(a.shape) for n, a in r.items()}
    var = {n: np.zeros(a.shape) for n, a in r.items()}
    for x in range(h):
        j = x // g
        qx, do, kx, vx = q[:, x], dout[:, x], k[:, j], v[:, j]
        p, _ = softmax(scale * (qx @ kx.T), see)
        o = p @ vx
        dp = do @ vx.T
        ds = p * (dp - (p * dp).sum(1, keepdims=True))
        dq, dk, dv = scale * (ds @ kx), scale * (ds.T @ qx), p.T @ do
        r["dq"][:, x] = dq
        r["dk"][:, j] += dk
        r["dv"][:, j] += dv
        # delta is formed from the rounded output of rounded weights; ds is
        # rounded as operand (fp32 sums of the scores: a few 2^-24 of them)
        d_delta = (np.abs(do) * (U * (p @ np.abs(vx)) + U * np.abs(o))).sum(1, keepdims=True)
        e = U * np.abs(ds) + p * d_delta + 2.0 ** -20 * p * (np.abs(do) @ np.abs(vx).T)
        tol["dq_tol"][:, x] = SLACK * (scale * (e @ np.abs(kx)) + U * np.abs(dq)) + 1e-7
        tol["dk_tol"][:, j] += SLACK * scale * (e.T @ np.abs(qx))
        tol["dv_tol"][:, j] += SLACK * U * (p.T @ np.abs(do))
        o_var = RMS ** 2 * ((p * p) @ (vx * vx) + o * o)
        delta_var = (do * do * o_var).sum(1, keepdims=True)
        ds_var = RMS ** 2 * ds * ds
        var["dq"][:, x] = scale ** 2 * (ds_var @ (kx * kx) + delta_var * (p @ kx) ** 2) + (RMS * dq) ** 2
        var["dk"][:, j] += scale ** 2 * ((ds_var + p * p * delta_var).T @ (qx * qx))
        var["dv"][:, j] += RMS ** 2 * ((p * p).T @ (do * do))
    for n in ("dk", "dv"):
        tol[n + "_tol"] += SLACK * U * np.abs(r[n]) + 1e-7
        var[n] += (RMS * r[n]) ** 2
    return {**r, **tol, **{n + "_rms": _norm(a) for n, a in var.items()}}


def new_tokens_see(n_q, n, tree=None):
    """[n_q, n]: what a request's n_q new tokens, the last of its n, see."""
    first = n - n_q
    see = np.zeros((n_q, n), bool)
    for i in range(n_q):
        for j in range(n):
            new = j - first
            see[i, j] = new < 0 or (new <= i if tree is None else new < 64 and bool((int(tree[i]) >> new) & 1))
    return see


# ---- 8-bit codes ------------------------------------------------------------------
def _e4m3_values():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = -x if c & 128 else x
    return v


E4M3 = _e4m3_values()


def e4m3(x):
    """Codes of x, |x| <= 448: nearest value, ties to the even code, the sign
    kept."""
    a = np.abs(x)
    grid = E4M3[:127]
    hi = np.minimum(np.searchsorted(grid, a), 126)
    lo = np.maximum(hi - 1, 0)
    up = grid[hi] - a
    down = a - grid[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(amax):
    """Smallest e in [-127, 127] with amax <= 448 2^e; -127 of nothing."""
    if amax == 0:
        return -127
    e = -127
    while amax > 448 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """The cache by its definition: codes [n_pages, kv, page_size, D] and
    exponents [n_pages, kv, page_size / 16] of keys and of values."""

    def __init__(self, n_pages, page, kv, d):
        self.page = page
        self.codes = {n: np.zeros((n_pages, kv, page, d), np.uint8) for n in "kv"}
        self.e = {n: np.zeros((n_pages, kv, page // BLOCK), np.int64) for n in "kv"}

    @classmethod
    def of_bytes(cls, k, v, ks, vs):
        """From the library's arrays."""
        n_pages, kv, blocks, d16 = k.shape[:4]
        c = cls(n_pages, blocks * BLOCK, kv, d16 * 16)
        c.codes["k"] = k.transpose(0, 1, 2, 4, 3, 5).reshape(c.codes["k"].shape).copy()
        # [p, h, b, d / 2, t / 4 % 2, d % 2, t / 8, t % 4] -> [p, h, b, t, d]
        c.codes["v"] = v.transpose(0, 1, 2, 6, 4, 7, 3, 5).reshape(c.codes["v"].shape).copy()
        c.e = {"k": ks.astype(np.int64) - 127, "v": vs.astype(np.int64) - 127}
        return c

    def append(self, name, x, table, n):
        """x [new, kv, D]: the last of a request's n tokens."""
        new = x.shape[0]
        start = n - new
        for blk in range(start // BLOCK, -(-n // BLOCK)):
            lo, hi = blk * BLOCK, (blk + 1) * BLOCK
            page, at = int(table[lo // self.page]), lo % self.page
            for h in range(x.shape[1]):
                mine = x[max(lo, start) - start:min(hi, n) - start, h]
                e = exponent(np.abs(mine).max())
                old = self.e[name][page, h, at // BLOCK]
                rows = self.codes[name][page, h, at:at + BLOCK]
                if start > lo:
                    e = max(e, old)
                    if e > old:
                        rows[:start - lo] = e4m3(E4M3[rows[:start - lo]] * 2.0 ** (old - e))
                rows[max(lo, start) - lo:min(hi, n) - lo] = e4m3(mine * 2.0 ** -e)
                self.e[name][page, h, at // BLOCK] = e

    def rows(self, name, table, n):
        """A request's n tokens [n, kv, D]."""
        j = np.arange(n)
        page, at = np.asarray(table)[j // self.page], j % self.page
        x = E4M3[self.codes[name][page, :, at]]
        return x * 2.0 ** self.e[name][page, :, at // BLOCK][..., None].astype(float)
