"""Latent attention in fp64 ([TE-DSV3] Description, MultiLatentAttention):
expanded form and its gradients, absorbed form over a paged cache, the cache
append. One sequence at a time, from the definition.

Each function also returns how far a kernel that rounds its matrix operands
to bf16 may be off, element by element: u = 2^-8 is the largest relative
error of a rounding to bf16 (8 significant bits: half a unit in the last
place, reached just above powers of two), sums of products are bounded by
the sums of their terms' absolute values, and terms of order u^2 and of fp32
are covered by SLACK.
"""
from __future__ import annotations

import numpy as np

NOPE, ROPE, VALUE, LATENT = 128, 64, 128, 512
U = 2.0 ** -8
SLACK = 1.1


def visible(n_q, n_k, causal):
    i, j = np.arange(n_q)[:, None], np.arange(n_k)[None]
    return (j <= i + n_k - n_q) if causal else np.ones((n_q, n_k), bool)


def softmax(s, see):
    """Weights and log-sum-exp of the visible scores of each row; a row
    without any has weights 0 and lse -inf."""
    s = np.where(see, s, -np.inf)
    m = np.max(s, axis=-1, initial=-np.inf, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    z = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(np.isfinite(m), m, 0.0)[..., 0] + np.log(z[..., 0])
    return p / np.where(z > 0, z, 1.0), lse


def attention(q, kv, k_rope, causal, scale):
    """q [n_q, h, 192], kv [n_k, h, 256], k_rope [n_k, 64] -> dict of out
    [n_q, h, 128], lse [n_q, h] and out's bound."""
    n_q, h = q.shape[:2]
    n_k = kv.shape[0]
    res = {"out": np.zeros((n_q, h, VALUE)), "lse": np.zeros((n_q, h)), "out_tol": np.zeros((n_q, h, VALUE))}
    see = visible(n_q, n_k, causal)
    for x in range(h):
        k = np.concatenate([kv[:, x, :NOPE], k_rope], 1)
        v = kv[:, x, NOPE:]
        p, res["lse"][:, x] = softmax(scale * (q[:, x] @ k.T), see)
        res["out"][:, x] = p @ v
        # the weights' rounding, the result's rounding
        res["out_tol"][:, x] = SLACK * U * (p @ np.abs(v) + np.abs(res["out"][:, x])) + 1e-7
    return res


def attention_backward(dout, q, kv, k_rope, causal, scale):
    """Gradients dq, dkv, dk_rope and their bounds."""
    n_q, h = q.shape[:2]
    n_k = kv.shape[0]
    see = visible(n_q, n_k, causal)
    r = {"dq": np.zeros(q.shape), "dkv": np.zeros(kv.shape), "dk_rope": np.zeros(k_rope.shape)}
    tol = {"dq_tol": np.zeros(q.shape), "dkv_tol": np.zeros(kv.shape), "dk_rope_tol": np.zeros(k_rope.shape)}
    for x in range(h):
        k = np.concatenate([kv[:, x, :NOPE], k_rope], 1)
        v, do, qx = kv[:, x, NOPE:], dout[:, x], q[:, x]
        p, _ = softmax(scale * (qx @ k.T), see)
        o = p @ v
        dp = do @ v.T
        ds = p * (dp - (p * dp).sum(1, keepdims=True))
        r["dq"][:, x] = scale * (ds @ k)
        dk = scale * (ds.T @ qx)
        dv = p.T @ do
        r["dkv"][:, x] = np.concatenate([dk[:, :NOPE], dv], 1)
        r["dk_rope"] += dk[:, NOPE:]
        # delta is formed from the rounded output of rounded weights; ds is
        # rounded as operand (fp32 sums of the scores: a few 2^-24 of them)
        d_delta = (np.abs(do) * (U * (p @ np.abs(v)) + U * np.abs(o))).sum(1, keepdims=True)
        e = U * np.abs(ds) + p * d_delta + 2.0 ** -20 * p * (np.abs(do) @ np.abs(v).T)
        tol["dq_tol"][:, x] = SLACK * (scale * (e @ np.abs(k)) + U * np.abs(r["dq"][:, x])) + 1e-7
        dk_tol = scale * (e.T @ np.abs(qx))
        tol["dkv_tol"][:, x, :NOPE] = SLACK * (dk_tol[:, :NOPE] + U * np.abs(dk[:, :NOPE])) + 1e-7
        tol["dkv_tol"][:, x, NOPE:] = SLACK * U * (p.T @ np.abs(do) + np.abs(dv)) + 1e-7
        tol["dk_rope_tol"] += SLACK * dk_tol[:, NOPE:] + 1e-7
    tol["dk_rope_tol"] += SLACK * U * np.abs(r["dk_rope"])
    return {**r, **tol}


def cached(q, w_kvb, rows, scale, tree=None):
    """Absorbed form for one request: q [n_q, h, 192] against its cache rows
    [n, 576], the n_q new tokens' the last; w_kvb [h, 256, 512]. tree: one
    integer a new token (bit j: sees new token j). Hidden rows may hold
    anything."""
    n_q, h = q.shape[:2]
    n = rows.shape[0]
    first = n - n_q
    see = np.zeros((n_q, n), bool)
    for i in range(n_q):
        for j in range(n):
            new = j - first
            see[i, j] = new < 0 or (new <= i if tree is None else new < 64 and bool((int(tree[i]) >> new) & 1))
    res = {"out": np.zeros((n_q, h, VALUE)), "lse": np.zeros((n_q, h)), "out_tol": np.zeros((n_q, h, VALUE)),
           "lse_tol": np.zeros((n_q, h))}
    for x in range(h):
        wk, wv = w_kvb[x, :NOPE], w_kvb[x, NOPE:]
        for i in range(n_q):
            c = rows[see[i]]                       # only what the token sees
            ql = q[i, x, :NOPE] @ wk
            s = scale * (c[:, :LATENT] @ ql + c[:, LATENT:] @ q[i, x, NOPE:])
            p, lse = softmax(s[None], np.ones((1, len(s)), bool))
            p = p[0]
            res["lse"][i, x] = lse[0]
            res["out"][i, x] = wv @ (p @ c[:, :LATENT])
            # the absorbed query's rounding moves each score by at most e; a
            # weight by (e + its mean) of itself; weights are rounded once, or
            # twice where the two halves of a tile had other references
            e = scale * U * (np.abs(c[:, :LATENT]) @ np.abs(ql))
            mean = p @ e
            move = (p * (e + mean + 2 * U)) @ np.abs(c[:, :LATENT])
            res["out_tol"][i, x] = SLACK * (np.abs(wv) @ move + U * np.abs(res["out"][i, x])) + 1e-6
            res["lse_tol"][i, x] = SLACK * mean + 1e-5
    return res


def rotate(x, angle, interleaved):
    """Pairs of the last axis (64 values) turned by angle [..., 32]."""
    y = np.empty_like(x)
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y[..., a] = x[..., a] * np.cos(angle) - x[..., b] * np.sin(angle)
    y[..., b] = x[..., a] * np.sin(angle) + x[..., b] * np.cos(angle)
    return y


def cache_row(kv_a, w, eps):
    """Normalized latents of rows [T, >= 512]."""
    c = kv_a[:, :LATENT]
    return c / np.sqrt((c * c).mean(1, keepdims=True) + eps) * w


# ---- root mean squares of the errors ------------------------------------------
# The bounds above hold for every element, and so are wide where many terms
# add up. The errors of the roundings are independent and of mean zero, each at
# most uniform over half a unit in the last place (root mean square
# U / sqrt(3) of the value, just above a power of two), so what they do to a
# row of results has a root mean square that the functions below give.
RMS = U / 3 ** 0.5


def _norm(var):
    return np.sqrt(var.sum(-1))


def cached_spread(q, w_kvb, rows, scale, tree=None):
    """cached()'s out and lse, with the root mean square of the error of each
    (token, head): the norm of out's 128 values (out_rms), lse (lse_rms). The
    absorbed query and the result are rounded once each, the weights at most
    twice (again where the two halves of a tile had other references). fp32 is
    out_floor and lse_floor, bounds and not root mean squares: scores are off
    by 2^-22 of their terms' absolute values, sums by 2^-20 of theirs."""
    n_q, h = q.shape[:2]
    n = rows.shape[0]
    first = n - n_q
    res = {"out": np.zeros((n_q, h, VALUE)), "lse": np.full((n_q, h), -np.inf), "out_rms": np.zeros((n_q, h)),
           "lse_rms": np.zeros((n_q, h)), "out_floor": np.zeros((n_q, h)), "lse_floor": np.zeros((n_q, h))}
    wk, wv = w_kvb[:, :NOPE], w_kvb[:, NOPE:]
    with np.errstate(invalid="ignore"):
        values = np.matmul(rows[None, :, :LATENT], wv.transpose(0, 2, 1))            # [h, n, 128]
    for i in range(n_q):
        new = np.arange(n) - first
        if tree is None:
            see = new <= i
        else:
            word = int(tree[i])
            see = np.array([v < 0 or (v < 64 and bool((word >> v) & 1)) for v in new.tolist()], bool)
        if not see.any():
            continue
        c, v = rows[see], values[:, see]
        ql = np.matmul(q[i, :, None, :NOPE], wk)[:, 0]                               # [h, 512]
        p, lse = softmax(scale * (ql @ c[:, :LATENT].T + q[i, :, NOPE:] @ c[:, LATENT:].T), True)
        out = np.matmul(p[:, None], v)[:, 0]
        # a score moves by scale q_r c_r times the error of q_lat's element r
        moved = np.matmul(c[:, :LATENT].T[None], p[..., None] * (v - out[:, None]))  # [h, 512, 128]
        var = (RMS * out) ** 2 + 2 * RMS ** 2 * np.matmul((p * p)[:, None], v * v)[:, 0]
        var += (scale * RMS) ** 2 * np.matmul((ql * ql)[:, None], moved * moved)[:, 0]
        res["out"][i], res["lse"][i], res["out_rms"][i] = out, lse, _norm(var)
        res["lse_rms"][i] = scale * RMS * _norm((ql * (p @ c[:, :LATENT])) ** 2)
        mass = np.matmul(np.abs(wv), (p @ np.abs(c[:, :LATENT]))[..., None])[..., 0]
        terms = np.abs(ql) @ np.abs(c[:, :LATENT]).T + np.abs(q[i, :, NOPE:]) @ np.abs(c[:, LATENT:]).T
        off = 2.0 ** -22 * scale * terms.max(1)
        res["out_floor"][i] = (2.0 ** -20 + 2 * off) * _norm(mass ** 2)
        res["lse_floor"][i] = off + 2.0 ** -20 * (1 + np.abs(lse))
    return res


def attention_spread(dout, q, kv, k_rope, causal, scale):
    """attention() and attention_backward(), with the root mean square of the
    error of each row of a head: out and dq (norms over a query's values), dk
    and dv (the two halves of a key's dkv), dk_rope (over the heads' sum). The
    weights, ds and the results are rounded once each; delta is formed from
    the rounded output of rounded weights."""
    n_q, h = q.shape[:2]
    n_k = kv.shape[0]
    see = visible(n_q, n_k, causal)
    r = {"out": np.zeros((n_q, h, VALUE)), "dq": np.zeros(q.shape), "dkv": np.zeros(kv.shape),
         "dk_rope": np.zeros(k_rope.shape)}
    rms = {"out_rms": np.zeros((n_q, h)), "dq_rms": np.zeros((n_q, h)), "dk_rms": np.zeros((n_k, h)),
           "dv_rms": np.zeros((n_k, h))}
    rope_var = np.zeros(k_rope.shape)
    for x in range(h):
        k = np.concatenate([kv[:, x, :NOPE], k_rope], 1)
        v, do, qx = kv[:, x, NOPE:], dout[:, x], q[:, x]
        p, _ = softmax(scale * (qx @ k.T), see)
        o = p @ v
        dp = do @ v.T
        ds = p * (dp - (p * dp).sum(1, keepdims=True))
        dq, dk, dv = scale * (ds @ k), scale * (ds.T @ qx), p.T @ do
        r["out"][:, x], r["dq"][:, x], r["dkv"][:, x] = o, dq, np.concatenate([dk[:, :NOPE], dv], 1)
        r["dk_rope"] += dk[:, NOPE:]
        o_var = RMS ** 2 * ((p * p) @ (v * v) + o * o)
        delta_var = (do * do * o_var).sum(1, keepdims=True)                 # one error a query, for all its keys
        ds_var = RMS ** 2 * ds * ds
        dk_var = scale ** 2 * ((ds_var + p * p * delta_var).T @ (qx * qx))
        rms["out_rms"][:, x] = _norm(o_var)
        rms["dq_rms"][:, x] = _norm(scale ** 2 * (ds_var @ (k * k) + delta_var * (p @ k) ** 2) + (RMS * dq) ** 2)
        rms["dk_rms"][:, x] = _norm(dk_var[:, :NOPE] + (RMS * dk[:, :NOPE]) ** 2)
        rms["dv_rms"][:, x] = _norm(RMS ** 2 * ((p * p).T @ (do * do) + dv * dv))
        rope_var += dk_var[:, NOPE:]
    return {**r, **rms, "dk_rope_rms": _norm(rope_var + (RMS * r["dk_rope"]) ** 2)}
