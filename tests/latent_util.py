"""Row by row comparison of latent attention with oracle.latent's spread: the
norm of a row's error against the root mean square that its roundings give."""
import numpy as np

# A row's error is a sum of independent errors, each uniform at most, so its
# tails are no heavier than a Gaussian's of the same root mean square: beyond
# 6 of them in the worst case (all of it in one direction) with a chance of
# 2e-8 a row. Many rows together lie close to their root mean square, and
# rounding errors stay below the uniform's (0.74 of it on average): 1.5.
ROW, ALL, MANY = 6.0, 1.5, 32


def row_excess(got, want, rms, floor=0.0):
    """By how much the worst row (last axis) leaves its bound, as a share of
    it; at most 0 where all hold. Rows whose result is not finite (lse of a
    query without keys) have to be equal."""
    off = np.linalg.norm(got - want, axis=-1)
    if off.size == 0:
        return 0.0
    bound = ROW * rms + floor + 1e-30
    worst = (off / bound).max() - 1
    if off.size >= MANY:
        all_bound = ALL * np.sqrt((rms ** 2).sum()) + np.sqrt((np.broadcast_to(floor, off.shape) ** 2).sum()) + 1e-30
        worst = max(worst, np.sqrt((off ** 2).sum()) / all_bound - 1)
    return worst


def lse_excess(got, ref):
    if not np.array_equal(np.isfinite(got), np.isfinite(ref["lse"])):
        return np.inf
    ok = np.isfinite(got)
    if not np.array_equal(got[~ok], ref["lse"][~ok]):
        return np.inf
    if not ok.any():
        return 0.0
    return (np.abs(got[ok] - ref["lse"][ok]) / (ROW * ref["lse_rms"][ok] + ref["lse_floor"][ok])).max() - 1


def decode_excess(out, lse, ref):
    """Of a request's out and lse against oracle.latent.cached_spread."""
    if not np.isfinite(out).all():
        return np.inf
    return max(row_excess(out, ref["out"], ref["out_rms"], ref["out_floor"]), lse_excess(lse, ref))
