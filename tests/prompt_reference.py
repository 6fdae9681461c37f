"""The norm, 8-bit rows and their products, the rotation and the log probabilities from their definitions in
64 bits with numpy: what the GPU tests compare with. Slow and plain; shares nothing with the library."""
import numpy as np


def int8_rows(t, factor=None):
    """codes int8, scales float64 of the rows of float64 t; the scale times factor [rows] where given."""
    t = np.asarray(t, np.float64)
    factor = np.ones(len(t)) if factor is None else factor
    bad = ~np.isfinite(t).all(-1) | ~np.isfinite(factor)
    safe = np.where(bad[:, None], 0.0, t)
    top = np.abs(safe).max(-1)
    codes = np.rint((127.0 * safe) / np.where(top > 0, top, 1.0)[:, None]).astype(np.int8)
    return codes, np.where(bad, np.nan, top * np.where(bad, 0.0, factor) / 127.0)


def norm(h, weight, eps):
    """y, and t and r of the 8-bit rows, of float64 h: what the sum holds."""
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((h * h).sum(-1) / h.shape[-1] + np.float64(np.float32(eps)))
        t = h * weight
        return h * r[:, None] * weight, t, r


def turn(x, row, interleaved):
    """x [T][heads][dim] float64 turned by row [T][rot] (cosines, sines), rounded to fp32."""
    half = row.shape[1] // 2
    cos, sin = row[:, None, :half].astype(np.float64), row[:, None, half:].astype(np.float64)
    y = x.copy()
    j = np.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    with np.errstate(all="ignore"):
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., a] * sin + x[..., b] * cos
        return y.astype(np.float32)


def table(positions, rot, base=10000.0):
    """fp32 [positions][rot]: cosines and sines."""
    angle = np.arange(positions)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def logprobs(x, tokens, scale, top):
    """A dict of the outputs for float64 x [R][V], and what bounds of their errors take: `away` = sum p |s d|
    and `away2` = sum p (s d)^2, d the distance to the row's largest."""
    R, V = x.shape
    got = {name: np.full(R, np.nan) for name in ("logprob", "entropy", "lse")}
    got["rank"] = np.full(R, -1, np.int32)
    got["top_ids"] = np.full((R, top), -1, np.int32)
    got["top_logprobs"] = np.full((R, top), -np.inf)
    got["away"], got["away2"] = np.zeros(R), np.zeros(R)
    for r in range(R):
        v = x[r]
        order = np.lexsort((np.arange(V), -np.where(np.isnan(v), -np.inf, v)))
        order = order[(v[order] > -np.inf)][:top]
        got["top_ids"][r, :len(order)] = order
        valid = 0 <= tokens[r] < V
        if valid:
            got["rank"][r] = (v > v[tokens[r]]).sum()
        if not valid:
            got["logprob"][r] = 0.0
        if np.isnan(v).any() or (v == np.inf).any():
            got["top_logprobs"][r] = np.nan
            continue
        if (v == -np.inf).all():
            got["lse"][r] = -np.inf
            continue
        m = v.max()
        d = scale * (v - m)
        p = np.exp(d)
        l = p.sum()
        p /= l
        live = p > 0
        got["lse"][r] = scale * m + np.log(l)
        got["entropy"][r] = np.log(l) - (p[live] * d[live]).sum()
        got["away"][r] = -(p[live] * d[live]).sum()
        got["away2"][r] = (p[live] * d[live] ** 2).sum()
        if valid:
            got["logprob"][r] = d[tokens[r]] - np.log(l)
        got["top_logprobs"][r, :len(order)] = d[order] - np.log(l)
    return got
