"""Plain fp64 definitions of the operators around the LM head: token statistics, the norm before
the head with its gradients, and 8-bit activation checkpoints. numpy only; shares no code with
the GPU path."""
from __future__ import annotations

import numpy as np

BLOCK = 32      # values of a checkpoint that share a scale


def token_stats(h, W, tokens=None, n_top=0):
    """h [n, d], W [V, d] float64; tokens [n] or None. Alternatives: the n_top largest logits,
    equal ones by rising id; past the vocabulary id -1, log-prob -inf."""
    z = np.asarray(h, np.float64) @ np.asarray(W, np.float64).T
    n, V = z.shape
    m = z.max(axis=1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(axis=1))
    lp = z - lse[:, None]
    out = {"z": z, "lse": lse, "entropy": -(np.exp(lp) * lp).sum(axis=1)}
    if tokens is not None:
        t = np.asarray(tokens)
        ok = (t >= 0) & (t < V)
        out["logp"] = np.where(ok, lp[np.arange(n), np.where(ok, t, 0)], 0.0)
    k = min(n_top, V)
    order = np.argsort(-z, axis=1, kind="stable")[:, :k]
    out["top_ids"] = np.full((n, n_top), -1, np.int32)
    out["top_logp"] = np.full((n, n_top), -np.inf)
    out["top_ids"][:, :k] = order
    out["top_logp"][:, :k] = np.take_along_axis(lp, order, axis=1)
    return out


def norm_forward(x, weight=None, bias=None, kind="layer", eps=1e-5):
    """(y, mean, rstd) by rows."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1) if kind == "layer" else np.zeros(len(x))
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    y = c * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def norm_backward(x, dy, mean, rstd, weight=None, kind="layer"):
    """(dx, dweight, dbias) for given statistics (mean is not read for rms)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    mu = np.asarray(mean, np.float64)[:, None] if kind == "layer" else 0.0
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (x - mu) * r
    g = dy * np.asarray(weight, np.float64) if weight is not None else dy
    dx = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * r, (dy * xh).sum(axis=0), dy.sum(axis=0)


def checkpoint(x):
    """(codes int8, scales uint8, values float64) of rows x held in 8 bits."""
    x = np.asarray(x, np.float64)
    rows, d = x.shape
    nb = -(-d // BLOCK)
    p = np.zeros((rows, nb * BLOCK))
    p[:, :d] = x
    p = p.reshape(rows, nb, BLOCK)
    codes = np.zeros(p.shape, np.int8)
    scales = np.zeros((rows, nb), np.uint8)
    values = np.zeros(p.shape)
    for r in range(rows):
        for b in range(nb):
            v = p[r, b]
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                values[r, b] = np.nan
                continue
            top, e = np.abs(v).max(), -126
            if top > 0:
                e = max(-126, int(np.frexp(top)[1]) - 8)
                while top > 127.0 * 2.0 ** e:      # the smallest exponent that holds it
                    e += 1
            e = min(e, 121)
            codes[r, b] = np.clip(np.rint(v / 2.0 ** e), -127, 127)
            scales[r, b] = e + 127
            values[r, b] = codes[r, b].astype(np.float64) * 2.0 ** e
    return codes.reshape(rows, -1)[:, :d], scales, values.reshape(rows, -1)[:, :d]
