"""fp64 oracle of the per-head norm with the rotation by position and of the log
probabilities, and of their gradients (numpy; one formula a line).

Heads are (tokens, heads, D); ``cos`` and ``sin`` (tokens, R/2), already looked up
for each token, with a token outside the table as None in ``good``.
"""

from __future__ import annotations

import numpy as np


def _pairs(R, interleaved):
    """Columns of both members of each rotated pair."""
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def turn(x, cos, sin, interleaved, sign=1.0):
    """x with each rotated pair (a, b) as (a cos - b sin, b cos + a sin)."""
    if cos is None:
        return x.copy()
    a, b = _pairs(2 * cos.shape[1], interleaved)
    c, s = cos[:, None, :], sign * sin[:, None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def head_rstd(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def head_forward(x, gamma, cos, sin, eps, interleaved=False, good=None):
    n = x * head_rstd(x, eps) * (1.0 if gamma is None else gamma)
    y = turn(n, cos, sin, interleaved)
    return y if good is None else np.where(good[:, None, None], y, 0.0)


def head_backward(dy, x, gamma, cos, sin, eps, interleaved=False, good=None):
    """(dx, dgamma)."""
    g = np.ones(x.shape[-1]) if gamma is None else gamma
    r = head_rstd(x, eps)
    u = turn(dy, cos, sin, interleaved, -1.0)
    if good is not None:
        u = np.where(good[:, None, None], u, 0.0)
    w = u * g
    dx = r * (w - x * r * r * (w * x).mean(-1, keepdims=True))
    return dx, (u * x * r).sum((0, 1))


def logprob_forward(z, tokens, scale, ignore=None):
    """(logprob, entropy, lse, maximum, log_sum, x = scale (z - maximum), p) of rows z."""
    with np.errstate(invalid="ignore", divide="ignore"):
        m = z.max(1)
        empty = np.isneginf(m)
        x = scale * (z - np.where(empty, 0.0, m)[:, None])
        e = np.exp(x)
        s = e.sum(1)
        l = np.log(s)
        p = np.where(empty[:, None], 0.0, e / s[:, None])
        px = p * np.where(np.isneginf(x), 0.0, x)
        entropy = np.where(empty, 0.0, l - px.sum(1))
        lse = np.where(empty, -np.inf, scale * np.where(empty, 0.0, m) + l)
        logprob = None
        if tokens is not None:
            has = has_token(tokens, z.shape[1], ignore)
            at = np.where(has, tokens, 0)
            logprob = np.where(has, np.where(empty, -np.inf, np.take_along_axis(x, at[:, None], 1)[:, 0] - l), 0.0)
    return logprob, entropy, lse, m, l, x, p


def has_token(tokens, V, ignore=None):
    has = (tokens >= 0) & (tokens < V)
    return has if ignore is None else has & (tokens != ignore)


def top_ids(z, k):
    """Ids of the k largest logits of each row, equal ones by id; -1 where a logit of -inf or NaN would follow."""
    key = np.where(np.isnan(z), -np.inf, z)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids = np.where(np.isneginf(np.take_along_axis(key, order, 1)), -1, order)
    if ids.shape[1] < k:
        ids = np.concatenate([ids, np.full((ids.shape[0], k - ids.shape[1]), -1)], 1)
    return ids


def logprob_backward(dlogprob, z, tokens, m, l, entropy, dentropy, dlse, scale, ignore=None):
    """dz from the given statistics m, l (and entropy)."""
    n, v = z.shape
    empty = np.isneginf(l)
    with np.errstate(invalid="ignore"):
        logp = np.where(empty[:, None], -np.inf, scale * (z - np.where(empty, 0.0, m)[:, None]) - np.where(empty, 0.0, l)[:, None])
    p = np.exp(logp)
    k = np.zeros((n, 1))
    g = np.zeros_like(z)
    if dlogprob is not None:
        has = has_token(tokens, v, ignore) & ~empty
        d = np.where(has, dlogprob, 0.0)
        k = k - d[:, None]
        g[np.arange(n)[has], tokens[has]] = d[has]
    if dlse is not None:
        k = k + dlse[:, None]
    if dentropy is not None:
        k = k - dentropy[:, None] * (np.where(np.isneginf(logp), 0.0, logp) + entropy[:, None])
    return scale * (g + p * k)
