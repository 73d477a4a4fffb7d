"""fp64 CPU oracle of the residual-stream operators: the block join and its
gradient, the token lookup and the table's gradient.  Plain numpy, one formula
a line, no code shared with the CUDA path.  Row tensors are (N, H) arrays; a
gate is (H,) or (B, H), its row k serving the rows k*N/B .. (k+1)*N/B - 1."""

from __future__ import annotations

import numpy as np


def _rows_of_gate(gate, N, H):
    if gate is None:
        return np.ones((N, H))
    gate = np.asarray(gate, dtype=np.float64).reshape(-1, H)
    return np.stack([gate[i * gate.shape[0] // N] for i in range(N)]) if N else np.ones((0, H))


def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).sum(axis=1) / v.shape[1] + eps)


def sandwich_forward(x, residual, gamma_post=None, gate=None, gamma_pre=None, eps=1e-6, residual_scale=1.0,
                     post=True, pre=True):
    """(y, h, rstd_post, rstd_pre); None where a norm is not taken.  h is not
    rounded."""
    N, H = x.shape
    rpost = rpre = y = None
    p = x
    if post:
        rpost = _rstd(x, eps)
        p = x * rpost[:, None] * (1.0 if gamma_post is None else gamma_post)
    h = residual_scale * residual + _rows_of_gate(gate, N, H) * p
    if pre:
        rpre = _rstd(h, eps)
        y = h * rpre[:, None] * (1.0 if gamma_pre is None else gamma_pre)
    return y, h, rpost, rpre


def sandwich_backward(dy, x, h, rstd_post, rstd_pre, gamma_post=None, gate=None, gamma_pre=None, dh_in=None,
                      residual_scale=1.0):
    """(dx, dres, dgamma_post, dgate, dgamma_pre) from the stored h and the
    saved statistics; dgate has the gate's shape."""
    N, H = x.shape
    dh = np.zeros((N, H)) if dh_in is None else np.array(dh_in, dtype=np.float64)
    dgpre = dgpost = dgate = None
    if rstd_pre is not None:
        r = rstd_pre[:, None]
        hh = h * r
        g = dy * (1.0 if gamma_pre is None else gamma_pre)
        dh = dh + r * (g - hh * (g * hh).sum(axis=1, keepdims=True) / H)
        dgpre = (dy * hh).sum(axis=0)
    dres = residual_scale * dh
    dp = _rows_of_gate(gate, N, H) * dh
    if rstd_post is None:
        p, dx = x, dp
    else:
        r = rstd_post[:, None]
        oh = x * r
        gp = 1.0 if gamma_post is None else gamma_post
        p = oh * gp
        q = dp * gp
        dx = r * (q - oh * (q * oh).sum(axis=1, keepdims=True) / H)
        dgpost = (dp * oh).sum(axis=0)
    if gate is not None:
        B = np.asarray(gate).reshape(-1, H).shape[0]
        dgate = (dh * p).reshape(B, N // B, H).sum(axis=1).reshape(np.shape(gate))
    return dx, dres, dgpost, dgate, dgpre


def lookup_forward(tokens, table, scale=1.0, gamma=None, eps=1e-6):
    """(y, h, rstd); a token outside the table is a row of zeros."""
    V, H = table.shape
    h = np.zeros((len(tokens), H))
    for i, t in enumerate(tokens):
        if 0 <= t < V:
            h[i] = scale * table[t]
    rstd = _rstd(h, eps)
    return h * rstd[:, None] * (1.0 if gamma is None else gamma), h, rstd


def lookup_backward(dh, tokens, V, scale=1.0, padding=-1):
    grad = np.zeros((V, dh.shape[1]))
    for i, t in enumerate(tokens):
        if 0 <= t < V and t != padding:
            grad[t] += scale * dh[i]
    return grad
