"""Plain fp64 forms of the linear attention with decay, the verification of
drafted tokens and the block norms (test infrastructure only): one token, one
row, one formula per line."""

from __future__ import annotations

import numpy as np

from .gdn_oracle import _f64, sequence_bounds


def linear(q, k, v, g, scale, Hq, Hv, cu_seqlens=None, num_seqs=1, initial_state=None, magnitudes=False):
    """S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over packed tokens.

    q, k [T, Hq, dk]; v [T, Hv, dv]; g [T, Hv] or [Hv]; initial_state
    [N or 1, Hv, dk, dv] or None.  ``magnitudes``: the same with absolute values
    of every input (the sums that error bounds are relative to).
    Returns dict(o, final, alpha)."""
    q, k, v, g, s0 = (_f64(x) for x in (q, k, v, g, initial_state))
    if magnitudes:
        q, k, v, s0 = (None if x is None else np.abs(x) for x in (q, k, v, s0))
        scale = abs(scale)
    T, _, dk = k.shape
    dv = v.shape[2]
    heads = np.arange(Hv) // (Hv // Hq)
    N = num_seqs if cu_seqlens is None else len(np.asarray(cu_seqlens).reshape(-1)) - 1
    alpha = np.exp(np.broadcast_to(g, (T, Hv)))
    o = np.zeros((T, Hv, dv))
    final = np.zeros((N, Hv, dk, dv))
    for s, (t0, t1) in enumerate(sequence_bounds(N, T // max(N, 1), cu_seqlens)):
        S = np.zeros((Hv, dk, dv)) if s0 is None else s0[s if s0.shape[0] > 1 else 0].copy()
        for t in range(t0, t1):
            S = alpha[t][:, None, None] * S + k[t][heads][:, :, None] * v[t][:, None, :]
            o[t] = scale * (q[t][heads][:, None, :] @ S)[:, 0]
        final[s] = S
    return dict(o=o, final=final, alpha=alpha)


def verify_row(p, q, x, u, n):
    """One row: p [K+1, V], q [K, V] or None, x [K], u [K+1], n drafts.
    Returns (tokens list of length K+1, number emitted)."""
    p, u = _f64(p), _f64(u)
    q = None if q is None else _f64(q)
    K, V = len(x), p.shape[1]
    out = [-1] * (K + 1)
    n = min(int(n), K)
    if n < 0:
        return out, 0
    a = 0
    while a < n:
        d = int(x[a])
        if not (0 <= d < V):
            break
        if not (u[a] * (1.0 if q is None else q[a, d]) < p[a, d]):
            break
        out[a] = d
        a += 1

    def positive(w):
        with np.errstate(invalid="ignore"):
            return np.where((w > 0) & (w < np.inf), w, 0.0)
    w = positive(p[a])
    if a < n:
        if q is not None:
            with np.errstate(invalid="ignore"):
                rest = positive(p[a] - q[a])
        else:
            rest = w.copy()
            if 0 <= int(x[a]) < V:
                rest[int(x[a])] = 0.0
        if rest.sum() > 0:
            w = rest
    c = np.cumsum(w)
    if c[-1] > 0:
        over = np.nonzero(c > u[K] * c[-1])[0]
        out[a] = int(over[0]) if len(over) else int(np.nonzero(w)[0][-1])
    return out, a + 1


def block_norm(y, gate=None, act="none", residual=None, scale=1.0, post=None, nxt=None, eps=1e-6):
    """(h, normed or None), and the magnitude |residual| + |scale * m| of h's terms."""
    y, gate, residual, post, nxt = (_f64(x) for x in (y, gate, residual, post, nxt))
    m = y
    if post is not None:
        yg = y.reshape(y.shape[0], y.shape[1] // post.size, post.size)
        m = (yg / np.sqrt((yg ** 2).mean(-1, keepdims=True) + eps) * post).reshape(y.shape)
    if act != "none":
        s = 1.0 / (1.0 + np.exp(-gate))
        m = m * (gate * s if act == "silu" else s)
    r = 0.0 if residual is None else residual
    h = r + scale * m
    normed = None if nxt is None else h / np.sqrt((h ** 2).mean(-1, keepdims=True) + eps) * nxt
    return h, normed, np.abs(r) + np.abs(scale * m)
