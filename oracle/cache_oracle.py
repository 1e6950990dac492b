"""Plain fp64 forms of the paged cache (append, attention), the beam selection and
the reordering of rows (test infrastructure only): one token, one row, one formula
per line."""

from __future__ import annotations

import numpy as np

from .gdn_oracle import _f64, sequence_bounds


def places(block_table, cache_lens, page_size, num_pages, cu_seqlens=None, tokens=None):
    """[(token row, sequence, place, page or -1, row in the page)] of every new token."""
    table, lens = np.asarray(block_table), np.asarray(cache_lens)
    N, cols = table.shape
    out = []
    for s, (t0, t1) in enumerate(sequence_bounds(N, (tokens or 0) // max(N, 1), cu_seqlens)):
        for t in range(t0, t1):
            at = int(lens[s]) - (t1 - t)
            page = int(table[s, at // page_size]) if 0 <= at < cols * page_size else -1
            out.append((t, s, at, page if 0 <= page < num_pages else -1, at % page_size))
    return out


def rotate(x, angles, rotary, interleaved):
    """x [..., d] turned by angles [..., rotary / 2]; and the size |x1| + |x2| of each element's terms."""
    y, size = x.copy(), np.abs(x)
    j = np.arange(rotary // 2)
    first, second = (2 * j, 2 * j + 1) if interleaved else (j, j + rotary // 2)
    c, s = np.cos(angles), np.sin(angles)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    size[..., first] = size[..., second] = np.abs(x[..., first]) + np.abs(x[..., second])
    return y, size


def append(k, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens=None, q=None, inv_freq=None, positions=None,
           pair_axis=None, interleaved=False):
    """k, v, q [T, H, d] packed.  Returns dict(q, k_cache, v_cache, q_size, k_size): new arrays; the sizes are the sums
    of magnitudes of the rotation's terms."""
    k, v, q, kc, vc, f = (_f64(x) for x in (k, v, q, k_cache, v_cache, inv_freq))
    kc, vc = kc.copy(), vc.copy()
    ks = np.abs(kc)
    q_out, qs = (None, None) if q is None else (q.copy(), np.abs(q))
    n = 0 if f is None else f.size
    for t, _, at, page, row in places(block_table, cache_lens, kc.shape[2], kc.shape[0], cu_seqlens, k.shape[0]):
        pos = np.full(n, at, dtype=np.float64)
        if positions is not None:
            p = np.asarray(positions).reshape(-1, k.shape[0])
            axis = np.zeros(n, dtype=int) if pair_axis is None else np.clip(np.asarray(pair_axis), 0, p.shape[0] - 1)
            pos = p[axis, t].astype(np.float64)
        angle = pos * f if n else np.zeros(0)
        if q is not None:
            q_out[t], qs[t] = rotate(q[t], angle, 2 * n, interleaved)
        if page >= 0:
            kc[page, :, row], ks[page, :, row] = rotate(k[t], angle, 2 * n, interleaved)
            vc[page, :, row] = v[t]
    return dict(q=q_out, k_cache=kc, v_cache=vc, q_size=qs, k_size=ks)


def attention(q, k_cache, v_cache, block_table, cache_lens, scale, cu_seqlens=None, window=0):
    """q [T, Hq, d] packed.  Returns dict(o, size, score): size = sum of w |v| / sum of w per element, score = the
    largest scale * sum |q| |k| over the row's keys."""
    q, kc, vc = (_f64(x) for x in (q, k_cache, v_cache))
    table, lens = np.asarray(block_table), np.asarray(cache_lens)
    T, Hq, d = q.shape
    pages, Hkv, ps, _ = kc.shape
    G = Hq // Hkv
    o, size, score = np.zeros_like(q), np.zeros_like(q), np.zeros((T, Hq, 1))
    room = table.shape[1] * ps
    for t, s, at, _, _ in places(table, lens, ps, pages, cu_seqlens, T):
        first = max(0, at - window + 1) if window else 0
        keys = [j for j in range(first, min(at + 1, room, max(int(lens[s]), 0)))
                if 0 <= table[s, j // ps] < pages]
        if not keys:
            continue
        keys = np.array(keys)
        where, row = table[s, keys // ps], keys % ps
        for h in range(Hkv):
            k, v = kc[where, h, row], vc[where, h, row]
            for g in range(h * G, h * G + G):
                with np.errstate(invalid="ignore", over="ignore"):
                    x = scale * (k @ q[t, g])
                    w = np.exp(x - x.max())
                    w = w / w.sum()
                    o[t, g] = (w[:, None] * v).sum(0)
                    size[t, g] = (w[:, None] * np.abs(v)).sum(0)
                    score[t, g] = scale * (np.abs(k) @ np.abs(q[t, g])).max()
    return dict(o=o, size=size, score=score)


def beam_select(logits, scores, K, finished=None, eos=-1, pad=0):
    """Returns tokens, parents [B, K], new scores [B, K], finished [B, K]."""
    x, s = _f64(logits), _f64(scores)
    B, W, V = x.shape
    done = np.zeros((B, W), dtype=bool) if finished is None else np.asarray(finished).astype(bool)
    tokens, parents = np.full((B, K), -1), np.full((B, K), -1)
    best, over = np.full((B, K), -np.inf), np.ones((B, K), dtype=bool)
    for b in range(B):
        every = []
        for w in range(W):
            if not np.isfinite(s[b, w]):
                continue
            if done[b, w]:
                every.append((-s[b, w], w, pad))
                continue
            row = x[b, w]
            if np.isnan(row).any() or (row == np.inf).any() or (row == -np.inf).all():
                continue
            m = row.max()
            c = (s[b, w] - np.log(np.exp(row - m).sum())) + (row - m)     # m apart: it may be -1e38
            every += [(-c[v], w, v) for v in np.nonzero(row > -np.inf)[0]]
        every.sort()
        for r, (c, w, v) in enumerate(every[:K]):
            tokens[b, r], parents[b, r], best[b, r] = v, w, -c
            over[b, r] = done[b, w] or v == eos
    return tokens, parents, best, over


def reorder(state, parents):
    """state [B * W, ...], parents [B, K]: out [B * K, ...]; rows of parents outside of [0, W) are None."""
    state, parents = np.asarray(state), np.asarray(parents)
    B, K = parents.shape
    W = state.shape[0] // B
    return [state[b * W + p] if 0 <= p < W else None for b in range(B) for p in parents[b].tolist()]
