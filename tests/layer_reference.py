"""The KDA layer's operators in float64 numpy, straight from their formulas
(one request and one token at a time), with the magnitudes the tests'
tolerances are derived from."""
from __future__ import annotations

import numpy as np


def _rows(lengths, cu):
    if cu is None:
        cu = np.concatenate([[0], np.cumsum(lengths)])
    return [(int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def live_slot(slot, n, slots):
    s = n if slot is None else int(slot[n])
    return s if 0 <= s < slots else -1


def delta_rule(q, k, v, g, beta, lengths, state=None, slot=None, init=None, scale=1.0):
    """Returns (out, state, size): size = the largest 2-norm of a state column
    plus |v| entry met, the magnitude all products are bounded by."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    T, H, V = v.shape
    K, grp = k.shape[-1], H // k.shape[1]
    heads = np.arange(H) // grp
    if g.ndim == 2:
        g = np.repeat(g[:, :, None], K, axis=2)
    out = np.zeros((T, H, V))
    pool = None if state is None else np.asarray(state, np.float64).copy()
    size = 0.0
    for n, (b, e) in enumerate(_rows(lengths, None)):
        s = 0 if pool is None else live_slot(slot, n, pool.shape[0])
        if s < 0:
            continue
        cont = pool is not None and (init is None or init[n] != 0)
        S = pool[s].copy() if cont else np.zeros((H, K, V))
        size = max(size, float(np.sqrt((S ** 2).sum(1)).max(initial=0.0)))
        for t in range(b, e):
            kt, qt = k[t][heads], q[t][heads]
            S *= np.exp(g[t])[:, :, None]
            u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, kt))
            S += kt[:, :, None] * u[:, None, :]
            out[t] = scale * np.einsum("hkv,hk->hv", S, qt)
            size = max(size, float(np.sqrt((S ** 2).sum(1)).max()) + float(np.abs(v[t]).max()))
        if pool is not None:
            pool[s] = S
    return out, pool, size


def conv(qkv, conv_w, lengths, conv_state=None, slot=None, init=None, eps=1e-6):
    """Returns ([q, k, v], conv_state)."""
    x, cw = np.asarray(qkv, np.float64), np.asarray(conv_w, np.float64)
    T, _, H, d = x.shape
    W = cw.shape[1]
    y = np.zeros_like(x)
    pool = None if conv_state is None else np.asarray(conv_state, np.float64).copy()
    for n, (b, e) in enumerate(_rows(lengths, None)):
        s = 0 if pool is None else live_slot(slot, n, pool.shape[0])
        if s < 0:
            continue
        past = np.zeros((W - 1, 3, H, d))
        if pool is not None and (init is None or init[n] != 0):
            past = pool[s].transpose(2, 0, 1, 3)
        line = np.concatenate([past, x[b:e]])
        for t in range(e - b):
            a = sum(cw[:, w] * line[t + w] for w in range(W))
            a = a / (1.0 + np.exp(-a))
            for p in (0, 1):
                a[p] /= np.sqrt((a[p] ** 2).sum(-1, keepdims=True) + eps)
            y[b + t] = a
        if pool is not None:
            pool[s] = line[e - b:].transpose(1, 2, 0, 3)
    return [y[:, 0], y[:, 1], y[:, 2]], pool


def gated_norm(o, z, w, eps=1e-6):
    o, z, w = (np.asarray(x, np.float64) for x in (o, z, w))
    return o / np.sqrt((o ** 2).mean(-1, keepdims=True) + eps) * w / (1.0 + np.exp(-z))


def chunk_map(lens, total, C, rows):
    """(cu_seqlens, pairs padded with -1 or cut to `rows`, number of chunks)."""
    cu = [0]
    for n in lens:
        cu.append(min(cu[-1] + max(int(n), 0), total))
    pairs = [(r, c) for r in range(len(lens)) for c in range(-(-(cu[r + 1] - cu[r]) // C))]
    count = len(pairs)
    pairs = (pairs + [(-1, -1)] * max(0, rows - count))[:rows]
    return (np.asarray(cu, np.int32), np.asarray(pairs, np.int32).reshape(-1, 2), count)
