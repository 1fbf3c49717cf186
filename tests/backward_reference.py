"""Gradients of the KDA layer's operators in float64 numpy, straight from the
recurrences (one request and one token at a time), and the values that an 8-bit
checkpoint stands for."""
from __future__ import annotations

import numpy as np

from tests.layer_reference import _rows, live_slot


def delta_rule_grad(dout, q, k, v, g, beta, lengths, state=None, dstate=None, slot=None,
                    init=None, scale=1.0):
    """Returns dict(dq, dk, dv, dg, dbeta) and the pool of state gradients
    (None without dstate)."""
    dout, q, k, v, g, beta = (np.asarray(x, np.float64) for x in (dout, q, k, v, g, beta))
    T, H, V = v.shape
    Hk, K = q.shape[1:]
    heads = np.arange(H) // (H // Hk)
    per_channel = g.ndim == 3
    a = np.exp(g if per_channel else np.repeat(g[:, :, None], K, axis=2))
    out = dict(dq=np.zeros((T, H, K)), dk=np.zeros((T, H, K)), dv=np.zeros((T, H, V)),
               dg=np.zeros((T, H, K)), dbeta=np.zeros((T, H)))
    pool = None if state is None else np.asarray(state, np.float64)
    dpool = None if dstate is None else np.asarray(dstate, np.float64).copy()
    slots = (pool if pool is not None else dpool)
    for n, (b, e) in enumerate(_rows(lengths, None)):
        s = 0 if slots is None else live_slot(slot, n, slots.shape[0])
        if s < 0:
            continue
        cont = init is None or init[n] != 0
        S = pool[s].copy() if pool is not None and cont else np.zeros((H, K, V))
        kept = []
        for t in range(b, e):
            kt = k[t][heads]
            mid = S * a[t][:, :, None]
            r = v[t] - np.einsum("hkv,hk->hv", mid, kt)
            S = mid + kt[:, :, None] * (beta[t][:, None] * r)[:, None, :]
            kept.append((mid, r, S))
        dS = dpool[s].copy() if dpool is not None else np.zeros((H, K, V))
        for t in reversed(range(b, e)):
            mid, r, S = kept.pop()
            kt, qt, do = k[t][heads], q[t][heads], scale * dout[t]
            out["dq"][t] = np.einsum("hkv,hv->hk", S, do)
            dS = dS + qt[:, :, None] * do[:, None, :]
            u = beta[t][:, None] * r
            du = np.einsum("hkv,hk->hv", dS, kt)
            dr = beta[t][:, None] * du
            out["dk"][t] = np.einsum("hkv,hv->hk", dS, u) - np.einsum("hkv,hv->hk", mid, dr)
            out["dbeta"][t] = (du * r).sum(-1)
            out["dv"][t] = dr
            dS = dS - kt[:, :, None] * dr[:, None, :]
            out["dg"][t] = (dS * mid).sum(-1)
            dS = a[t][:, :, None] * dS
        if dpool is not None:
            dpool[s] = dS if cont else 0.0
    for x in ("dq", "dk"):
        out[x] = out[x].reshape(T, Hk, H // Hk, K).sum(2)
    if not per_channel:
        out["dg"] = out["dg"].sum(-1)
    return out, dpool


def conv_grad(dq, dk, dv, qkv, conv_w, lengths, conv_state=None, dconv_state=None, slot=None,
              init=None, eps=1e-6):
    """Returns (dqkv, dconv_w, pool of window gradients)."""
    x, cw = np.asarray(qkv, np.float64), np.asarray(conv_w, np.float64)
    T, _, H, d = x.shape
    W = cw.shape[1]
    dn = np.stack([np.asarray(t, np.float64) for t in (dq, dk, dv)], 1)
    dx, dcw = np.zeros_like(x), np.zeros_like(cw)
    pool = None if conv_state is None else np.asarray(conv_state, np.float64)
    dpool = None if dconv_state is None else np.asarray(dconv_state, np.float64).copy()
    slots = pool if pool is not None else dpool
    for n, (b, e) in enumerate(_rows(lengths, None)):
        s = 0 if slots is None else live_slot(slot, n, slots.shape[0])
        if s < 0:
            continue
        cont = init is None or init[n] != 0
        past = np.zeros((W - 1, 3, H, d))
        if pool is not None and cont:
            past = pool[s].transpose(2, 0, 1, 3)
        line = np.concatenate([past, x[b:e]])
        dline = np.zeros_like(line)
        if dpool is not None:
            dline[e - b:] += dpool[s].transpose(2, 0, 1, 3)
        for t in range(e - b):
            a = sum(cw[:, w] * line[t + w] for w in range(W))
            sg = 1.0 / (1.0 + np.exp(-a))
            y, dy = a * sg, dn[b + t].copy()
            for p in (0, 1):
                r = 1.0 / np.sqrt((y[p] ** 2).sum(-1, keepdims=True) + eps)
                u = y[p] * r
                dy[p] = r * (dy[p] - u * (u * dy[p]).sum(-1, keepdims=True))
            da = dy * sg * (1.0 + a * (1.0 - sg))
            for w in range(W):
                dline[t + w] += cw[:, w] * da
                dcw[:, w] += da * line[t + w]
        dx[b:e] = dline[W - 1:]
        if dpool is not None:
            dpool[s] = dline[:W - 1].transpose(1, 2, 0, 3) if cont else 0.0
    return dx, dcw, dpool


def gated_norm_grad(dout, o, z, w, eps=1e-6):
    """Returns (do, dz, dw)."""
    dout, o, z, w = (np.asarray(x, np.float64) for x in (dout, o, z, w))
    r = 1.0 / np.sqrt((o ** 2).mean(-1, keepdims=True) + eps)
    n, s = o * r, 1.0 / (1.0 + np.exp(-z))
    rest = 1.0 / (1.0 + np.exp(z))  # 1 - s, of which 16 digits would be lost where s is 1
    dn = dout * w * s
    do = r * (dn - n * (dn * n).mean(-1, keepdims=True))
    return do, dout * w * n * s * rest, (dout * n * s).reshape(-1, len(w)).sum(0)


def checkpoint(x):
    """(codes, scale) of vectors x [.., d] (finite): scale in float32, the division
    and the rounding to the nearest even integer exact."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1)
    scale = (top / 127.0).astype(np.float32)
    scale[top < 2.0 ** -110] = 0.0
    step = scale.astype(np.float64)[..., None]
    codes = np.where(step > 0, np.rint(x / np.where(step > 0, step, 1.0)), 0.0)
    return codes.astype(np.int8), scale
