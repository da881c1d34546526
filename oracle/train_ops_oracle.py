"""fp64 oracle of the operators around the layer: layer norm, the router's
balance and z losses, and the orthogonalised weight update (Muon).

Written from the formulas; shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

QUINTIC = (float(np.float32(3.4445)), float(np.float32(-4.7750)), float(np.float32(2.0315)))


# ----------------------------------------------------------------- layer norm

def layernorm(s, w=None, b=None, eps=1e-5):
    s = np.asarray(s, np.float64)
    mu = s.mean(1)
    rstd = 1.0 / np.sqrt(((s - mu[:, None]) ** 2).mean(1) + eps)
    y = (s - mu[:, None]) * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mu, rstd


def layernorm_bwd(dy, s, w=None, eps=1e-5, dres=None):
    """dx, dw, db, and the sums of the absolute terms of dw and db (for error bounds)."""
    dy, s = np.asarray(dy, np.float64), np.asarray(s, np.float64)
    _, mu, rstd = layernorm(s, eps=eps)
    h = (s - mu[:, None]) * rstd[:, None]
    v = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd[:, None] * (v - v.mean(1, keepdims=True) - h * (v * h).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * h).sum(0), dy.sum(0), np.abs(dy * h).sum(0), np.abs(dy).sum(0)


# ----------------------------------------------------------------- balance loss

def counted_rows(logits, seq, mask):
    """Token indices of each sequence that count."""
    T = logits.shape[0]
    seq = [0, T] if seq is None else [int(v) for v in seq]
    rows = []
    for lo, hi in zip(seq[:-1], seq[1:]):
        r = np.arange(lo, max(lo, hi))
        if mask is not None:
            r = r[np.asarray(mask)[r] != 0]
        rows.append(r[~np.all(np.isneginf(logits[r]), axis=1)])
    return rows


def balance_loss(logits, idx, alpha, zeta, seq=None, mask=None, counts=None):
    """loss [2], counts, probs, lse.  Given ``counts`` the loss uses those (its gradient treats them as constants)."""
    lg = np.asarray(logits, np.float64)
    T, E = lg.shape
    k = idx.shape[1]
    rows = counted_rows(lg, seq, mask)
    S = len(rows)
    cnt = np.zeros((S, E), np.int64)
    probs = np.zeros((S, E))
    lse = np.zeros(T)
    bal = z = 0.0
    live, n_all = sum(len(r) > 0 for r in rows), sum(len(r) for r in rows)
    for s, r in enumerate(rows):
        if len(r) == 0:
            continue
        m = lg[r].max(1, keepdims=True)
        ex = np.exp(lg[r] - m)
        tot = ex.sum(1, keepdims=True)
        probs[s] = (ex / tot).mean(0)
        lse[r] = (m + np.log(tot))[:, 0]
        cnt[s] = np.bincount(np.asarray(idx)[r].ravel(), minlength=E)
        c = cnt[s] if counts is None else counts[s]
        bal += alpha * E / live * float((c / (k * len(r)) * probs[s]).sum())
        z += zeta / n_all * float((lse[r] ** 2).sum())
    return np.array([bal, z]), cnt, probs, lse


def balance_loss_bwd(logits, idx, alpha, zeta, seq=None, mask=None, dloss=(1.0, 1.0), gates=None, dgates=None):
    lg = np.asarray(logits, np.float64)
    T, E = lg.shape
    k = idx.shape[1]
    rows = counted_rows(lg, seq, mask)
    _, cnt, _, lse = balance_loss(logits, idx, alpha, zeta, seq, mask)
    live, n_all = sum(len(r) > 0 for r in rows), sum(len(r) for r in rows)
    dl = np.zeros((T, E))
    for s, r in enumerate(rows):
        if len(r) == 0:
            continue
        p = np.exp(lg[r] - lg[r].max(1, keepdims=True))  # not from lse, whose rounding loses log E at the lowest logits
        p /= p.sum(1, keepdims=True)
        a = dloss[0] * alpha * E * cnt[s] / (k * len(r) ** 2 * live)
        dl[r] = p * (a - (p * a).sum(1, keepdims=True)) + dloss[1] * 2 * zeta / n_all * lse[r][:, None] * p
    if gates is not None:
        g, dg = np.asarray(gates, np.float64), np.asarray(dgates, np.float64)
        part = g * (dg - (g * dg).sum(1, keepdims=True))
        np.add.at(dl, (np.arange(T)[:, None], np.asarray(idx)), part)
    return dl


# ----------------------------------------------------------------- orthogonalised update

def orthogonalize(g, steps=5, coef=None, eps=1e-7):
    """Newton-Schulz iteration of each matrix of g [E, rows, cols]."""
    out = np.empty(np.shape(g), np.float64)
    for e, m in enumerate(np.asarray(g, np.float64)):
        tall = m.shape[0] > m.shape[1]
        x = m.T if tall else m
        n = np.sqrt((x * x).sum())
        x = x / (n + eps) if n > 0 else x
        for i in range(steps):
            a, b, c = QUINTIC if coef is None else coef[i]
            gram = x @ x.T
            x = a * x + (b * gram + c * (gram @ gram)) @ x
        out[e] = x.T if tall else x
    return out


def muon_step(g, mom, w, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=1.0, steps=5, coef=None, eps=1e-7):
    g, mom, w = (np.asarray(v, np.float64) for v in (g, mom, w))
    m2 = momentum * mom + g
    u = g + momentum * m2 if nesterov else m2
    o = orthogonalize(u, steps, coef, eps)
    return (1.0 - lr * weight_decay) * w - lr * scale * o, m2, o
