"""fp64 oracle of routing by scores, the shared expert's dense product and the
AdamW step with states in 32 or 8 bits.

Written from the formulas; shares no code with the HIP path.
"""
from __future__ import annotations

import math

import numpy as np

# ----------------------------------------------------------------- routing by scores


def scores(logits, kind):
    lg = np.asarray(logits, np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-lg))
    out = np.zeros_like(lg)
    with np.errstate(invalid="ignore"):
        for t, row in enumerate(lg):
            if np.isnan(row).any() or np.isposinf(row).any():
                out[t] = np.nan
            elif not np.isneginf(row).all():
                e = np.exp(row - row.max())
                out[t] = e / e.sum()
    return out


def _rank(values):
    """Positions in falling order, NaN last, ties by position."""
    return sorted(range(len(values)), key=lambda i: (math.isnan(values[i]), -values[i] if not math.isnan(values[i]) else 0.0, i))


def route_scored(logits, k, kind="softmax", bias=None, groups=1, top_groups=1, group_best=1, renorm=True, scale=1.0):
    s = scores(logits, kind)
    T, E = s.shape
    with np.errstate(invalid="ignore"):
        c = s if bias is None else s + np.asarray(bias, np.float64)
    idx = np.zeros((T, k), np.int64)
    size = E // groups
    for t in range(T):
        allowed = range(E)
        if top_groups < groups:
            worth = []
            for g in range(groups):
                part = c[t, g * size:(g + 1) * size]
                worth.append(math.nan if np.isnan(part).any() else sum(sorted(part.tolist())[-group_best:]))
            keep = sorted(_rank(worth)[:top_groups])
            allowed = [e for g in keep for e in range(g * size, (g + 1) * size)]
        order = _rank([c[t, e] for e in allowed])
        idx[t] = [allowed[i] for i in order[:k]]
    g = gates(logits, idx, kind, renorm, scale)
    counts = np.bincount(idx.ravel(), minlength=E)
    src = np.argsort(idx.ravel(), kind="stable")
    dst = np.empty_like(src)
    dst[src] = np.arange(T * k)
    return {"topk_idx": idx, "gates": g, "counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]),
            "perm_src": src, "perm_dst": dst, "mx_blk_offsets": np.concatenate([[0], np.cumsum(-(-counts // 32))])}


def gates(logits, idx, kind, renorm=True, scale=1.0):
    """The gates of the chosen experts; k scores that sum to 0 give zeros."""
    lg = np.asarray(logits, np.float64)
    rows = np.arange(lg.shape[0])[:, None]
    s = scores(lg, kind)[rows, idx]
    if not renorm:
        return scale * s
    if kind == "softmax":  # from the chosen logits: the others' part divides out
        s = np.where(np.isnan(s), s, scores(lg[rows, idx], kind))
    tot = s.sum(1, keepdims=True)
    return scale * np.where(tot == 0, 0.0, s / np.where(tot == 0, 1.0, tot))


def route_scored_bwd(logits, idx, dgates, kind="softmax", renorm=True, scale=1.0):
    lg, dg = np.asarray(logits, np.float64), np.asarray(dgates, np.float64)
    T, E = lg.shape
    k = idx.shape[1]
    rows = np.arange(T)[:, None]
    s = scores(lg, kind)
    sk = s[rows, idx]
    ds = np.zeros((T, E))
    if renorm:
        tot = sk.sum(1)
        tot = np.where(tot == 0, np.inf, tot)[:, None, None]
        jac = np.eye(k)[None] / tot - sk[:, :, None] / tot ** 2  # d gate_j / d score_i at [j, i]
        ds[rows, idx] = scale * np.einsum("tj,tji->ti", dg, jac)
    else:
        ds[rows, idx] = scale * dg
    if kind == "sigmoid":
        return ds * s * scores(-lg, kind)
    return s * (ds - (ds * s).sum(1, keepdims=True))


def bias_update(counts, bias, rate):
    n = np.asarray(counts, np.int64)
    n = n.sum(0) if n.ndim == 2 else n
    return np.asarray(bias, np.float64) + rate * np.sign(int(n.sum()) - len(n) * n)


# ----------------------------------------------------------------- dense product

_ERF = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _ERF(z / math.sqrt(2.0)))
    return z


def dact(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + _ERF(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def linear(x, w, bias=None, name="none", residual=None):
    """y and z, and the sums of the absolute terms of z (for error bounds)."""
    z = x @ w + (0.0 if bias is None else bias)
    y = act(z, name) + (0.0 if residual is None else residual)
    return y, z, np.abs(x) @ np.abs(w) + (0.0 if bias is None else np.abs(bias))


def linear_bwd(dy, x, w, z=None, name="none", in_z=None, in_name="none", dres=None):
    """dx, dw, db, and the sums of the absolute terms of each."""
    dz = dy if name == "none" else dy * dact(z, name)
    inner = 1.0 if in_name == "none" else dact(in_z, in_name)
    dx = (dz @ w.T) * inner + (0.0 if dres is None else dres)
    a = np.abs(dz)
    return dx, x.T @ dz, dz.sum(0), (a @ np.abs(w).T) * np.abs(inner), np.abs(x).T @ a, a.sum(0)


# ----------------------------------------------------------------- AdamW

def mix(h):
    h = np.asarray(h, np.uint64) & np.uint64(0xFFFFFFFF)
    for shift, mul in ((16, 0x7FEB352D), (15, 0x846CA68B), (16, 1)):
        h = ((h ^ (h >> np.uint64(shift))) * np.uint64(mul)) & np.uint64(0xFFFFFFFF)
    return h


def random_halves(seed, tensor, step, n):
    """High and low 16 bits of the hash of every element."""
    gold = 0x9E3779B9
    key = int(mix((int(mix((seed + gold * tensor) % 2 ** 32)) + gold * step) % 2 ** 32))
    h = mix((np.arange(n, dtype=np.uint64) * np.uint64(gold) + np.uint64(key)) & np.uint64(0xFFFFFFFF))
    return (h >> np.uint64(16)).astype(np.int64), (h & np.uint64(0xFFFF)).astype(np.int64)


def e4m3(code):
    """The value of an E4M3 code (no NaN codes are used)."""
    code = np.asarray(code, np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e.astype(np.float64) - 10))
    return np.where(code & 128, -v, v)


GRID = e4m3(np.arange(127))  # 0 .. 448


def encode(x, r, root=False):
    """Codes [32 n] and bytes [n] of blocks of 32: rounded up where the place between two codes plus (r + 1/2) / 2^16
    reaches 1."""
    b = np.asarray(x, np.float64).reshape(-1, 32)
    codes, byte = np.zeros(b.shape, np.int64), np.zeros(len(b), np.int64)
    r = (np.asarray(r, np.float64).reshape(-1, 32) + 0.5) / 65536
    for n, row in enumerate(b):
        if not np.isfinite(row).all():
            byte[n] = 255
            continue
        e = -127
        while np.abs(row).max() > 448 * 2.0 ** e:
            e += 1
        byte[n] = e + 127
        y = np.abs(row) * 2.0 ** -e
        lo = np.searchsorted(GRID, y, side="right") - 1
        hi = np.minimum(lo + 1, 126)
        gap = np.where(hi > lo, GRID[hi] - GRID[lo], 1.0)
        c = np.where((y - GRID[lo]) / gap + r[n] >= 1.0, hi, lo)
        if root:
            c = np.where((c == 0) & (y > 0), 1, c)
        else:
            c = c | np.where(np.signbit(row), 128, 0)
        codes[n] = c
    return codes.reshape(-1), byte


def decode(codes, byte):
    s = np.where(np.asarray(byte) == 255, np.nan, np.exp2(np.asarray(byte, np.float64) - 127))
    return (e4m3(codes).reshape(-1, 32) * s[:, None]).reshape(-1)


def adamw(w, g, m, v, lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, grad_scale=1.0):
    """w', m', v' of one tensor."""
    w, g, m, v = (np.asarray(a, np.float64) for a in (w, g, m, v))
    # numbers of 64 bits: an np.float32 among them would round 1 - lr weight_decay to 32
    lr, b1, b2, eps, weight_decay, grad_scale = map(float, (lr, *betas, eps, weight_decay, grad_scale))
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = (1 - lr * weight_decay) * w - lr * (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return w, m, v
