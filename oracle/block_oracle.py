"""CPU oracle of the operators around the expert products: the gate with expert
groups, the combine fused with its norms, and the 8-bit activation checkpoint.

TEST INFRASTRUCTURE ONLY, as moe_oracle: plain float64 statements, nothing
rounded inside except where the definition rounds (the checkpoint's integers).
"""
from __future__ import annotations

import math

import numpy as np


def _scores(logits, sigmoid):
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(axis=1, keepdims=True)
        e = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(m), 0.0, m)))
        z = e.sum(axis=1, keepdims=True)
        return np.divide(e, z, out=np.zeros_like(e), where=z != 0)


def _shares(logits, sigmoid):
    """The chosen scores over their sum, which a common factor leaves alone: by their logarithms, so that
    scores below the smallest number have their shares too; 0 where all are out of service."""
    l = np.asarray(logits, np.float64)
    log_s = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l))) if sigmoid else l
    top = log_s.max()
    if np.isneginf(top):
        return np.zeros_like(l)
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.exp(log_s - top)
    return w / w.sum()


def gate_group(logits, K, groups, topk_groups, sigmoid=False, bias=None, renorm=False, group_max=False, scale=1.0):
    """idx [T,K] and gate [T,K] of the group-limited gate, one row at a time.

    c = s + bias (without a bias the logits, in the same order); a group ranks by
    its two largest scores (its largest with group_max), experts at -inf counting
    for nothing; Python's stable sort leaves equal values in index order."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    n = E // groups
    s = _scores(l, sigmoid)
    ident = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    idx = np.zeros((T, K), np.int32)
    for t in range(T):
        out = np.isneginf(l[t]) | np.isnan(l[t])
        c = l[t].copy() if bias is None else s[t] + ident
        c[out | np.isnan(c)] = -np.inf
        of_groups = c if bias is not None or group_max else np.where(np.isneginf(c), -np.inf, s[t])
        ranks = []
        for g in range(groups):
            best = sorted(of_groups[g * n:(g + 1) * n], reverse=True)
            two = not group_max and n > 1 and best[1] != -np.inf
            ranks.append(best[0] + best[1] if two else best[0])
        kept = sorted(range(groups), key=lambda g: (-ranks[g], g))[:topk_groups]
        allowed = sorted(e for g in kept for e in range(g * n, (g + 1) * n))
        idx[t] = sorted(allowed, key=lambda e: (-c[e], e))[:K]
    gate = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if renorm:
        gate = np.stack([_shares(l[t, idx[t]], sigmoid) for t in range(T)]) if T else gate
    gate = scale * gate
    gate[np.isnan(l).any(axis=1)] = np.nan
    return idx, gate


def gate_group_bwd(d_gate, logits, idx, sigmoid=False, renorm=False, scale=1.0):
    """d_logits of gate_group's gates, by the chain rule through the scores."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    K = idx.shape[1]
    s = _scores(l, sigmoid)
    d = np.zeros((T, E))
    for t in range(T):
        if renorm:
            q = _shares(l[t, idx[t]], sigmoid)
            inner = sum(d_gate[t, k] * q[k] for k in range(K))
            for k, e in enumerate(idx[t]):
                d[t, e] += scale * q[k] * (d_gate[t, k] - inner) * (1 - s[t, e] if sigmoid else 1)
            continue
        ds = np.zeros(E)
        for k, e in enumerate(idx[t]):
            ds[e] += scale * d_gate[t, k]
        d[t] = ds * s[t] * (1 - s[t]) if sigmoid else s[t] * (ds - ds @ s[t])
    return d


def rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)


def combine_norm(h, gate, dst_row, K, eps, row_scale=None, residual=None, w_post=None, res_scale=None, w_next=None):
    """y and xn (None without w_next): combine, norm after the block, gate and
    residual scale, residual, norm before the next block."""
    if h is None:
        y = np.array(residual, np.float64)
    else:
        T, H = len(h) // K, h.shape[1]
        rows = np.arange(T * K) if dst_row is None else np.asarray(dst_row, np.int64)
        g = np.ones((T, K)) if gate is None else gate
        n = np.zeros((T, H))
        for k in range(K):
            n += g[:, k:k + 1] * h[rows.reshape(T, K)[:, k]]
        if w_post is not None:
            n = n * rms(n, eps) * w_post
        if res_scale is not None:
            n = n * res_scale
        if row_scale is not None:
            n = n * np.asarray(row_scale)[:, None]
        y = n if residual is None else residual + n
    return y, None if w_next is None else y * rms(y, eps) * w_next


def rms_bwd(d, x, eps):
    """Gradient of x * rms(x) against d."""
    q = rms(x, eps)
    return q * d - q ** 3 * x * (d * x).mean(axis=1, keepdims=True)


def combine_norm_bwd(dy, dxn, h, gate, dst_row, K, eps, y, row_scale=None, w_post=None, res_scale=None, w_next=None):
    """Gradients of combine_norm, the norm before the next block taken at y."""
    out = {}
    D = np.zeros(0)
    if dy is not None:
        D = np.array(dy, np.float64)
    if w_next is not None:
        out["dw_next"] = (dxn * y * rms(y, eps)).sum(axis=0)
        more = rms_bwd(dxn * w_next, y, eps)
        D = more if dy is None else D + more
    out["d_res"] = D
    if h is None:
        return out
    T, H = D.shape
    rows = (np.arange(T * K) if dst_row is None else np.asarray(dst_row, np.int64)).reshape(T, K)
    g = np.ones((T, K)) if gate is None else gate
    z = sum(g[:, k:k + 1] * h[rows[:, k]] for k in range(K))
    u = z * rms(z, eps) if w_post is not None else z
    one = np.ones(H)
    w = one if w_post is None else w_post
    a = one if res_scale is None else res_scale
    s = np.ones(T) if row_scale is None else np.asarray(row_scale)
    out["d_scale"] = (D * a * w * u).sum(axis=1)
    out["d_res_scale"] = (s[:, None] * D * w * u).sum(axis=0)
    out["dw_post"] = (s[:, None] * D * a * u).sum(axis=0)
    P = s[:, None] * a * w * D
    dz = rms_bwd(P, z, eps) if w_post is not None else P
    out["dz"] = dz
    out["dh"] = np.zeros_like(h)
    out["d_gate"] = np.zeros((T, K))
    for k in range(K):
        out["dh"][rows[:, k]] = g[:, k:k + 1] * dz
        out["d_gate"][:, k] = (dz * h[rows[:, k]]).sum(axis=1)
    return out


def ckpt_pack(x, run=32):
    """q int8 [rows, N] and scale uint8 [rows, ceil(N/run)] of the checkpoint."""
    x = np.asarray(x, np.float64)
    rows, N = x.shape
    runs = -(-N // run)
    q = np.zeros((rows, N), np.int8)
    scale = np.zeros((rows, runs), np.uint8)
    for r in range(rows):
        for b in range(runs):
            v = x[r, b * run:(b + 1) * run]
            if not np.isfinite(v).all():
                scale[r, b] = 255
                continue
            a = np.abs(v).max()
            e = -126
            if a > 127 * 2.0 ** -126:
                e = max(-126, math.frexp(a)[1] - 8)  # a < 2^(e+8): below the answer, so count up to it
                while 127 * 2.0 ** e < a:
                    e += 1
            scale[r, b] = e + 127
            q[r, b * run:(b + 1) * run] = np.rint(v / 2.0 ** e)  # numpy rounds halves to even
    return q, scale


def ckpt_unpack(q, scale, run=32):
    s = np.repeat(np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127)), run, axis=1)
    return q.astype(np.float64) * s[:, :q.shape[1]]
