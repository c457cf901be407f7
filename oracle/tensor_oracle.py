"""CPU oracle of the operators on the experts' weight tensors: weights of 4 bits with
group scales, and the momentum step with an orthogonalised update.

TEST INFRASTRUCTURE ONLY, as moe_oracle: plain float64 statements; the packed form's rule is
stated in fp32 where the definition rounds there.
"""
from __future__ import annotations

import numpy as np


def w4_pack(w, axis, group):
    """q uint32 [E, out, B * 16] and scale float64 [E, out, B * 128 / group] of w [E, rows, cols]."""
    w = np.asarray(w, np.float64)
    w = np.swapaxes(w, 1, 2) if axis == 0 else w
    E, out, n = w.shape
    B = -(-n // 128)
    x = np.zeros((E, out, B * 128), np.float32)
    x[:, :, :n] = w
    x = x.reshape(E, out, -1, group)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(x).max(axis=3)  # NaN where there is one
        bad = ~(a < 2.0 ** 127)
        m, e = np.frexp((np.where(bad, 0, a) * (np.float32(1) / np.float32(7))).astype(np.float32).astype(np.float64))
        s = np.maximum(np.ldexp(np.ceil(m * 32), e - 5), 2.0 ** -126)
        m, e = np.frexp(s)  # the number of 5 significant bits below s, where the group fits it without error
        lo = s - np.ldexp(1.0, e - np.where(m > 0.5, 5, 6))
        step = lo[..., None]
        low = (lo >= 2.0 ** -126) & (7 * lo == a) & (np.rint(x / step) * step == x).all(axis=3)
        s = np.where(low, lo, s)
        q = np.rint(np.where(bad[..., None], 0, x) / s[..., None].astype(np.float32))
    s[bad] = np.nan
    code = (q.astype(np.int64) + 8).reshape(E, out, B, 4, 4, 8)  # block, run of 32, word, input
    shift = np.array([4 * (i // 2) + 16 * (i % 2) for i in range(8)])
    words = (code << shift).sum(axis=-1).astype(np.uint32)
    return np.swapaxes(words, 3, 4).reshape(E, out, B * 16), s


def w4_unpack(q, scale, axis, group, n):
    """The weights [E, rows, cols] that the packed form stands for; n: inputs of an output."""
    E, out, words = q.shape
    w = np.swapaxes(q.reshape(E, out, -1, 4, 4), 3, 4)[..., None]
    shift = np.array([4 * (i // 2) + 16 * (i % 2) for i in range(8)], np.uint32)
    code = ((w >> shift) & 15).astype(np.float64) - 8
    x = (code.reshape(E, out, -1, group) * scale[..., None]).reshape(E, out, -1)[:, :, :n]
    return np.swapaxes(x, 1, 2) if axis == 0 else x


def orthogonalize(x, steps, a, b, c, eps):
    """Newton-Schulz steps on each matrix of x [E, M, N]."""
    out = np.empty(np.shape(x), np.float64)
    for e, u in enumerate(np.asarray(x, np.float64)):
        size = np.sqrt((u ** 2).sum())
        u = u / (size + eps) if size > 0 else u * 0
        for _ in range(steps):
            A = u @ u.T if u.shape[0] <= u.shape[1] else u.T @ u
            P = b * A + c * A @ A
            u = a * u + (P @ u if u.shape[0] <= u.shape[1] else u @ P)
        out[e] = u
    return out


def muon_step(w, dw, m, beta, nesterov, lr, decay, scale, steps, a, b, c, eps):
    """(w_out, m_out, O) of a momentum step."""
    m = beta * np.asarray(m, np.float64) + dw
    o = orthogonalize(dw + beta * m if nesterov else m, steps, a, b, c, eps)
    return (1 - lr * decay) * np.asarray(w, np.float64) - lr * scale * o, m, o
