"""Float64 CPU oracle of the operators next to the step: the 4-bit matrix-vector product
and linear attention with a decay for each head. Test infrastructure only; plain loops over
the definitions, no code shared with the CUDA path."""

from __future__ import annotations

import numpy as np

Q4_0, Q4_1, Q4_K, PLANES = 2, 3, 12, 64


def planes_values(nibbles: np.ndarray, scales: np.ndarray, mins, group: int):
    """(q, scale, offset) of every value of the plane form: nibbles [rows][cols / 2] bytes,
    16 bytes per 32 values (byte i: value i low, value 16 + i high), one f16 scale (and
    offset) per `group` values; without offsets the value is scale (q - 8)."""
    rows = nibbles.shape[0]
    b = nibbles.reshape(rows, -1, 16)
    q = np.concatenate([b & 15, b >> 4], axis=-1).reshape(rows, -1).astype(np.float64)
    s = np.repeat(scales.astype(np.float64), group, axis=1)
    m = -8.0 * s if mins is None else np.repeat(mins.astype(np.float64), group, axis=1)
    return q, s, m


def block_values(rows_bytes: np.ndarray, cols: int, qtype: int):
    """(q, scale, offset) of every value of rows of Q4_0, Q4_1 or Q4_K blocks."""
    rows = rows_bytes.shape[0]
    if qtype == Q4_K:
        b = rows_bytes.reshape(rows, -1, 144)
        d = b[..., 0:2].copy().view(np.float16)[..., 0].astype(np.float64)
        dmin = b[..., 2:4].copy().view(np.float16)[..., 0].astype(np.float64)
        q = np.empty(b.shape[:2] + (8, 32))
        s = np.empty(b.shape[:2] + (8,))
        m = np.empty(b.shape[:2] + (8,))
        for j in range(8):
            p = b[..., 4:16].astype(np.int64)
            if j < 4:
                sc, mn = p[..., j] & 63, p[..., j + 4] & 63
            else:
                sc = (p[..., j + 4] & 15) | ((p[..., j - 4] >> 6) << 4)
                mn = (p[..., j + 4] >> 4) | ((p[..., j] >> 6) << 4)
            run = b[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
            q[..., j, :] = (run >> 4) if j % 2 else (run & 15)
            s[..., j], m[..., j] = d * sc, -dmin * mn
        return (q.reshape(rows, cols), np.repeat(s.reshape(rows, -1), 32, axis=1),
                np.repeat(m.reshape(rows, -1), 32, axis=1))
    size = 18 if qtype == Q4_0 else 20
    b = rows_bytes.reshape(rows, -1, size)
    d = b[..., 0:2].copy().view(np.float16)[..., 0].astype(np.float64)
    m = -8.0 * d if qtype == Q4_0 else b[..., 2:4].copy().view(np.float16)[..., 0].astype(np.float64)
    q = np.concatenate([b[..., -16:] & 15, b[..., -16:] >> 4], axis=-1).astype(np.float64)
    return q.reshape(rows, cols), np.repeat(d, 32, axis=1), np.repeat(m, 32, axis=1)


def matvec(q, s, m, x):
    """(y, a): y = W x for the rows of x [T][cols], and a, the sum of the magnitudes of the
    terms scale q x and offset x that a kernel adds up (what its roundings are relative to)."""
    x = x.astype(np.float64)
    return x @ (s * q + m).T, np.abs(x) @ (np.abs(s) * q + np.abs(m)).T


def linattn(q, k, v, g, state, scale):
    """One sequence and head: q, k [T][dk], v [T][dv], g [T], state [dk][dv] (not changed).
    Returns (o, new state, a_o, a_state), the last two with every term's magnitude summed."""
    q, k, v, g = (np.asarray(a, np.float64) for a in (q, k, v, g))
    S = np.array(state, np.float64)
    A = np.abs(S)
    o = np.zeros((len(q), S.shape[1]))
    ao = np.zeros_like(o)
    for t in range(len(q)):
        lam = np.exp(g[t])
        S = lam * S + np.outer(k[t], v[t])
        A = lam * A + np.abs(np.outer(k[t], v[t]))
        o[t] = scale * (q[t] @ S)
        ao[t] = abs(scale) * (np.abs(q[t]) @ A)
    return o, S, ao, A
