"""Bounds of the attention over the 8-bit cache that count a row's weights each by its own size, and caches whose
weights and scales lie far apart."""

from __future__ import annotations

import numpy as np

from oracle import ops_oracle as oo
from tests.kv8_cases import FEW_ROWS, HALF, LEAST, U32, types

# How far off a weight may be as an operand, relative to itself: f32 rows' have 24 bits and an exponential within 2^-22; of
# 16-bit rows' sequences of few rows one f16 rounding of a normal number (2^-11) or better; of many rows two bf16 parts,
# whose roundings are off by 2^-8 of the weight and 2^-8 of that (2^-16), and the exponential.
FEW = {"f32": 2.0 ** -21, "f16": 2.0 ** -10.9, "bf16": 2.0 ** -10.9}
MANY = 2.0 ** -15.9


def is_many(c, n):
    return c.type != "f32" and c.D <= 128 and n * (c.H // c.G) > FEW_ROWS and c.H // c.G <= 128


def rows_of(c, q, rows=1, scale=None):
    """(row, head, output, bound) for every `rows`-th row of each sequence and its last one.

    A score is off by at most (D 3/4 + 64) 2 2^-24 d, d the sum of its terms' magnitudes (products of 24-bit parts, each
    with a rounding or cut of the sum), so a weight's numerator and the sum of all by that much each; the weight by its own
    rounding as an operand, and the products' sum by one rounding a token and 64 for its parts: all relative to
    sum p |v|, whatever the weights' sizes. Weights below f32's smallest normal number (2^-126) may be 0, with
    2^16 for the references' slack. The output is rounded once."""
    q = q.reshape(c.N, c.H, c.D)
    scale = c.D ** -0.5 if scale is None else scale
    for b, (past, n) in enumerate(c.seqs):
        kv = {}
        part = MANY if is_many(c, n) else FEW[c.type]
        for i in range(n):
            if i % rows and i != n - 1:
                continue
            row, pos = int(c.offsets[b]) + i, past + i
            for h in range(c.H):
                g = h // (c.H // c.G)
                if g not in kv:
                    kv[g] = c.tokens(b, past + n, g, 0) + c.tokens(b, past + n, g, 1)[:1]
                k, held, v = kv[g]
                at = np.arange(len(k))
                seen = held & (at <= pos)
                if c.window:
                    seen &= at > pos - c.window
                want, a, d, _ = oo.attention(q[row, h], k, v, seen, scale, None if c.sinks is None else c.sinks[h])
                tol = (2 * (c.D * 3 / 4 + 64) * 2 * U32 * d + part + (seen.sum() + 64) * U32) * a
                tol = tol + seen.sum() * 2.0 ** -110 * np.abs(v[seen]).max(initial=0)
                yield row, h, want, tol + HALF[c.type] * (np.abs(want) + tol) + LEAST[c.type]


def check(c, o, q, rows=1, scale=None):
    o = np.asarray(o.double().cpu() if hasattr(o, "cpu") else o, np.float64).reshape(c.N, c.H, c.D)
    for row, h, want, tol in rows_of(c, q, rows, scale):
        err = np.abs(o[row, h] - want)
        assert np.all(err <= tol), (row, h, float(np.max(err / tol)), float(np.max(np.abs(want))), float(np.max(err)))


def dominate(c, gap, value):
    """Each sequence's first token has a score about `gap` powers of two above all others', and values of `value`
    codes, as a trained model's first token has: nearly all weight and next to no value. Returns what q has at dimension 0."""
    one = 64 if c.code == "i8" else 0x38 + 8 * 7  # 64 units of i8 and 128 of e4m3 are 1 under the cache's scales
    for g in range(c.G):
        for page in range(c.n_pages):
            c.codes_of(c.cache, page, g, 0)[:, 0] = 0
        for b in range(c.B):
            page = c.table[b, 0]
            if page >= 0:
                k, v = c.codes_of(c.cache, page, g, 0), c.codes_of(c.cache, page, g, 1)
                k[0], v[0] = 0, value
                k[0, 0] = one
    return gap * np.log(2.0) * c.D ** 0.5


def behind(c, gap, value):
    """q for such a cache, on the GPU (with the cache) and as float64."""
    import torch
    first = dominate(c, gap, value)
    c.upload()
    q = torch.from_numpy(c.rng.standard_normal((c.N, c.H, c.D))).cuda()
    q[..., 0] = first
    q = q.flatten(1).to(types()[c.type][1])
    return q, q.double().cpu().numpy()


def far_values(c, scales):
    """V's scale bytes, a page each; K says that tokens of the third page have no weight."""
    pages = c.table[0]
    for j, byte in enumerate(scales):
        c.scales_of(c.cache, pages[j], 0, 1)[:] = byte
    for j, (a, byte) in enumerate([(2, 120), (1, 120), (-127, 122), (0, 120), (1, 120)]):
        c.codes_of(c.cache, pages[j], 0, 0)[:] = (a & 255) if c.code == "i8" else abs(a) | (128 if a < 0 else 0) if a != -127 else 0xfe
        c.scales_of(c.cache, pages[j], 0, 0)[:] = byte
