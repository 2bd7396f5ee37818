"""The bounds of tests/kv8_bounds.py take right outputs and refuse wrong ones (on the CPU)."""

import numpy as np
import pytest

from oracle import ops_oracle as oo
from tests.kv8_bounds import check, dominate, far_values, rows_of
from tests.kv8_cases import Cache

torch = pytest.importorskip("torch")
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}


def rows(c, first):
    q = c.rng.standard_normal((c.N, c.H, c.D))
    q[..., 0] = first
    return torch.from_numpy(q.reshape(c.N, -1)).to(TORCH[c.type]).double().numpy()


def outputs(c, q, weights):
    """All rows with their weights (relative to the largest) as `weights` rounds them, rounded to the type."""
    o = np.zeros((c.N, c.H, c.D))
    for i in range(c.N):
        for h in range(c.H):
            g = h // (c.H // c.G)
            k, v = (c.tokens(0, c.seqs[0][0] + i + 1, g, w)[0] for w in (0, 1))
            s = c.D ** -0.5 * (k @ q.reshape(c.N, c.H, c.D)[i, h])
            w = np.exp(s - s.max())
            o[i, h] = weights(w) @ v / w.sum()
    return torch.from_numpy(o).to(TORCH[c.type]).double().numpy()


def f16_of(w):
    return (w * 8).astype(np.float16).astype(np.float64) / 8


def two_parts(w):
    hi = torch.from_numpy(w).to(torch.bfloat16).double()
    return (hi + (torch.from_numpy(w) - hi).to(torch.bfloat16).double()).numpy()


@pytest.mark.parametrize("type", list(TORCH))
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_dominant_token(type, code):
    """Weights whose bits go by their own size pass; f16 numbers times 2^3 below a dominant token's do not."""
    c = Cache([(0, 150)], H=2, G=1, D=64, type=type, code=code, spread=0.0, seed=21)
    q = rows(c, dominate(c, 27, 0))
    check(c, outputs(c, q, lambda w: w), q, rows=7)
    check(c, outputs(c, q, two_parts), q, rows=7)
    for wrong in (outputs(c, q, f16_of), np.zeros((c.N, c.H, c.D))):
        with pytest.raises(AssertionError):
            check(c, wrong, q, rows=7)


@pytest.mark.parametrize("type", list(TORCH))
@pytest.mark.parametrize("scales", [(20, 121, 150, 121, 90), (60, 30, 180, 130, 30)])
def test_scales_far_apart(type, scales):
    """An output of 0, or of something for rows that see small values only, is refused."""
    c = Cache([(0, 80)], H=2, G=1, D=64, page=16, block=16, type=type, seed=12)
    far_values(c, scales)
    q = np.full((c.N, 128), 2.0)
    good = np.zeros((c.N, c.H, c.D))
    for row, h, want, _ in rows_of(c, q):
        good[row, h] = want
    good = torch.from_numpy(good).to(TORCH[type]).double().numpy()
    check(c, good, q)
    for lo, hi in ((0, 16), (16, 32), (48, 80)):  # rows that see no large value, or with next to no weight
        for wrong in (0.0, good[lo:hi] * 1.02):
            if type == "f16" and np.abs(good[lo:hi]).max() < 2.0 ** -20:
                continue  # (what f16 has no numbers for)
            bad = good.copy()
            bad[lo:hi] = wrong
            with pytest.raises(AssertionError):
                check(c, bad, q)
