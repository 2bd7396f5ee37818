"""Attention over the 8-bit cache at the ends of its numbers: rows of q and keys whose sizes are far from 1 and whose
scores are not, keys far apart, scales of 2^-127, positions far behind the table. Bounds: tests/kv8_bounds.py."""

import numpy as np
import pytest

from tests.kv8_bounds import check, rows_of
from tests.kv8_cases import Cache, types

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]


def keys_at(c, byte):
    """All scales of K, with a spread of a few powers of two."""
    for g in range(c.G):
        for p in range(c.n_pages):
            s = c.scales_of(c.cache, p, g, 0)
            s[:] = np.clip(byte + c.rng.integers(-1, 2, s.shape), 0, 254)


@pytest.mark.parametrize("type,power", [("bf16", 100), ("bf16", 121), ("f32", 100), ("f32", 121), ("bf16", -100), ("f32", -100),
                                        ("bf16", -120), ("f32", -120), ("f16", 12), ("f16", -12)])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("step", [True, False])
def test_factors_far_from_1(type, power, code, step):
    """q of 2^power, K of about 2^-power (from scale bytes of 0 on): scores of a few units, as for sizes around 1."""
    c = Cache([(300, 1), (40, 1)] if step else [(200, 90), (0, 70)], D=64, type=type, code=code, seed=41)
    keys_at(c, (121 if code == "i8" else 120) - power)
    c.upload()
    q, _ = c.rows(c.H * c.D, 2.0 ** power)
    check(c, c.attend(q, step=step), q.double().cpu().numpy(), rows=11)


@pytest.mark.parametrize("type", ["bf16", "f32"])
@pytest.mark.parametrize("step", [True, False])
def test_a_scale_of_0_is_no_zero(type, step):
    """Byte 0 stands for 2^-127 in K as well."""
    c = Cache([(200, 1)] if step else [(100, 80)], D=64, type=type, seed=42)
    for g in range(c.G):
        for p in range(c.n_pages):
            c.scales_of(c.cache, p, g, 0)[:] = 0
    c.upload()
    q, _ = c.rows(c.H * c.D, 2.0 ** 119)
    o = c.attend(q, step=step)
    check(c, o, q.double().cpu().numpy(), rows=11)
    assert not torch.equal(o, c.attend(q * 0, step=step))


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("window", [0, 16])
@pytest.mark.parametrize("bytes", [(121, 165, 119, 122, 120), (120, 120, 0, 120, 1), (119, 180, 100, 121, 120), (121, 121, 148, 121, 142)])
def test_keys_far_apart(type, code, window, bytes):
    """A row's scores do not depend on keys that it does not see, whatever their size."""
    c = Cache([(0, 80), (300, 70)], H=4, G=2, D=64, page=16, block=16, type=type, code=code, window=window, seed=43)
    for g in range(c.G):
        for j, byte in enumerate(bytes):
            for page in (c.table[0, j], c.table[1, 16 + j]):
                c.scales_of(c.cache, page, g, 0)[:] = byte
    c.upload()
    q, qd = c.rows(c.H * c.D)
    check(c, c.attend(q), qd)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("past", [2 ** 30 - 100, 2 ** 30, 2 ** 30 + 5, 2 ** 31 - 1])
@pytest.mark.parametrize("window", [0, 16, 2 ** 30 - 150, 2 ** 30 + 2, 2 ** 30 + 2 ** 28, 2 ** 30 + 2 ** 28 + 1, 2 ** 31 - 5, 2 ** 31 - 1])
def test_positions_far_behind_the_table(type, past, window):
    """A row at position p sees the held positions from p - window + 1 on, as one at position 1000 does with that first one."""
    c = Cache([(0, 200), (40, 70)], H=4, G=2, D=64, page=16, block=4, type=type, window=window, seed=44).upload()
    q, _ = c.rows(c.H * c.D)
    first = past - window + 1 if window else None
    c.d_past[:] = past
    o = c.attend(q)
    if first is not None and first > 1000:
        assert not o.any()
        return
    c.d_past[:] = 1000
    c.window = 1001 - first if window else 0
    want = c.attend(q)
    assert torch.equal(o, want) and (want[0] != 0).any() == (first is None or first < 208)


def test_f32_sums_have_no_bias():
    """Sums of positive values, each rounded to nearest: what the roundings leave on average over 10^5 outputs is far below one of
    them (2^-24). A sum that is cut at each step is off by steps / 2 times that, always down; the bound is four roundings."""
    c = Cache([(961, 214), (0, 551), (5840, 754)], H=16, G=1, D=64, type="f32", seed=45)
    for p in range(c.n_pages):
        codes = c.codes_of(c.cache, p, 0, 1)
        codes[:] = np.maximum(codes & 127, 1)
    c.upload()
    q, qd = c.rows(c.H * c.D)
    o = c.attend(q)
    check(c, o, qd, rows=17)
    o = o.double().cpu().numpy().reshape(c.N, c.H, c.D)
    off = [(o[row, h] / want - 1).mean() for row, h, want, _ in rows_of(c, qd, rows=17)]
    assert len(off) * c.D > 9e4 and abs(np.mean(off)) <= 2.0 ** -22
