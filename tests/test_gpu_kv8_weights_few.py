"""As tests/test_gpu_kv8_weights.py, for single tokens and short parts of prompts."""

import pytest

from tests.kv8_bounds import behind, check
from tests.kv8_cases import Cache

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gap,value", [(12, 0), (19, 0), (27, 0), (27, 1), (45, 0), (90, 0)])
def test_steps_behind_a_dominant_token(type, code, D, gap, value):
    """The first token shares its scale with others of its block, so the scale says nothing of its value."""
    c = Cache([(0, 1), (40, 1), (1500, 1), (3000, 1)], H=8, G=2, D=D, type=type, code=code, spread=0.0, seed=32)
    q, qd = behind(c, gap, value)
    check(c, c.attend(q, step=True), qd)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("H", [4, 16])
def test_short_parts_behind_a_dominant_token(type, H):
    """A few tokens behind a long cache: eights and sixteens of rows."""
    c = Cache([(1000, 12), (500, 3), (0, 2)], H=H, G=4, D=128, type=type, spread=0.0, window=800, seed=33)
    q, qd = behind(c, 25, 0)
    check(c, c.attend(q), qd)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("scale", [-0.125, 0.0, 1.5])
def test_steps_of_any_factor(type, scale):
    c = Cache([(300, 1), (40, 1), (2000, 1)], D=64, type=type, seed=34).upload()
    q, qd = c.rows(c.H * c.D)
    check(c, c.attend(q, step=True, cfg=c.cfg(scale=scale)), qd, rows=11, scale=scale)
