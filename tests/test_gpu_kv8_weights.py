"""Attention over the 8-bit cache where nearly all weight is on tokens of next to no value: the others' weights
keep their bits whatever their size. Bounds: tests/kv8_bounds.py, relative to sum p |v|."""

import numpy as np
import pytest

from tests.kv8_bounds import behind, check, far_values, rows_of
from tests.kv8_cases import Cache, types

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gap,value", [(12, 0), (19, 0), (27, 0), (27, 1), (45, 0), (90, 0)])
def test_prompts_behind_a_dominant_token(type, code, D, gap, value):
    c = Cache([(0, 300), (0, 1), (900, 70)], H=8, G=2, D=D, type=type, code=code, spread=0.0, sinks=D == 128, seed=31)
    q, qd = behind(c, gap, value)
    check(c, c.attend(q), qd, rows=17)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("scales", [(20, 121, 150, 121, 90), (60, 30, 180, 130, 30), (200, 150, 120, 60, 121), (30, 60, 90, 120, 150)])
def test_values_far_apart(type, code, step, scales):
    """A token's value reaches the rows that see it, whatever the values that others see."""
    c = Cache([(79, 1)] if step else [(0, 80)], H=2, G=1, D=64, page=16, block=16, type=type, code=code, seed=12)
    far_values(c, scales)
    c.upload()
    q = torch.full((c.N, 128), 2.0, dtype=types()[type][1], device="cuda")
    if type == "f16" and max(scales) > 140:  # (values beyond f16)
        o = c.attend(q, step=step).double().cpu().numpy().reshape(c.N, c.H, c.D)
        for row, h, want, tol in rows_of(c, q.double().cpu().numpy()):
            if abs(want).max() < 60000:
                assert (abs(o[row, h] - want) <= tol).all(), (row, h)
        return
    check(c, c.attend(q, step=step), q.double().cpu().numpy())


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("scale", [-0.125, 0.0, 1.5])
def test_prompts_of_any_factor(type, scale):
    c = Cache([(200, 90), (0, 150)], D=64, type=type, seed=34).upload()
    q, qd = c.rows(c.H * c.D)
    check(c, c.attend(q, cfg=c.cfg(scale=scale)), qd, rows=11, scale=scale)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("rise", [0, 14, 38])
def test_sinks_far_above(type, rise):
    """A sink of 2^100 times all tokens' weight, where the later tokens' scores are `rise` powers of two above the first ones'."""
    c = Cache([(0, 290)] * 40, H=4, G=2, D=64, type=type, sinks=True, spread=0.0, seed=35)  # (several groups a CTA)
    for g in range(c.G):
        for page in range(c.n_pages):
            c.codes_of(c.cache, page, g, 0)[:, 0] = 0
        for b in range(c.B):
            for page in c.table[b, 2:]:
                if page >= 0:
                    c.codes_of(c.cache, page, g, 0)[:, 0] = 64
    c.sinks[:] = (100 + rise) * np.log(2.0)
    c.upload()
    q = torch.from_numpy(c.rng.standard_normal((c.N, c.H, c.D))).cuda()
    q[..., 0] = rise * np.log(2.0) * c.D ** 0.5
    q = q.flatten(1).to(types()[type][1])
    check(c, c.attend(q), q.double().cpu().numpy(), rows=71)
