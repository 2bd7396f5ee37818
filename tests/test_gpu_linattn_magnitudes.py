"""Linear attention prompts whose values differ by many powers of ten inside one tile of tokens.

The bounds are those of tests/test_gpu_linattn.py, element by element relative to the summed
magnitudes of an element's own terms, so they do not widen with what other tokens, other
sequences of a reset or (in f32 and bf16, whose operands keep each value's own bits) other
channels hold."""

import numpy as np
import pytest

from tests.test_gpu_linattn import TYPES, Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPE_NAMES = list(TYPES)


def scaled(c, name, rows, factor):
    """Rows of an input times a factor (a number, or one for each row or channel), rounded to its type."""
    t = getattr(c, name)
    f = torch.as_tensor(np.asarray(factor, np.float64), device="cuda")
    if f.dim() == 1:
        f = f[:, None, None]
    t[rows] = (t[rows].double() * f).to(t.dtype)


@pytest.mark.parametrize("lens", [[330], [700, 90]], ids=["whole", "cut"])
@pytest.mark.parametrize("ratio", [1e4, 1e6, 1e8])
@pytest.mark.parametrize("type,names", [("f32", "k"), ("f32", "v"), ("f32", "q"), ("f32", "kv"), ("bf16", "k"),
                                        ("bf16", "kv"), ("f16", "k"), ("f16", "v")])
def test_large_values_before_a_reset(type, names, ratio, lens):
    """What was before a reset takes no bits from what comes after it, in the same tile."""
    c = Case(lens, H=2, dk=128, dv=128, type=type, seed=31)
    cut = lens[0] - 40  # a reset inside a chunk of the first sequence
    c.g[cut] = -float("inf")
    before, after = slice(0, cut), slice(cut, lens[0])
    for name in names:
        if type == "f16":  # split between the two sides: f16 spans 6e-8 .. 65504
            scaled(c, name, before, min(ratio ** 0.5, 2e3))
            scaled(c, name, after, min(ratio ** 0.5, 2e3) / ratio)
        else:
            scaled(c, name, before, ratio)
    if type == "f16" and names == "k":
        scaled(c, "q", before, 1e-3)  # outputs inside f16
    want = c.want()
    o = c.prefill()
    c.check(o, c.state, want)
    # the tokens after the reset and the state they leave, by themselves
    ro, rs = want[0][cut:lens[0]], want[1][0]
    if type != "f16":
        assert np.linalg.norm(c.state[0].double().cpu().numpy() - rs) <= 2.0 ** -19 * np.linalg.norm(rs)
    if type == "f32":
        assert np.linalg.norm(o[cut:lens[0]].double().cpu().numpy() - ro) <= 2.0 ** -19 * np.linalg.norm(ro)


@pytest.mark.parametrize("type", TYPE_NAMES)
def test_large_values_before_a_strong_decay(type):
    """The same where the earlier tokens do not vanish but are worth less than the later ones."""
    c = Case([130, 300], H=2, dk=128, dv=64, type=type, seed=32)
    for at in (100, 400):
        c.g[at] = -40.0
        scaled(c, "k", slice(at - 30, at), 1e3 if type == "f16" else 1e7)
        if type == "f16":
            scaled(c, "q", slice(at - 30, at), 1e-2)
    want = c.want()
    c.check(c.prefill(), c.state, want)


@pytest.mark.parametrize("lens", [[330], [600, 70]], ids=["whole", "cut"])
@pytest.mark.parametrize("type", TYPE_NAMES)
def test_keys_and_values_of_opposite_size(type, lens):
    """Tokens of large keys and small values beside tokens of small keys and large values: their
    products, and so their shares of state and outputs, are alike."""
    c = Case(lens, H=2, dk=128, dv=128, type=type, seed=33)
    r = 10.0 ** np.random.default_rng(34).uniform(*((-2, 2) if type == "f16" else (-5, 5)), sum(lens))
    scaled(c, "k", slice(None), r)
    scaled(c, "v", slice(None), 1 / r)
    want = c.want()
    c.check(c.prefill(), c.state, want)


@pytest.mark.parametrize("lens", [[330], [600, 70]], ids=["whole", "cut"])
@pytest.mark.parametrize("type", TYPE_NAMES)
def test_channels_of_different_size(type, lens):
    """Channels of q and k whose sizes cancel in the scores, and channels of v of different sizes.
    (f16 holds decayed keys, states and scores in 22 bits of the largest: a narrower span.)"""
    c = Case(lens, H=2, dk=96, dv=128, type=type, seed=35)
    rng, span = np.random.default_rng(36), 1 if type == "f16" else 4
    f = torch.from_numpy(10.0 ** rng.uniform(-span, span, 96)).cuda()
    c.q.copy_((c.q.double() / f).to(c.q.dtype))
    c.k.copy_((c.k.double() * f).to(c.k.dtype))
    f = torch.from_numpy(10.0 ** rng.uniform(-span, span, 128)).cuda()
    c.v.copy_((c.v.double() * f).to(c.v.dtype))
    want = c.want()
    c.check(c.prefill(), c.state, want)
