"""Linear attention prompts whose outputs are rows of a wider buffer and whose first sequence does
not start at token 0, and values that are not finite in heads of every width: element by element
against the float64 oracle with the bounds of tests/test_gpu_linattn.py."""

import numpy as np
import pytest

from tests.test_gpu_linattn import TYPES, Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

WIDTHS = [(128, 128), (72, 40), (8, 8), (64, 128), (128, 64), (96, 72), (120, 96), (16, 120)]


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 72), (72, 40), (128, 64)])
@pytest.mark.parametrize("n", [20, 150, 700])
def test_rows_of_a_wider_buffer(n, dk, dv, type):
    """Covered rows hold the oracle's outputs at their places; nothing else of the buffer changes."""
    H = 3
    c = Case([n, n], H=H, G=1, dk=dk, dv=dv, type=type)
    off = np.array([5, n, 2 * n - 7])
    c.begin = off
    want = c.want()
    buf = torch.full((2 * n, H * dv + 24), 7.0, dtype=TYPES[type][1], device="cuda")
    c.prefill(offsets=torch.from_numpy(off.astype(np.int32)).cuda(), o=buf, o_stride=H * dv + 24)
    assert (buf[:, H * dv:] == 7).all() and (buf[:5] == 7).all() and (buf[2 * n - 7:] == 7).all()
    o = torch.zeros(2 * n, H, dv, dtype=buf.dtype, device="cuda")
    o[5:2 * n - 7] = buf[5:2 * n - 7, :H * dv].unflatten(1, (H, dv))
    c.check(o, c.state, want)


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "g"])
@pytest.mark.parametrize("dk,dv", WIDTHS[1:])
def test_non_finite_does_not_reach_back(dk, dv, where, bad, type):
    """A NaN or an infinity at one token reaches no earlier token, no other sequence or head, and
    one of v no other channel."""
    if where == "g" and bad > 0:
        bad = float("nan")
    c = Case([200, 90], H=2, dk=dk, dv=dv, type=type)
    t = 170
    want = c.want()
    if where == "g":
        c.g[t, 1] = bad
    else:
        getattr(c, where)[t, 1, 5] = bad
    o = c.prefill()
    ok, oks = np.ones((290, 2, dv), bool), np.ones((2, 2, dk, dv), bool)
    if where == "v":
        ok[t:200, 1, 5] = oks[0, 1, :, 5] = False
    elif where == "q":
        ok[t, 1] = False
    else:
        ok[t:200, 1] = oks[0, 1] = False
    on = lambda m: torch.from_numpy(m).cuda()
    c.check(torch.where(on(ok), o, 0), torch.where(on(oks), c.state, 0),
            tuple(np.where(m, w, 0) for m, w in zip((ok, oks, ok, oks), want)))
    if where == "v":
        assert not torch.isfinite(o[t:200, 1, 5]).any() and not torch.isfinite(c.state[0, 1, :, 5]).any()
    else:
        assert not torch.isfinite(o[t, 1]).any() and (where == "q" or not torch.isfinite(o[t:200, 1]).any())


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_non_finite_early_value_in_a_long_prompt(dk, dv, type):
    """The same in a prompt that is cut into units, from near its start."""
    c = Case([700, 130], H=2, dk=dk, dv=dv, type=type, decay="head")
    c.v[65, 1, 5] = 0
    want = c.want()
    c.v[65, 1, 5] = float("nan")
    o = c.prefill()
    ok, oks = np.ones((830, 2, dv), bool), np.ones((2, 2, dk, dv), bool)
    ok[65:700, 1, 5] = oks[0, 1, :, 5] = False
    on = lambda m: torch.from_numpy(m).cuda()
    c.check(torch.where(on(ok), o, 0), torch.where(on(oks), c.state, 0),
            tuple(np.where(m, w, 0) for m, w in zip((ok, oks, ok, oks), want)))
    assert not torch.isfinite(o[65:700, 1, 5]).any() and not torch.isfinite(c.state[0, 1, :, 5]).any()
