"""Attention over the 8-bit cache where a row tile is cut over many CTAs: sums of 25 and more of them are joined in two
levels, and two such stretches can meet in sixteen CTAs. Groups of tokens: 128 for prompts, 16 or 32 for steps. And tiles of
one token, where more than 64 heads share a key/value head. Bounds: tests/kv8_bounds.py."""

import pytest

import expert_ffn_decode_gb300 as ffn
from tests.kv8_bounds import check
from tests.kv8_cases import Cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]


def repeats(c, q, qd, step, rows=1):
    """Against the bounds, and the same bits again in the workspace that the first call used."""
    ws = torch.zeros(ffn.moe_kv8_workspace_size(c.cfg()), dtype=torch.uint8, device="cuda")
    o = c.attend(q, step=step, ws=ws)
    check(c, o, qd, rows=rows)
    for _ in range(2):
        assert torch.equal(o, c.attend(q, step=step, ws=ws))
    ffn.check(ffn.moe_workspace_status(ws, torch.cuda.current_stream()))


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("seqs", [[(20000, 1)], [(20000, 1), (9000, 1)], [(7000, 1), (0, 1), (7000, 1), (30, 1), (5000, 1)]], ids=str)
@pytest.mark.parametrize("dims", [dict(H=4, G=1, D=64), dict(H=16, G=1, D=128), dict(H=2, G=1, D=256, code="e4m3")], ids=str)
def test_steps_over_many_ctas(type, seqs, dims):
    c = Cache(seqs, type=type, seed=51, **dims).upload()
    q, qd = c.rows(c.H * c.D)
    repeats(c, q, qd, True)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("seqs,H", [([(20000, 16)], 4), ([(20000, 100)], 2), ([(9000, 64), (11000, 64)], 4),
                                    ([(6000, 50), (0, 3), (6000, 60), (5500, 70)], 2)], ids=str)
@pytest.mark.parametrize("D,code", [(64, "i8"), (128, "e4m3")])
def test_prompts_over_many_ctas(type, seqs, H, D, code):
    c = Cache(seqs, H=H, G=1, D=D, type=type, code=code, sinks=True, seed=52).upload()
    q, qd = c.rows(c.H * c.D)
    repeats(c, q, qd, False, rows=23)


def test_a_window_over_many_ctas():
    """A long sequence's first groups are behind the window; the parts are of what is left."""
    c = Cache([(20000, 80), (300, 40)], H=4, G=1, D=128, type="bf16", window=7000, holes={(0, 250), (0, 251)}, seed=53).upload()
    q, qd = c.rows(c.H * c.D)
    repeats(c, q, qd, False, rows=23)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("H", [65, 80, 127, 128, 129, 200])
def test_many_heads_of_one_key(type, H):
    """Tiles of one token (up to 128 heads a key/value head), and the other kernel beyond."""
    c = Cache([(0, 3), (200, 4), (17, 1), (0, 0), (1000, 2)], H=H, G=1, D=64, type=type, seed=54).upload()
    q, qd = c.rows(c.H * c.D)
    repeats(c, q, qd, False)
