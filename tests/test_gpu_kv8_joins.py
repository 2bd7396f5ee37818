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


@pytest.mark.parametrize("type", TYPES)
def test_captured_prompts(type):
    """A packed batch for both kernels, captured and replayed with other inputs and positions beside another call on another
    stream, with and without programmatic launches: the same bits as calls one at a time."""
    c = Cache([(500, 60), (0, 2), (30, 1), (0, 0), (900, 90)], H=8, G=2, D=64, type=type, seed=55).upload()
    d = Cache([(2000, 3), (100, 200)], H=8, G=1, D=128, type=type, seed=56).upload()
    (q, _), (q2, _) = c.rows(c.H * c.D), d.rows(d.H * d.D)
    ws = torch.zeros(ffn.moe_kv8_workspace_size(c.cfg()), dtype=torch.uint8, device="cuda")
    o, want2 = torch.empty_like(q), d.attend(q2)
    side, graphs = torch.cuda.Stream(), []
    for flags in (0, ffn.MOE_NO_PDL):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ffn.check(ffn.moe_kv8_attn_prefill(q, c.d_cache, c.d_offsets, c.d_past, c.d_table, None, c.cfg(flags=flags), o, ws,
                                               ws.numel(), torch.cuda.current_stream()))
    for t in range(3):
        q.copy_(torch.randn(q.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(t)))
        c.d_past.copy_(torch.tensor([500 - 100 * t, t, 30 + t, 0, 900 - 33 * t], dtype=torch.int32))
        want = c.attend(q)
        for g in graphs:
            o.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            with torch.cuda.stream(side):
                o2 = d.attend(q2)
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(o2, want2)
    ffn.check(ffn.moe_workspace_status(ws, torch.cuda.current_stream()))
