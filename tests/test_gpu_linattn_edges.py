"""Linear attention prompts: offsets that go back, many sequences, rows in wider buffers and
values that are not finite in narrow heads. Bounds: tests/test_gpu_linattn.py."""

import numpy as np
import pytest

import expert_ffn_decode_gb300 as ffn
from oracle import ops_oracle as oo
from tests.test_gpu_linattn import TYPES, Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def call(c, offsets, ws):
    o = torch.full((sum(c.lens), c.H, c.dv), float("nan"), dtype=TYPES[c.type][1], device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ffn.check(ffn.moe_linattn_prefill(c.q, c.k, c.v, c.g, off, c.slots, c.cfg(), c.state, o, ws, ws.numel(),
                                      torch.cuda.current_stream()))
    return o


@pytest.mark.parametrize("type", list(TYPES))
def test_offsets_that_go_back_and_rise_again(type):
    """Sequences that share tokens ask for more units than the call's tokens have: the ones without
    room keep their state and rows and the status says so, whatever the workspace held."""
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream()
    dims = dict(H=16, dk=64, dv=64, type=type)
    c = Case([600, 300, 300], seed=1, **dims)
    want = c.want()
    c.check(call(c, [0, 600, 900, 1200], ws), c.state, want)  # leaves decays and states in the workspace
    ffn.check(ffn.moe_workspace_status(ws, st))
    c = Case([1000, 100, 100], seed=2, **dims)
    before = c.state.clone()
    c.begin = np.array([0, 1000, 1000, 1000])
    want = c.want(before)
    o = call(c, [0, 1000, 200, 1200], ws)
    assert ffn.moe_workspace_status(ws, st) == ffn.MOE_ERR_INVALID_CFG and "offsets" in ffn.moe_last_error()
    assert torch.equal(c.state[1:], before[1:])
    assert torch.isnan(o[1000:]).all()
    c.check(torch.where(torch.isnan(o), 0, o), c.state, want)
    c = Case([600, 300, 300], seed=3, **dims)  # and the workspace serves the next call
    want = c.want()
    c.check(call(c, [0, 600, 900, 1200], ws), c.state, want)
    ffn.check(ffn.moe_workspace_status(ws, st))


def oracle_range(c, i, j, start):
    """Outputs, state and their magnitudes of tokens i .. j - 1 from the states `start` [H][dk][dv]."""
    host = lambda a: a.double().cpu().numpy()
    q, k, v, g = (host(a)[i:j] for a in (c.q, c.k, c.v, c.g))
    return [np.stack(x, a) for a, x in zip((1, 0, 1, 0), zip(*(
        oo.linattn(q[:, h * c.G // c.H], k[:, h * c.G // c.H], v[:, h], g[:, h], start[h], c.scale) for h in range(c.H))))]


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("n", [40, 150])
def test_short_sequences_that_share_tokens(type, n):
    """Where the call's units suffice (here each sequence is one), sequences may share tokens."""
    c = Case([n, 1, 9], H=2, dk=64, dv=64, type=type)
    before = c.state.double().cpu().numpy()
    ws = torch.zeros(ffn.moe_linattn_workspace_size(c.cfg()), dtype=torch.uint8, device="cuda")
    call(c, [0, n, 10, n + 10], ws)
    ffn.check(ffn.moe_workspace_status(ws, torch.cuda.current_stream()))
    got = c.state.double().cpu().numpy()
    for b, i, j in ((0, 0, n), (2, 10, n + 10)):
        _, s, _, a = oracle_range(c, i, j, before[b])
        assert np.all(np.abs(got[b] - s) <= (2 * n + c.dk + 64) * 2.0 ** -24 * a)
    assert np.array_equal(got[1], before[1])


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("longest", [300, 700])
def test_thousands_of_sequences(type, longest):
    """Far more sequences than one round of the search takes, with and without some that are cut."""
    rng = np.random.default_rng(51)
    lens = [int(n) for n in rng.integers(0, 4, 3000)]
    for b in (0, 255, 256, 1999, 2999):
        lens[b] = longest
    c = Case(lens, H=2, G=1, dk=16, dv=24, type=type, decay="reset")
    want = c.want()
    c.check(c.prefill(), c.state, want)
