"""The operators next to the step without a GPU: their entry points refuse bad arguments on
the host, and their oracle agrees with the step's block decoders and with closed forms."""

import os

import numpy as np
import pytest

import expert_ffn_decode_gb300 as ffn
from expert_ffn_decode_gb300 import synth
from oracle import moe_oracle as mo
from oracle import ops_oracle as oo


@pytest.fixture(scope="module")
def built():
    if not os.path.exists(ffn.LIB_PATH):
        from expert_ffn_decode_gb300 import build
        build.build()
    return ffn.lib()


# Addresses that are never read: every call below is refused before a launch.
X, W, S, M, B, Y = (1 << 24, 1 << 26, 1 << 28, 1 << 29, 1 << 30, 1 << 32)


def mv_cfg(**kw):
    return ffn.make_matvec_cfg(**{**dict(rows=64, cols=256, n_vec=2, qtype=ffn.MOE_Q4_1), **kw})


def mv(cfg, x=X, w=W, s=None, m=None, b=None, y=Y):
    return ffn.moe_q4_matvec(x, w, s, m, b, cfg, y, None)


@pytest.mark.parametrize("kw", [
    dict(rows=0), dict(rows=-1), dict(cols=0), dict(cols=31), dict(cols=48), dict(cols=16416), dict(n_vec=-1),
    dict(qtype=0), dict(qtype=14), dict(qtype=12, cols=288), dict(group=32), dict(qtype=64),
    dict(qtype=64, group=16), dict(qtype=64, group=64, cols=96), dict(qtype=64, group=256),
    dict(x_type=2), dict(y_type=29), dict(flags=2), dict(flags=256), dict(x_stride=255), dict(x_stride=-256),
    dict(y_stride=63), dict(x_stride=1 << 40),
], ids=str)
def test_matvec_refuses_cfg(built, kw):
    assert mv(mv_cfg(**kw)) == ffn.MOE_ERR_INVALID_CFG
    assert ffn.moe_last_error()


def test_matvec_refuses_pointers(built):
    planes = mv_cfg(qtype=ffn.MOE_Q4_PLANES, group=64)
    assert mv(mv_cfg(), x=None) == ffn.MOE_ERR_NULL_PTR
    assert mv(mv_cfg(), w=None) == ffn.MOE_ERR_NULL_PTR
    assert mv(mv_cfg(), y=None) == ffn.MOE_ERR_NULL_PTR
    assert mv(planes) == ffn.MOE_ERR_NULL_PTR                       # no scales
    assert mv(mv_cfg(), s=S) == ffn.MOE_ERR_INVALID_CFG             # blocks hold their own
    assert mv(mv_cfg(), m=M) == ffn.MOE_ERR_INVALID_CFG
    for kw in (dict(x=X + 4), dict(w=W + 8), dict(y=Y + 2), dict(b=B + 2)):
        assert mv(mv_cfg(), **kw) == ffn.MOE_ERR_ALIGNMENT, kw
    for kw in (dict(s=S + 2), dict(s=S, m=M + 2)):
        assert mv(planes, **kw) == ffn.MOE_ERR_ALIGNMENT, kw
    assert mv(mv_cfg(x_stride=258)) == ffn.MOE_ERR_ALIGNMENT
    assert mv(mv_cfg(x_type=ffn.MOE_BF16, x_stride=260)) == ffn.MOE_ERR_ALIGNMENT
    assert mv(mv_cfg(), y=X + 1024) == ffn.MOE_ERR_INVALID_CFG and "overlap" in ffn.moe_last_error()
    # y inside x's rows of a wider buffer, in the columns that x takes
    assert mv(mv_cfg(x_stride=512, y_stride=512), y=X + 4 * 200) == ffn.MOE_ERR_INVALID_CFG
    # nothing to do: no pointer is looked at
    assert mv(mv_cfg(n_vec=0), x=None, w=None, y=None) == ffn.MOE_OK
    assert ffn.lib().moe_q4_matvec(X, W, None, None, None, None, Y, None) == ffn.MOE_ERR_NULL_PTR


Q, K, V, G, O, ST, WS, OFF, SL = (i << 34 for i in range(1, 10))


def la_cfg(**kw):
    return ffn.make_linattn_cfg(**{**dict(n_seq=2, n_tokens=10, n_heads=4, key_dim=64, value_dim=128,
                                          n_qk_heads=2, scale=0.125), **kw})


def pre(cfg, q=Q, k=K, v=V, g=G, off=OFF, sl=None, st=ST, o=O, ws=WS, n=1 << 40):
    return ffn.moe_linattn_prefill(q, k, v, g, off, sl, cfg, st, o, ws, n, None)


def step(cfg, q=Q, k=K, v=V, g=G, sl=None, st=ST, o=O):
    return ffn.moe_linattn_step(q, k, v, g, sl, cfg, st, o, None)


@pytest.mark.parametrize("kw", [
    dict(n_seq=-1), dict(n_seq=65536), dict(n_tokens=-1), dict(n_heads=0), dict(n_heads=2048, n_qk_heads=2),
    dict(n_qk_heads=3), dict(n_qk_heads=0), dict(key_dim=0), dict(key_dim=12), dict(key_dim=136),
    dict(value_dim=4), dict(value_dim=256), dict(n_states=-1), dict(type=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(flags=1), dict(flags=1024), dict(q_stride=127), dict(k_stride=8),
    dict(v_stride=511), dict(o_stride=-512), dict(v_stride=1 << 40),
], ids=str)
def test_linattn_refuses_cfg(built, kw):
    cfg = la_cfg(**kw)
    assert ffn.moe_linattn_workspace_size(cfg) == 0
    assert pre(cfg) == ffn.MOE_ERR_INVALID_CFG and ffn.moe_last_error()
    assert step(la_cfg(**{"n_tokens": 2, **kw})) == ffn.MOE_ERR_INVALID_CFG


def test_linattn_refuses_pointers(built):
    for name in ("q", "k", "v", "g", "st", "o"):
        assert pre(la_cfg(), **{name: None}) == ffn.MOE_ERR_NULL_PTR, name
        assert step(la_cfg(n_tokens=2), **{name: None}) == ffn.MOE_ERR_NULL_PTR, name
        off = 2 if name == "g" else 8
        assert pre(la_cfg(), **{name: {"q": Q, "k": K, "v": V, "g": G, "st": ST, "o": O}[name] + off}) == \
            ffn.MOE_ERR_ALIGNMENT, name
    assert pre(la_cfg(), ws=None) == ffn.MOE_ERR_NULL_PTR
    assert pre(la_cfg(), ws=WS + 16) == ffn.MOE_ERR_ALIGNMENT
    assert pre(la_cfg(), off=OFF + 2) == ffn.MOE_ERR_ALIGNMENT
    assert pre(la_cfg(), sl=SL + 1) == ffn.MOE_ERR_ALIGNMENT
    assert pre(la_cfg(), n=64) == ffn.MOE_ERR_WORKSPACE
    assert pre(la_cfg(q_stride=132)) == ffn.MOE_ERR_ALIGNMENT
    assert pre(la_cfg(n_states=1)) == ffn.MOE_ERR_INVALID_CFG            # two sequences, one state, no slots
    assert pre(la_cfg(n_tokens=11), off=None) == ffn.MOE_ERR_INVALID_CFG  # 11 tokens are not two equal sequences
    assert step(la_cfg()) == ffn.MOE_ERR_INVALID_CFG                     # 10 tokens, two sequences
    assert pre(la_cfg(), o=V) == ffn.MOE_ERR_INVALID_CFG and "overlap" in ffn.moe_last_error()
    assert pre(la_cfg(), o=Q + 256) == ffn.MOE_ERR_INVALID_CFG
    # a view of the same rows in v's columns
    assert pre(la_cfg(v_stride=1024, o_stride=1024), o=V + 2 * 504) == ffn.MOE_ERR_INVALID_CFG
    assert pre(la_cfg(n_seq=0, n_tokens=0), q=None, st=None, ws=None) == ffn.MOE_OK
    assert step(la_cfg(n_seq=0, n_tokens=0), q=None, st=None) == ffn.MOE_OK
    assert ffn.lib().moe_linattn_workspace_size(None) == 0


def test_workspace_size(built):
    n = ffn.moe_linattn_workspace_size(la_cfg())
    assert n >= 512 and n % 256 == 0


def test_workspace_holds_every_units_state(built):
    """A prompt that is cut needs a state for each unit of each head; one that stays whole none."""
    small = ffn.moe_linattn_workspace_size(la_cfg(n_seq=1, n_tokens=200))
    large = ffn.moe_linattn_workspace_size(la_cfg(n_seq=1, n_tokens=4096))
    assert small == 512
    units = -(-4096 // 128)  # at most this many: units have at least 128 tokens
    state = 4 * 64 * 128 * 4
    assert 512 + 2 * state < large <= 2 * units * (state + 64) + 1024


@pytest.mark.parametrize("qtype", [oo.Q4_0, oo.Q4_1, oo.Q4_K])
def test_oracle_blocks_against_the_steps(qtype):
    """The oracle's (q, scale, offset) give the values of the step's pinned decoders."""
    rng = np.random.default_rng(1)
    rows, cols = 3, 512
    b = synth.any_blocks(rng, qtype, rows * cols // synth.BLOCK_VALUES[qtype]).reshape(rows, -1)
    q, s, m = oo.block_values(b, cols, qtype)
    ref = (mo.dequant_q4k if qtype == oo.Q4_K else lambda *a: mo.dequant_rows(*a, qtype))(b.reshape(-1), rows, cols)
    np.testing.assert_allclose(s * q + m, ref, rtol=0, atol=1e-15)


def test_oracle_planes_are_q4_blocks():
    """Planes of group 32 hold what Q4_1 (with offsets) and Q4_0 (without) blocks hold."""
    rng = np.random.default_rng(2)
    b = synth.any_blocks(rng, oo.Q4_1, 4 * 6).reshape(4, 6, 20)
    d, m = (np.ascontiguousarray(b[..., i:i + 2]).view(np.float16)[..., 0] for i in (0, 2))
    nib = b[..., 4:].reshape(4, -1)
    for mins, qtype, blocks in ((m, oo.Q4_1, b), (None, oo.Q4_0, np.concatenate([b[..., :2], b[..., 4:]], -1))):
        for u, w in zip(oo.planes_values(nib, d, mins, 32), oo.block_values(blocks.reshape(4, -1), 192, qtype)):
            np.testing.assert_array_equal(u, w)


def test_oracle_linattn_closed_forms():
    rng = np.random.default_rng(3)
    T, dk, dv = 12, 8, 16
    q, k, v = rng.standard_normal((T, dk)), rng.standard_normal((T, dk)), rng.standard_normal((T, dv))
    S0 = rng.standard_normal((dk, dv))
    g = -rng.random(T)
    G = np.cumsum(g)
    o, S, _, _ = oo.linattn(q, k, v, g, S0, 0.5)
    D = np.tril(np.exp(G[:, None] - G[None, :]))
    np.testing.assert_allclose(o, 0.5 * (((q @ k.T) * D) @ v + np.exp(G)[:, None] * (q @ S0)), rtol=1e-12)
    np.testing.assert_allclose(S, np.exp(G[-1]) * S0 + (k * np.exp(G[-1] - G)[:, None]).T @ v, rtol=1e-12)
    g[5] = -np.inf  # a reset: what follows does not see what was before
    o, S, _, _ = oo.linattn(q, k, v, g, S0, 0.5)
    o2, S2, _, _ = oo.linattn(q[5:], k[5:], v[5:], g[5:], 0 * S0, 0.5)
    np.testing.assert_allclose(o[5:], o2, rtol=1e-12)
    np.testing.assert_allclose(S, S2, rtol=1e-12)


@pytest.mark.parametrize("type", [ffn.MOE_BF16, ffn.MOE_F32])
@pytest.mark.parametrize("heads", [1, 4, 16, 37, 100, 304])
def test_workspace_grows_with_the_tokens(built, heads, type):
    """A workspace for the longest call serves the shorter ones, however many sequences they have."""
    sizes = [ffn.moe_linattn_workspace_size(la_cfg(n_seq=b, n_tokens=n, n_heads=heads, n_qk_heads=1, n_states=9, type=type))
             for n in range(1, 5000, 61) for b in (1, 7)]
    assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))
