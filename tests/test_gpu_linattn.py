"""Linear attention with a decay for each head on the GPU against the float64 oracle.

Tolerances, element by element, relative to the summed magnitudes a_o and a_state of the
terms (the oracle's last results): a term passes at most two f32 roundings a token it lives
through and dk + 64 more, so (2 T + dk + 64) 2^-24; o is then rounded once (half a step of its
type). For 16-bit types the prompt form may hold scores and states in two 16-bit parts
while it multiplies (2^-17 relative each): 2^-16 a_o more. Over whole outputs in f32 these
roundings average out: a relative 2-norm of 2^-19."""

import numpy as np
import pytest

import expert_ffn_decode_gb300 as ffn
from oracle import ops_oracle as oo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": (ffn.MOE_F32, torch.float32, 2.0 ** -24, 0.0), "f16": (ffn.MOE_F16, torch.float16, 2.0 ** -11, 2.0 ** -16),
         "bf16": (ffn.MOE_BF16, torch.bfloat16, 2.0 ** -8, 2.0 ** -16)}


class Case:
    """Seeded inputs on the host (rounded to the type) and on the device."""

    def __init__(self, lens, H=2, G=None, dk=64, dv=64, type="bf16", decay="token", n_states=None, slots=None,
                 fresh=False, fused=False, seed=0, amp=1.0):
        G = G or H
        rng = np.random.default_rng([seed, sum(lens), len(lens), dk, dv])
        self.lens, self.H, self.G, self.dk, self.dv, self.type, self.fresh = lens, H, G, dk, dv, type, fresh
        n, T = len(lens), sum(lens)
        dt = TYPES[type][1]
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
        q, k, v = f(T, G, dk), f(T, G, dk) / dk ** 0.5, f(T, H, dv) * amp
        if fused:
            buf = torch.cat([a.reshape(T, -1) for a in (q, k, v)] + [f(T, 16)], 1).to(dt).cuda()
            self.q, self.k, self.v = (a.unflatten(1, (-1, d)) for a, d in
                                      zip(buf.split([G * dk, G * dk, H * dv, 16], 1), (dk, dk, dv)))
        else:
            self.q, self.k, self.v = (a.to(dt).cuda() for a in (q, k, v))
        if decay == "head":
            g = -2.0 ** (-1.0 - np.arange(H))
        else:
            g = -np.log1p(np.exp(rng.standard_normal((T, H)) - 1))
            if decay == "reset":
                g[rng.random((T, H)) < 0.08] = -np.inf
                g[rng.random((T, H)) < 0.05] = -30.0
                g[rng.random((T, H)) < 0.05] = 0.0
        self.decay, self.g = decay, torch.from_numpy(g.astype(np.float32)).cuda()
        self.n_states = n_states or max(n, 1)
        self.slots = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
        self.state = f(self.n_states, H, dk, dv).cuda()
        self.begin = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.offsets = torch.from_numpy(self.begin).cuda()
        self.scale = dk ** -0.5

    def cfg(self, **kw):
        flags = (ffn.MOE_FRESH_STATE if self.fresh else 0) | (0 if self.decay == "head" else ffn.MOE_TOKEN_DECAY)
        return ffn.make_linattn_cfg(**{**dict(
            n_seq=len(self.lens), n_tokens=sum(self.lens), n_heads=self.H, key_dim=self.dk, value_dim=self.dv,
            n_qk_heads=self.G, n_states=self.n_states, type=TYPES[self.type][0], scale=self.scale, flags=flags,
            q_stride=self.q.stride(0), k_stride=self.k.stride(0), v_stride=self.v.stride(0)), **kw})

    def want(self, state=None):
        """(o, state, a_o, a_state) in float64; rows of inactive sequences are 0."""
        T = sum(self.lens)
        host = lambda a: a.double().cpu().numpy()
        q, k, v, g = host(self.q), host(self.k), host(self.v), host(self.g)
        st = host(self.state if state is None else state)
        o, ao, as_ = np.zeros((T, self.H, self.dv)), np.zeros((T, self.H, self.dv)), np.abs(st)
        slots = range(len(self.lens)) if self.slots is None else self.slots.tolist()
        for b, s in enumerate(slots):
            if not 0 <= s < self.n_states:
                continue
            i, j = self.begin[b], self.begin[b + 1]
            for h in range(self.H):
                gh = np.full(j - i, g[h]) if self.decay == "head" else g[i:j, h]
                c = h * self.G // self.H
                o[i:j, h], st[s, h], ao[i:j, h], as_[s, h] = oo.linattn(
                    q[i:j, c], k[i:j, c], v[i:j, h], gh, 0 * st[s, h] if self.fresh else st[s, h], self.scale)
        return o, st, ao, as_

    def check(self, o, state, want, label=""):
        ro, rs, ao, as_ = want
        n = 2 * max(self.lens + [1]) + self.dk + 64
        half, extra = TYPES[self.type][2:]
        o, state = o.double().cpu().numpy(), state.double().cpu().numpy()
        tol = half * np.abs(ro) + (n * 2.0 ** -24 + extra) * ao
        if self.type == "f16":
            tol = tol + 2.0 ** -25  # half a step of its smallest numbers
        assert np.all(np.abs(o - ro) <= tol), (label, "o", float(np.nanmax(np.abs(o - ro) / (tol + 1e-300))),
                                               np.argwhere(~(np.abs(o - ro) <= tol))[:4])
        tol = n * 2.0 ** -24 * as_
        assert np.all(np.abs(state - rs) <= tol), (label, "state", float(np.nanmax(np.abs(state - rs) / (tol + 1e-300))),
                                                   np.argwhere(~(np.abs(state - rs) <= tol))[:4])
        assert np.linalg.norm(state - rs) <= 2.0 ** -19 * np.linalg.norm(rs) + 1e-30, (label, "state norm")
        if self.type == "f32":
            assert np.linalg.norm(o - ro) <= 2.0 ** -19 * np.linalg.norm(ro) + 1e-30, (label, "o norm")

    def prefill(self, stream=None, offsets="own", o=None, **kw):
        cfg = self.cfg(**kw)
        ws = torch.zeros(ffn.moe_linattn_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        if o is None:
            o = torch.full((sum(self.lens), self.H, self.dv), float("nan"), dtype=TYPES[self.type][1], device="cuda")
        st = stream or torch.cuda.current_stream()
        off = self.offsets if isinstance(offsets, str) else offsets
        ffn.check(ffn.moe_linattn_prefill(self.q, self.k, self.v, self.g, off, self.slots, cfg, self.state, o, ws,
                                          ws.numel(), st))
        ffn.check(ffn.moe_workspace_status(ws, st))
        return o

    def step(self, stream=None, **kw):
        o = torch.full((len(self.lens), self.H, self.dv), float("nan"), dtype=TYPES[self.type][1], device="cuda")
        ffn.check(ffn.moe_linattn_step(self.q, self.k, self.v, self.g, self.slots, self.cfg(**kw), self.state, o,
                                       stream or torch.cuda.current_stream()))
        return o


PREFILL = [
    dict(lens=[1]), dict(lens=[2, 0, 5], decay="reset"), dict(lens=[63, 64, 65], dk=128, dv=128),
    dict(lens=[40], dk=128, dv=128, decay="head", fresh=True), dict(lens=[0, 0], fresh=True),
    dict(lens=[130, 17, 0, 1, 300], H=4, G=2, dk=128, dv=128, decay="reset", fused=True),
    dict(lens=[257], H=3, G=1, dk=72, dv=40, decay="head"), dict(lens=[100, 90], dk=8, dv=8),
    dict(lens=[513, 20], dk=128, dv=64, decay="reset", fresh=True), dict(lens=[320], dk=64, dv=128, fused=True),
    dict(lens=[300, 200], dk=96, dv=96, n_states=5, slots=[4, 1]), dict(lens=[90], dk=32, dv=112),
    dict(lens=[128, 64, 200, 3], dk=128, dv=128, n_states=6, slots=[5, -1, 2, 6], decay="reset"),
    dict(lens=[900], H=1, dk=128, dv=128, decay="reset", amp=100.0), dict(lens=[640], H=1, dk=128, dv=128, decay="head"),
    dict(lens=[1, 1, 1, 70], dk=120, dv=128, decay="token", fresh=True, n_states=9, slots=[0, 8, 3, 7]),
]


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("kw", PREFILL, ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()).replace(" ", ""))
def test_prefill(kw, type):
    c = Case(type=type, **kw)
    first = c.state.clone()
    want = c.want()
    o = c.prefill()
    c.check(o, c.state, want)
    got = c.state.clone()
    c.state.copy_(first)
    again = c.prefill()
    assert torch.equal(o, again) and torch.equal(got, c.state)  # repeat calls agree bit for bit


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("kw", [
    dict(lens=[1]), dict(lens=[1] * 7, H=10, dk=72, dv=40, n_states=9, slots=[3, 0, -1, 8, 9, 5, 1]),
    dict(lens=[1] * 5, H=4, G=1, dk=128, dv=128, decay="reset", fused=True), dict(lens=[1] * 3, dk=8, dv=120, decay="head"),
    dict(lens=[1] * 2, dk=64, dv=64, fresh=True), dict(lens=[1] * 40, H=16, G=8, dk=128, dv=128, decay="head"),
    dict(lens=[1] * 3, H=5, dk=104, dv=24, decay="reset"), dict(lens=[1] * 39, H=8, G=4, dk=72, dv=40, decay="reset"),
    dict(lens=[1] * 80, H=4, dk=128, dv=32), dict(lens=[1] * 80, H=4, dk=24, dv=64), dict(lens=[1] * 31, H=10, dk=96, dv=88),
], ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items() if k != "lens") + f",n={len(d['lens'])}")
def test_step(kw, type):
    c = Case(type=type, **kw)
    want = c.want()
    c.check(c.step(), c.state, want)


@pytest.mark.parametrize("type", list(TYPES))
def test_prompt_then_tokens(type):
    """A prompt and single tokens give what one longer prompt gives, on the same states."""
    c = Case([150, 70], H=4, G=2, dk=128, dv=128, type=type, decay="reset")
    want = c.want()
    keep = 4  # the last tokens of each sequence go one by one
    rows = [[i for i in range(c.begin[b], c.begin[b + 1] - keep)] for b in range(2)]
    first = torch.tensor(sum(rows, []), device="cuda")
    o = torch.full((220, 4, 128), float("nan"), dtype=TYPES[type][1], device="cuda")
    p = Case([146, 66], H=4, G=2, dk=128, dv=128, type=type, decay="reset")
    p.q, p.k, p.v, p.g = (a[first].contiguous() for a in (c.q, c.k, c.v, c.g))
    p.state = c.state
    o[first] = p.prefill()
    for i in range(keep):
        at = torch.tensor([c.begin[1] - keep + i, c.begin[2] - keep + i], device="cuda")
        s = Case([1, 1], H=4, G=2, dk=128, dv=128, type=type)
        s.q, s.k, s.v, s.g = (a[at].contiguous() for a in (c.q, c.k, c.v, c.g))
        s.state = c.state
        o[at] = s.step()
    c.check(o, c.state, want)


@pytest.mark.parametrize("type", list(TYPES))
def test_equal_sequences_without_offsets(type):
    c = Case([70, 70, 70], dk=64, dv=128, type=type)
    want = c.want()
    c.check(c.prefill(offsets=None), c.state, want)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("n", [20, 150])
def test_uncovered_and_padded_rows_are_not_written(type, n):
    """Offsets that leave tokens out and an o with padding: only covered rows change."""
    c = Case([n, n], H=2, dk=64, dv=64, type=type, decay="head")
    want = c.want()
    off = torch.tensor([5, n, 2 * n - 7], dtype=torch.int32, device="cuda")
    buf = torch.full((2 * n, 2 * 64 + 32), 7.0, dtype=TYPES[type][1], device="cuda")
    c.prefill(offsets=off, o=buf, o_stride=160)
    assert (buf[:, 128:] == 7).all() and (buf[:5] == 7).all() and (buf[2 * n - 7:] == 7).all()
    assert torch.isfinite(buf).all() and not (buf[5:2 * n - 7, :128] == 7).all(1).any()
    del want


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_bad_offsets_stay_in_bounds(type):
    """Offsets below 0, past the end and descending are clamped: the others' results stand."""
    c = Case([40, 100, 30], dk=64, dv=64, type=type, n_states=4, slots=[0, 1, 2])
    want = c.want()
    off = torch.tensor([-5, 40, 140, 1 << 30], dtype=torch.int32, device="cuda")  # clamps to 0, 40, 140, 170
    c.check(c.prefill(offsets=off), c.state, want)
    c = Case([40, 100, 30], dk=64, dv=64, type=type, n_states=4, slots=[0, 1, 2])
    before = c.state.clone()
    off = torch.tensor([0, 40, 20, 20], dtype=torch.int32, device="cuda")  # 40 tokens, then two empty ones
    o = c.prefill(offsets=off)
    c.check(o[:40], c.state[:1], tuple(w[:m] for w, m in zip(c.want(before), (40, 1, 40, 1))))
    assert torch.equal(c.state[1:], before[1:]) and torch.isnan(o[40:]).all()


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "g"])
def test_non_finite_does_not_reach_back(type, bad, where):
    """A NaN or an infinity at one token reaches no earlier token, no other sequence or head."""
    if where == "g" and bad > 0:
        bad = float("nan")
    c = Case([200, 90], H=2, dk=128, dv=128, type=type)
    want = c.want()
    t = 170
    if where == "g":
        c.g[t, 1] = bad
    else:
        getattr(c, where)[t, 1, 5] = bad
    o = c.prefill()
    ok = np.ones((290, 2), bool)
    ok[t:200, 1] = False
    c.check(torch.where(torch.from_numpy(ok).cuda()[..., None], o, 0), torch.where(
        torch.tensor([[True, False], [True, True]], device="cuda")[..., None, None], c.state, 0),
        tuple(np.where(m[(...,) + (None,) * (w.ndim - 2)], w, 0) for w, m in
              zip(want, (ok, np.array([[1, 0], [1, 1]], bool), ok, np.array([[1, 0], [1, 1]], bool)))))
    if where == "q":
        assert not torch.isfinite(o[t, 1]).all() and torch.isfinite(o[t + 1:200, 1]).all()
    elif where == "v":  # only that value's channel
        assert not torch.isfinite(o[t:200, 1, 5]).any() and torch.isfinite(o[t:200, 1, 6:]).all()
        assert not torch.isfinite(c.state[0, 1, :, 5]).any() and torch.isfinite(c.state[0, 1, :, 6:]).all()
    else:
        assert not torch.isfinite(o[t:200, 1]).any()


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_value_early_in_a_long_prompt(type, bad):
    """A value of v that is not finite near the start of a prompt that is cut into several units
    keeps to its channel all the way, outputs and state."""
    c = Case([700, 130], H=2, dk=128, dv=128, type=type, decay="head")
    c.v[65, 1, 5] = 0
    want = c.want()
    c.v[65, 1, 5] = bad
    o = c.prefill()
    ok = torch.ones(830, 2, 128, dtype=torch.bool, device="cuda")
    ok[65:700, 1, 5] = False
    oks = torch.ones(2, 2, 128, 128, dtype=torch.bool, device="cuda")
    oks[0, 1, :, 5] = False
    assert not torch.isfinite(o[65:700, 1, 5]).any() and not torch.isfinite(c.state[0, 1, :, 5]).any()
    m, ms = ok.cpu().numpy(), oks.cpu().numpy()
    c.check(torch.where(ok, o, 0), torch.where(oks, c.state, 0),
            tuple(np.where(x, w, 0) for x, w in zip((m, ms, m, ms), want)))


@pytest.mark.parametrize("type", list(TYPES))
def test_many_sequences_few_of_them_long(type):
    """More sequences than a CTA counts in one go, some cut into units, some empty or inactive."""
    rng = np.random.default_rng(12)
    lens = [int(n) for n in rng.integers(0, 4, 300)]
    for b, n in ((3, 513), (70, 300), (255, 140), (256, 129), (290, 128), (299, 400)):
        lens[b] = n
    slots = [int(x) for x in rng.permutation(310)[:300]]
    for b in (5, 70, 120, 290):
        slots[b] = -1 - b
    c = Case(lens, H=2, G=1, dk=64, dv=32, type=type, decay="reset", n_states=310, slots=slots)
    want = c.want()
    c.check(c.prefill(), c.state, want)


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("lens,H", [([450, 450], 2), ([1300], 30), ([700, 60, 500], 24)])
def test_long_prompts(lens, H, type):
    """Prompts of several units, with few and with many heads, with and without offsets."""
    c = Case(lens, H=H, G=H // 2, dk=128, dv=64, type=type, decay="token")
    first = c.state.clone()
    want = c.want()
    c.check(c.prefill(), c.state, want)
    if len(set(lens)) == 1:
        c.state.copy_(first)
        c.check(c.prefill(offsets=None), c.state, want)


def test_one_workspace_for_calls_of_any_size():
    """A workspace that other calls have used gives what a fresh one gives."""
    ws = None
    for lens, H, type in (([900, 200], 4, "bf16"), ([500], 2, "f32"), ([2000], 3, "f16"), ([900, 200], 4, "bf16")):
        c = Case(lens, H=H, dk=128, dv=128, type=type)
        want, cfg = c.want(), c.cfg()
        if ws is None:
            ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
        o = torch.empty(sum(lens), H, 128, dtype=TYPES[type][1], device="cuda")
        st = torch.cuda.current_stream()
        ffn.check(ffn.moe_linattn_prefill(c.q, c.k, c.v, c.g, c.offsets, None, cfg, c.state, o, ws, ws.numel(), st))
        ffn.check(ffn.moe_workspace_status(ws, st))
        c.check(o, c.state, want)


def test_fresh_state_ignores_what_was_there():
    c = Case([80, 0, 30], dk=64, dv=64, type="bf16", fresh=True)
    want = c.want()
    c.state.fill_(float("nan"))
    c.check(c.prefill(), c.state, want)
    s = Case([1, 1], dk=64, dv=64, type="f32", fresh=True)
    want = s.want()
    s.state.fill_(float("nan"))
    s.check(s.step(), s.state, want)


@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_side_stream_and_graph(type):
    """Prompts on a side stream, then steps replayed from a captured graph."""
    c = Case([300, 100], H=4, dk=128, dv=128, type=type)
    want = c.want()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o = c.prefill(stream=st)
    st.synchronize()
    c.check(o, c.state, want)
    s = Case([1] * 6, H=4, dk=128, dv=128, type=type)
    first = s.state.clone()
    o = torch.zeros(6, 4, 128, dtype=TYPES[type][1], device="cuda")
    cfg = s.cfg()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            ffn.check(ffn.moe_linattn_step(s.q, s.k, s.v, s.g, s.slots, cfg, s.state, o, torch.cuda.current_stream()))
    s.state.copy_(first)
    g.replay()
    torch.cuda.synchronize()
    st3 = first
    for _ in range(3):
        ro, rs, ao, as_ = s.want(st3)
        st3 = torch.from_numpy(rs).cuda()
    s.check(o, s.state, (ro, rs, ao, as_))


def test_states_past_32_bits():
    """A pool of more than 2^31 values: the last state is read and written where it is."""
    H, d = 32, 128
    n = (1 << 31) // (H * d * d) + 2
    c = Case([150], H=H, dk=d, dv=d, type="bf16")
    s = Case([1], H=H, dk=d, dv=d, type="bf16")
    pool = torch.empty(n, H, d, d, device="cuda")
    pool[n - 1] = c.state[0]
    want = c.want()
    c.slots = s.slots = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    c.state = s.state = pool
    c.n_states = s.n_states = n
    o = c.prefill()
    c.check(o, pool[n - 1:], want)
    s.slots, s.n_states, s.state = None, 1, pool[n - 1:]
    want = s.want()
    s.slots, s.n_states, s.state = c.slots, n, pool
    s.check(s.step(), pool[n - 1:], want)


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("lens,H", [([448] * 8, 10), ([512] * 3 + [1, 0, 512], 16), ([1500, 60, 0, 200], 30), ([33] * 5, 16),
                                    ([200] * 4, 2)],
                         ids=["equal", "some-empty", "one-long", "short", "few-heads"])
def test_whole_or_cut(lens, H, offsets, type):
    """Calls around the point where sequences are cut into units, and around the walk's."""
    if not offsets and len(set(lens)) > 1:
        lens = [max(lens)] * 3
    c = Case(lens, H=H, dk=64, dv=40, type=type, decay="reset")
    want = c.want()
    c.check(c.prefill(**({} if offsets else {"offsets": None})), c.state, want)


def test_many_sequences_with_one_length():
    """More sequences than one round of the search takes, which the offsets leave whole."""
    c = Case([130] * 300, H=1, dk=32, dv=32, type="bf16")
    want = c.want()
    c.check(c.prefill(), c.state, want)
